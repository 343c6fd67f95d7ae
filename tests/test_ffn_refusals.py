"""What the dense feed-forward entry points refuse, at the C boundary and in the
binding, without a GPU (nothing is launched)."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.environ.get("Q4MOE_ABI_LIB") or os.path.join(ROOT, "moe_experts_amd", "libq4moe.so")
P = 1 << 20  # never dereferenced: every call below fails its checks
EINVAL, ESHAPE, EALIGN, EWS, EBIG = -1, -2, -3, -4, -6


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        from moe_experts_amd import build
        build.build()
    L = ctypes.CDLL(LIB)
    p, i, z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    for n, a in (("q4_0_glu", [p] * 4 + [i] * 4), ("q4_0_glu_gemm", [p] * 6 + [i] * 4),
                 ("q4_0_glu_backward", [p] * 6 + [i] * 4), ("q4_0_gemm_backward", [p] * 3 + [i] * 3),
                 ("q4_0_gemv_lora", [p] * 7 + [i] * 5), ("q4_0_gemm_lora", [p] * 7 + [i] * 5)):
        getattr(L, n).argtypes = a + [p, z, p]
        f = getattr(L, n + "_workspace_bytes")
        f.restype, f.argtypes = z, [i] * (4 if n.endswith("lora") else 3)
    return L


#: name: (pointers, sizes of a valid call). Sizes: M, N, K, then act or R and L.
VALID = {
    "q4_0_glu": (4, (2, 64, 96, 0)),
    "q4_0_glu_gemm": (6, (40, 128, 64, 1)),
    "q4_0_glu_backward": (6, (40, 128, 64, 0)),
    "q4_0_gemm_backward": (3, (40, 128, 64)),
    "q4_0_gemv_lora": (7, (2, 64, 96, 16, 3)),
    "q4_0_gemm_lora": (7, (40, 128, 64, 16, 3)),
}
DECODE = ("q4_0_glu", "q4_0_gemv_lora")
BIG = 1 << 40  # a workspace size that is large enough


def call(lib, name, ptrs=None, sizes=None, ws=P, ws_bytes=BIG):
    n, s = VALID[name]
    ptrs = [P] * n if ptrs is None else ptrs
    return getattr(lib, name)(*ptrs, *(s if sizes is None else sizes), ws, ws_bytes, None)


def with_size(name, at, v):
    s = list(VALID[name][1])
    s[at] = v
    return s


@pytest.mark.parametrize("name", VALID)
def test_null_pointers(lib, name):
    n = VALID[name][0]
    for i in range(n):
        ptrs = [P] * n
        ptrs[i] = None
        assert call(lib, name, ptrs) == EINVAL


def test_g_and_u_come_together(lib):
    # both null is the call without them: it gets as far as the workspace
    assert call(lib, "q4_0_glu_gemm", [P, P, P, P, None, P]) == EINVAL
    assert call(lib, "q4_0_glu_gemm", [P, P, P, P, P, None]) == EINVAL
    sizes = (40, 128, 2048, 0)
    assert call(lib, "q4_0_glu_gemm", [P, P, P, P, None, None], sizes, None, 0) == EWS


@pytest.mark.parametrize("name", VALID)
def test_sizes(lib, name):
    for at in range(3):
        for v in (0, -1):
            assert call(lib, name, sizes=with_size(name, at, v)) == EINVAL
    block = 32 if name in DECODE else 64
    assert call(lib, name, sizes=with_size(name, 1, block + 16)) == ESHAPE
    if name in DECODE:
        assert call(lib, name, sizes=with_size(name, 0, 9)) == ESHAPE
    else:
        assert call(lib, name, sizes=with_size(name, 1, 96)) == ESHAPE
        assert call(lib, name, sizes=with_size(name, 2, 96)) == ESHAPE
        assert call(lib, name, sizes=with_size(name, 0, 1 << 30)) == EBIG
    s = with_size(name, 1, 1 << 20)
    s[2] = 1 << 20
    assert call(lib, name, sizes=s) == EBIG


@pytest.mark.parametrize("name", ["q4_0_glu", "q4_0_glu_gemm", "q4_0_glu_backward"])
def test_unknown_activation(lib, name):
    for v in (-1, 2):
        assert call(lib, name, sizes=with_size(name, 3, v)) == EINVAL


@pytest.mark.parametrize("name", ["q4_0_gemv_lora", "q4_0_gemm_lora"])
def test_ranks_and_adapters(lib, name):
    for v, code in ((0, EINVAL), (-8, EINVAL), (4, ESHAPE), (12, ESHAPE), (136, ESHAPE)):
        assert call(lib, name, sizes=with_size(name, 3, v)) == code
    for v in (0, -1):
        assert call(lib, name, sizes=with_size(name, 4, v)) == EINVAL
    if name == "q4_0_gemv_lora":
        assert call(lib, name, sizes=with_size(name, 2, 12)) == ESHAPE


#: bytes of alignment of each pointer, in order
ALIGN = {
    "q4_0_glu": (4, 2, 2, 4),
    "q4_0_glu_gemm": (16, 2, 2, 16, 16, 16),
    "q4_0_glu_backward": (16, 16, 16, 2, 2, 16),
    "q4_0_gemm_backward": (16, 2, 16),
    "q4_0_gemv_lora": (16, 2, 16, 16, 4, 4, 4),
    "q4_0_gemm_lora": (16, 2, 16, 16, 4, 4, 16),
}


@pytest.mark.parametrize("name", VALID)
def test_alignment(lib, name):
    for i, a in enumerate(ALIGN[name]):
        ptrs = [P] * len(ALIGN[name])
        ptrs[i] = P + a // 2
        assert call(lib, name, ptrs) == EALIGN


@pytest.mark.parametrize("name", VALID)
def test_workspace(lib, name):
    s = list(VALID[name][1])
    s[1], s[2] = 1024, 2048
    need = getattr(lib, name + "_workspace_bytes")(*s[:4 if name.endswith("lora") else 3])
    assert need > 0
    assert call(lib, name, sizes=s, ws=None, ws_bytes=0) == EWS
    assert call(lib, name, sizes=s, ws_bytes=need - 1) == EWS
    assert call(lib, name, sizes=s, ws=P + 16, ws_bytes=need) == EALIGN


@pytest.mark.parametrize("name", VALID)
def test_workspace_sizes_over_extreme_shapes(lib, name):
    """Sizing never fails and is 0 for what the entry point refuses."""
    f = getattr(lib, name + "_workspace_bytes")
    vals = (-1, 0, 1, 8, 9, 32, 64, 96, 4096, 65536, (1 << 31) - 64, (1 << 31) - 1)
    for M in vals:
        for N in vals:
            for K in vals:
                for R in ((-8, 8, 12, 128, 136) if name.endswith("lora") else (None,)):
                    args = (M, N, K) if R is None else (M, N, K, R)
                    got = f(*args)
                    bad = min(M, N, K) <= 0 or N % 32 or (R is not None and R not in (8, 128))
                    bad = bad or (M > 8 if name in DECODE else N % 64 or K % 64)
                    if bad:
                        assert got == 0, args


def test_binding_refuses_what_the_library_cannot_see():
    import moe_experts_amd as q4
    K, N, M, R, L = 64, 64, 2, 8, 2
    W = torch.zeros(K * (N // 32) * 18, dtype=torch.uint8)
    x, X = torch.zeros(M, K), torch.zeros(M, K, dtype=torch.float16)
    with pytest.raises(ValueError, match="device tensor"):
        q4.q4_0_glu(x, W, W, N)
    with pytest.raises(ValueError, match="act must be"):
        q4.q4_0_glu(x, W, W, N, act="tanh")
    with pytest.raises(ValueError, match="multiple of 32"):
        q4.q4_0_glu(x, W, W, 48)
    with pytest.raises(ValueError, match="multiple of 64"):
        q4.q4_0_glu_gemm(X, W, W, 96)
    with pytest.raises(ValueError, match="together"):
        q4.q4_0_glu_gemm(X, W, W, N, G=X)
    with pytest.raises(ValueError, match=r"\[M, K\]"):
        q4.q4_0_glu_gemm(X[0], W, W, N)
    with pytest.raises(ValueError, match=r"\[L, R, K\]"):
        q4.q4_0_gemv_lora(x, W, N, X, X, torch.zeros(M, dtype=torch.int32), torch.zeros(L))
    with pytest.raises(ValueError, match="device tensor"):
        q4.q4_0_gemm_backward(X.bfloat16(), W, K)


def calls_that_want_gradients():
    """(entry point, its inputs that can require a gradient, the call)."""
    import moe_experts_amd as q4
    K, N, M, R, L = 64, 64, 2, 8, 2
    W = torch.zeros(K * (N // 32) * 18, dtype=torch.uint8)
    x, X = torch.zeros(M, K), torch.zeros(M, K, dtype=torch.float16)
    dY, G, U = torch.zeros(M, N).bfloat16(), torch.zeros(M, N).half(), torch.zeros(M, N).half()
    A, Bl = torch.zeros(L, R, K).half(), torch.zeros(L, N, R).half()
    ids, s = torch.zeros(M, dtype=torch.int32), torch.zeros(L)
    return [
        ("q4_0_glu", (x,), lambda: q4.q4_0_glu(x, W, W, N)),
        ("q4_0_glu_gemm", (X,), lambda: q4.q4_0_glu_gemm(X, W, W, N)),
        ("q4_0_glu_backward", (dY, G, U), lambda: q4.q4_0_glu_backward(dY, G, U, W, W, K)),
        ("q4_0_gemm_backward", (dY,), lambda: q4.q4_0_gemm_backward(dY, W, K)),
        ("q4_0_gemv_lora", (x, A, Bl, s), lambda: q4.q4_0_gemv_lora(x, W, N, A, Bl, ids, s)),
        ("q4_0_gemm_lora", (X, A, Bl, s), lambda: q4.q4_0_gemm_lora(X, W, N, A, Bl, ids, s)),
    ]


@pytest.mark.parametrize("which", range(6), ids=lambda i: calls_that_want_gradients()[i][0])
def test_a_gradient_that_would_be_lost_is_refused(which, monkeypatch):
    """The calls record nothing for torch's autograd: on inputs that require a gradient their
    results would quietly have none. (CPU tensors; the check of the device and the library's call
    are stand-ins.)"""
    from moe_experts_amd import binding
    ran = []
    monkeypatch.setattr(binding, "_dev", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(binding, "_run", lambda *a: ran.append(a))
    name, inputs, call = calls_that_want_gradients()[which]
    for t in inputs:
        t.requires_grad_()
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        assert not ran
        # without recording, what a Function's forward runs under too, the call is made
        for off in (torch.no_grad(), torch.inference_mode()):
            with off:
                call()
            assert ran.pop()
        t.requires_grad_(False)
    call()
    assert ran


def test_plan_over_extreme_shapes(lib):
    """The plan of a shape fails as its call does, and else names a kernel."""
    i, ptr = ctypes.c_int, ctypes.POINTER(ctypes.c_int)
    lib.q4_0_ffn_plan.argtypes = [i] * 4 + [ptr] * 3
    rows, splits, steps = (i(7) for _ in range(3))
    refs = [ctypes.byref(v) for v in (rows, splits, steps)]
    for form in (-1, 4):
        assert lib.q4_0_ffn_plan(form, 65, 64, 64, *refs) == EINVAL
    for at in range(3):
        assert lib.q4_0_ffn_plan(0, 65, 64, 64, *refs[:at], None, *refs[at + 1:]) == EINVAL
    assert (rows.value, splits.value, steps.value) == (7, 7, 7)
    names = ("q4_0_glu_gemm", "q4_0_glu_backward", "q4_0_gemm_backward", "q4_0_gemm_lora")
    vals = (-1, 0, 1, 64, 65, 96, 4096, 65536, (1 << 31) - 64, (1 << 31) - 1)
    for form, name in enumerate(names):
        for M in vals:
            for N in vals:
                for K in vals:
                    rc = lib.q4_0_ffn_plan(form, M, N, K, *refs)
                    s = [M, N, K] + list(VALID[name][1][3:])
                    if rc == 0:
                        assert rows.value in (0, 64, 128, 256) and splits.value >= 1
                        assert steps.value >= 1
                    else:  # the call's own check, which comes before anything is enqueued
                        assert call(lib, name, sizes=s) == rc
