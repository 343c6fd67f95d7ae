"""What the 8-bit entry points refuse, at the C boundary and in the binding, without
a GPU (nothing is launched)."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.environ.get("Q4MOE_ABI_LIB") or os.path.join(ROOT, "moe_experts_amd", "libq4moe.so")
P = 1 << 20  # never dereferenced: every call below fails its checks
EINVAL, ESHAPE, EALIGN, EWS, EBIG = -1, -2, -3, -4, -6
BIG = 1 << 40  # a workspace size that is large enough
MAX_K = 131056


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        from moe_experts_amd import build
        build.build()
    L = ctypes.CDLL(LIB)
    p, i, z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    for n, ptrs in (("i8_gemv", 4), ("i8_gemm", 5), ("i8_gemm_backward", 4),
                    ("i8_gemm_backward_weight", 4)):
        getattr(L, n).argtypes = [p] * ptrs + [i] * (4 if n == "i8_gemm" else 3) + [p, z, p]
        f = getattr(L, n + "_workspace_bytes")
        f.restype, f.argtypes = z, [i] * 3
    L.i8_quantize.argtypes = [p, i, p, p, i, i, p]
    L.i8_dequantize.argtypes = [p, p, p, i, i, i, p]
    return L


#: name: pointers' alignments in order, sizes (M, N, K) of a valid call that needs a workspace
VALID = {
    "i8_gemv": ((4, 16, 4, 16), (8, 64, 11008)),
    "i8_gemm": ((16, 4, 16, 4, 16), (130, 64, 65536)),
    "i8_gemm_backward": ((16, 16, 4, 16), (40, 4096, 64)),
    "i8_gemm_backward_weight": ((16, 16, 4, 16), (4096, 128, 64)),
}


def call(lib, name, ptrs=None, sizes=None, ws=P, ws_bytes=BIG, type_=1):
    align, s = VALID[name]
    ptrs = [P] * len(align) if ptrs is None else ptrs
    extra = [type_] if name == "i8_gemm" else []
    return getattr(lib, name)(*ptrs, *extra, *(s if sizes is None else sizes), ws, ws_bytes, None)


def with_size(name, at, v):
    s = list(VALID[name][1])
    s[at] = v
    return s


@pytest.mark.parametrize("name", VALID)
def test_null_pointers(lib, name):
    for i in range(len(VALID[name][0])):
        ptrs = [P] * len(VALID[name][0])
        ptrs[i] = None
        assert call(lib, name, ptrs) == EINVAL


@pytest.mark.parametrize("name", VALID)
def test_sizes(lib, name):
    for at in range(3):
        for v in (0, -1):
            assert call(lib, name, sizes=with_size(name, at, v)) == EINVAL
    for v in (4, 12, 68):
        assert call(lib, name, sizes=with_size(name, 1, v)) == ESHAPE
    for v in (8, 24, 4100, MAX_K + 16):
        assert call(lib, name, sizes=with_size(name, 2, v)) == ESHAPE
    if name == "i8_gemv":
        assert call(lib, name, sizes=with_size(name, 0, 9)) == ESHAPE
    else:
        assert call(lib, name, sizes=with_size(name, 0, (1 << 31) - 1)) == EBIG
    s = with_size(name, 1, 1 << 15)
    s[2] = 1 << 16  # W is 2 GiB
    assert call(lib, name, sizes=s) == EBIG


def test_results_of_two_gigabytes(lib):
    # 65544 x 16384 results: 2^30 and a little more, too many for 2 bytes and for 4
    for M, N, K, type_, code in ((65544, 16384, 16, 1, EBIG), (65528, 16384, 16, 1, EALIGN),
                                 (65528, 16384, 16, 2, EALIGN), (65528, 16384, 16, 0, EBIG)):
        assert call(lib, "i8_gemm", [P, P, P, P, P + 8], (M, N, K), type_=type_) == code
    # dX of M x K, dW of N x K, bf16
    assert call(lib, "i8_gemm_backward", sizes=(16384, 8, 65552)) == EBIG
    assert call(lib, "i8_gemm_backward_weight", sizes=(8, 16384, 65552)) == EBIG
    # x of i8_gemv is fp32: 8 x K never reaches 2 GiB within the other limits
    assert call(lib, "i8_gemv", [P, P, P, P + 8], (8, 8, MAX_K)) == EALIGN


def test_unknown_types(lib):
    for t in (-1, 3):
        assert call(lib, "i8_gemm", type_=t) == EINVAL
        assert lib.i8_quantize(P, t, P, P, 4, 4, None) == EINVAL
        assert lib.i8_dequantize(P, P, P, t, 4, 4, None) == EINVAL


@pytest.mark.parametrize("name", VALID)
def test_alignment(lib, name):
    align = VALID[name][0]
    for i, a in enumerate(align):
        ptrs = [P] * len(align)
        ptrs[i] = P + a // 2
        assert call(lib, name, ptrs) == EALIGN


@pytest.mark.parametrize("name", VALID)
def test_workspace(lib, name):
    s = VALID[name][1]
    need = getattr(lib, name + "_workspace_bytes")(*s)
    assert need > 0
    assert call(lib, name, ws=None, ws_bytes=0) == EWS
    assert call(lib, name, ws_bytes=need - 1) == EWS
    assert call(lib, name, ws=P + 16, ws_bytes=need) == EALIGN


@pytest.mark.parametrize("name", VALID)
def test_workspace_sizes_over_extreme_shapes(lib, name):
    """Sizing never fails and is 0 for what the entry point refuses."""
    f = getattr(lib, name + "_workspace_bytes")
    vals = (-1, 0, 1, 8, 9, 16, 64, 72, 130, 4096, 65536, MAX_K, MAX_K + 16, (1 << 27) - 8,
            (1 << 31) - 64, (1 << 31) - 1)
    for M in vals:
        for N in vals:
            for K in vals:
                got = f(M, N, K)
                bad = min(M, N, K) <= 0 or N % 8 or K % 16 or K > MAX_K
                bad = bad or N * K >= 1 << 31 or M * K >= 1 << 31 or 2 * M * N >= 1 << 31
                if bad or (name == "i8_gemv" and M > 8):
                    assert got == 0, (M, N, K)


def test_plan_over_extreme_shapes(lib):
    """The plan of a shape fails as its call does, and else names a kernel."""
    i, ptr = ctypes.c_int, ctypes.POINTER(ctypes.c_int)
    lib.i8_gemm_plan.argtypes = [i] * 4 + [ptr] * 4
    out = [i(7) for _ in range(4)]
    refs = [ctypes.byref(v) for v in out]
    for form in (-1, 3):
        assert lib.i8_gemm_plan(form, 65, 64, 64, *refs) == EINVAL
    for at in range(4):
        assert lib.i8_gemm_plan(0, 65, 64, 64, *refs[:at], None, *refs[at + 1:]) == EINVAL
    assert [v.value for v in out] == [7] * 4
    vals = (-1, 0, 1, 8, 16, 17, 64, 72, 4096, 65536, MAX_K, MAX_K + 16, (1 << 27) - 8, (1 << 31) - 1)
    for form, name in enumerate(("i8_gemm", "i8_gemm_backward", "i8_gemm_backward_weight")):
        for M in vals:
            for N in vals:
                for K in vals:
                    rc = lib.i8_gemm_plan(form, M, N, K, *refs)
                    if rc != 0:  # the call's own check, which comes before anything is enqueued
                        assert call(lib, name, sizes=(M, N, K)) == rc
                        continue
                    rows, cols, splits, steps = (v.value for v in out)
                    assert splits >= 1 and steps >= 1 and (rows == 0) == (cols == 0)
                    depth = K if form == 0 else 2 * (N if form == 1 else M)
                    total = (depth + 127) // 128
                    assert (splits - 1) * steps < total <= splits * steps  # none is empty


def test_rows(lib):
    q, d = lib.i8_quantize, lib.i8_dequantize
    for bad in ((None, P, P), (P, None, P), (P, P, None)):
        assert q(bad[0], 1, bad[1], bad[2], 4, 4, None) == EINVAL
        assert d(bad[0], bad[1], bad[2], 1, 4, 4, None) == EINVAL
    for M, K in ((0, 4), (4, 0), (-1, 4), (4, -1)):
        assert q(P, 1, P, P, M, K, None) == EINVAL
        assert d(P, P, P, 1, M, K, None) == EINVAL
    for t, M, K, code in ((1, 1 << 15, 1 << 15, EBIG), (0, 1 << 15, 1 << 14, EBIG),
                          (2, 1 << 30, 1, EBIG), (1, 1 << 15, (1 << 15) - 1, EALIGN)):
        assert q(P, t, P, P + 2, M, K, None) == code
        assert d(P, P + 2, P, t, M, K, None) == code
    for t, off in ((0, 2), (1, 1), (2, 1)):
        assert q(P + off, t, P, P, 4, 4, None) == EALIGN
        assert d(P, P, P + off, t, 4, 4, None) == EALIGN


def test_binding_refuses_what_the_library_cannot_see():
    import tests.built  # noqa: F401
    import moe_experts_amd as q4
    M, N, K = 3, 8, 32
    x = torch.zeros(M, K)
    X, W = torch.zeros(M, K, dtype=torch.int8), torch.zeros(N, K, dtype=torch.int8)
    sx, sw = torch.zeros(M), torch.zeros(N)
    dY = torch.zeros(M, N, dtype=torch.bfloat16)
    for call_ in (lambda: q4.i8_quantize(x), lambda: q4.i8_dequantize(X, sx),
                  lambda: q4.i8_gemv(x, W, sw), lambda: q4.i8_gemm(X, sx, W, sw),
                  lambda: q4.i8_gemm_backward(dY, W, sw),
                  lambda: q4.i8_gemm_backward_weight(dY, X, sx)):
        with pytest.raises(ValueError, match="device tensor"):
            call_()
    with pytest.raises(TypeError, match="dtype"):
        q4.i8_quantize(x.double())
    with pytest.raises(TypeError, match="dtype"):
        q4.i8_dequantize(X, sx, dtype=torch.float64)
    with pytest.raises(TypeError, match="dtype"):
        q4.i8_gemm(X, sx, W, sw, dtype=torch.int32)
    with pytest.raises(ValueError, match=r"\[M, K\]"):
        q4.i8_quantize(x[0])
    with pytest.raises(ValueError, match=r"\[M, K\]"):
        q4.i8_dequantize(X[0], sx)
    with pytest.raises(ValueError, match=r"\[N, K\]"):
        q4.i8_gemv(x, W[:, :16], sw)
    with pytest.raises(ValueError, match=r"\[N, K\]"):
        q4.i8_gemm(X, sx, W.reshape(-1), sw)
    with pytest.raises(ValueError, match=r"\[N, K\]"):
        q4.i8_gemm_backward(dY, W.reshape(-1), sw)
    with pytest.raises(ValueError, match=r"\[M, K\]"):
        q4.i8_gemm_backward_weight(dY, X[:2], sx)


def test_a_gradient_that_would_be_lost_is_refused(monkeypatch):
    """On inputs that require a gradient the calls' results would quietly have none. (CPU tensors;
    the check of the device and the library's calls are stand-ins.)"""
    import tests.built  # noqa: F401
    import moe_experts_amd as q4
    from moe_experts_amd import binding
    ran = []
    monkeypatch.setattr(binding, "_dev", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(binding, "_run", lambda *a: ran.append(a))
    monkeypatch.setattr(binding, "_call", lambda *a: ran.append(a))
    M, N, K = 3, 8, 32
    x = torch.zeros(M, K)
    X, W = torch.zeros(M, K, dtype=torch.int8), torch.zeros(N, K, dtype=torch.int8)
    sx, sw = torch.zeros(M), torch.zeros(N)
    dY = torch.zeros(M, N, dtype=torch.bfloat16)
    for inputs, call_ in (((x,), lambda: q4.i8_quantize(x)),
                          ((sx,), lambda: q4.i8_dequantize(X, sx)),
                          ((x, sw), lambda: q4.i8_gemv(x, W, sw)),
                          ((sx, sw), lambda: q4.i8_gemm(X, sx, W, sw)),
                          ((dY, sw), lambda: q4.i8_gemm_backward(dY, W, sw)),
                          ((dY, sx), lambda: q4.i8_gemm_backward_weight(dY, X, sx))):
        for t in inputs:
            t.requires_grad_()
            with pytest.raises(ValueError, match="requires a gradient"):
                call_()
            assert not ran
            with torch.no_grad():
                call_()
            assert ran.pop()
            t.requires_grad_(False)
        call_()
        assert ran.pop()


WIDE = (1 << 32) + 64  # loses its upper bits where a C int is taken


@pytest.mark.parametrize("at", range(3))
@pytest.mark.parametrize("name", VALID)
def test_sizes_that_are_no_c_ints(name, at):
    """Not the shape that their lower 32 bits would be."""
    import tests.built  # noqa: F401  (binding loads the library)
    from moe_experts_amd import binding
    sizes = [64, 64, 64]
    sizes[at] = WIDE
    with pytest.raises(binding.Q4Error) as e:
        getattr(binding, name + "_workspace_bytes")(*sizes)
    assert e.value.status == EBIG
    if name in binding.I8_FORMS:
        with pytest.raises(binding.Q4Error) as e:
            binding.i8_gemm_plan(name, *sizes)
        assert e.value.status == EBIG


def test_tensors_whose_sizes_are_no_c_ints():
    """Tensors without memory: the sizes are refused first."""
    import tests.built  # noqa: F401
    from moe_experts_amd import binding as b

    def t(rows, cols, dtype):
        return torch.empty((rows, cols) if cols else (rows,), dtype=dtype, device="meta")

    i8, f32, f16, bf16 = torch.int8, torch.float32, torch.float16, torch.bfloat16
    for m, k in ((WIDE, 1), (1, WIDE)):
        with pytest.raises(b.Q4Error) as e:
            b.i8_quantize(t(m, k, f16))
        assert e.value.status == EBIG
        with pytest.raises(b.Q4Error) as e:
            b.i8_dequantize(t(m, k, i8), t(m, 0, f32))
        assert e.value.status == EBIG
    for at in range(3):
        s = [1, 8, 16]
        s[at] = WIDE
        M, N, K = s
        sx, sw = t(M, 0, f32), t(N, 0, f32)
        for call in (lambda: b.i8_gemv(t(M, K, f32), t(N, K, i8), sw),
                     lambda: b.i8_gemm(t(M, K, i8), sx, t(N, K, i8), sw),
                     lambda: b.i8_gemm_backward(t(M, N, bf16), t(N, K, i8), sw),
                     lambda: b.i8_gemm_backward_weight(t(M, N, bf16), t(M, K, i8), sx)):
            with pytest.raises(b.Q4Error) as e:
                call()
            assert e.value.status == EBIG
