"""Dense feed-forward operators over Q4_0 weights against 64-bit references,
element by element within bounds counted from the roundings (tests/ffn_ref.py)."""
import numpy as np
import pytest
import torch

from moe_experts_amd import datagen
from tests import ffn_ref as ref
from tests.gpu_util import dev, guarded, guarded_ws, guards_intact, to_dev, ws_guards_intact

pytestmark = pytest.mark.gpu


def weights(seed, K, N, **kw):
    return datagen.q4_0_random(seed, K, N, **kw)


def host(t):
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16().to(dev())


def values(t):
    return t.float().cpu().numpy()


def gradient(seed, M, N):
    r = datagen.rng(seed)
    size = np.exp(r.standard_normal((M, 1)) * 2 - 9)
    return bf16(r.standard_normal((M, N)) * size)


def adapters(seed, L, R, K, N):
    r = datagen.rng(seed)
    A = (r.standard_normal((L, R, K)) / np.sqrt(K)).astype(np.float16)
    Bl = (r.standard_normal((L, N, R)) * 0.1).astype(np.float16)
    return A, Bl, r.uniform(-2, 2, L).astype(np.float32)


def nan_ws(nbytes):
    """A guarded workspace whose bytes read as NaN in fp16 and fp32."""
    return guarded_ws(nbytes, fill=0xFF)


# ------------------------------------------------------------------ gated block, decode
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,K,N", [
    (1, 1, 32), (1, 37, 32), (1, 300, 512), (1, 2048, 512), (2, 1000, 544), (3, 64, 32),
    (3, 513, 160), (4, 1024, 256), (5, 777, 96), (8, 2048, 512), (8, 1030, 1056), (7, 1, 64),
    (3, 31, 32), (4, 33, 288), (3, 262200, 32),
])
def test_glu(M, K, N, act):
    from moe_experts_amd import q4_0_glu, q4_0_glu_workspace_bytes
    x, Wg, Wu = datagen.activations(1, M, K), weights(2, K, N), weights(3, K, N)
    full, h = guarded(M * N)
    need = q4_0_glu_workspace_bytes(M, N, K)
    wfull, ws = nan_ws(need)
    q4_0_glu(to_dev(x), to_dev(Wg), to_dev(Wu), N, act=act, h=h.view(M, N), ws=ws)
    ref.check(host(h).reshape(M, N), ref.glu(x, Wg, Wu, act))
    assert guards_intact(full, M * N) and ws_guards_intact(wfull, need, 0xFF)


def test_glu_odd_matrix_addresses():
    """Both matrices at 2-byte aligned addresses, then only the second: the tiles that need
    16-byte segments are left for those that do not."""
    from moe_experts_amd import q4_0_glu
    K, N = 256, 512
    Wg, Wu = weights(4, K, N), weights(5, K, N)
    n = Wg.size
    buf = torch.zeros(2 * n + 64, dtype=torch.uint8, device=dev())
    for og, ou in ((2, n + 6), (0, n + 18)):
        g, u = buf[og:og + n], buf[ou:ou + n]
        g.copy_(to_dev(Wg).view(-1))
        u.copy_(to_dev(Wu).view(-1))
        for M in (1, 6):
            x = datagen.activations(6, M, K)
            ref.check(host(q4_0_glu(to_dev(x), g, u, N)), ref.glu(x, Wg, Wu, "silu"))


def test_glu_full_size():
    from moe_experts_amd import q4_0_glu
    K, N = 4096, 11008
    Wg, Wu = weights(7, K, N), weights(8, K, N)
    dg, du = to_dev(Wg), to_dev(Wu)
    for M in (1, 8):
        x = datagen.activations(9, M, K)
        got = host(q4_0_glu(to_dev(x), dg, du, N, act="gelu"))
        want = ref.glu(x, Wg, Wu, "gelu")
        ref.check(got, want)
        # roundings of a sum of K terms go both ways: their norm grows with its root
        assert np.linalg.norm(got - want[0]) <= 1e-5 * np.linalg.norm(want[0])


# ------------------------------------------------------------------ gated block, prompt
GEMM_SHAPES = [
    (1, 64, 64), (1, 256, 192), (2, 1024, 64), (33, 320, 320), (63, 512, 128), (64, 2048, 64),
    (65, 128, 192), (128, 576, 256), (129, 64, 64), (200, 1024, 128), (256, 192, 320),
    (257, 448, 64), (300, 2048, 192), (700, 128, 128),
]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,K,N", GEMM_SHAPES)
def test_glu_gemm(M, K, N, act):
    from moe_experts_amd import q4_0_glu_gemm, q4_0_glu_gemm_workspace_bytes
    x = datagen.to_f16(datagen.activations(11, M, K))
    Wg, Wu = weights(12, K, N), weights(13, K, N)
    need = q4_0_glu_gemm_workspace_bytes(M, N, K)
    wfull, ws = nan_ws(max(need, 256))
    bufs = [guarded(M * N, dtype=torch.float16, fill=1232.0) for _ in range(3)]
    H, G, U = (b[1].view(M, N) for b in bufs)
    dx, dg, du = to_dev(x), to_dev(Wg), to_dev(Wu)
    q4_0_glu_gemm(dx, dg, du, N, act=act, H=H, G=G, U=U, ws=ws)
    for got, want, what in zip((H, G, U), ref.glu_gemm(x, Wg, Wu, act), "HGU"):
        ref.check(host(got), want, what)
    assert all(guards_intact(b[0], M * N, fill=1232.0) for b in bufs)
    assert ws_guards_intact(wfull, max(need, 256), 0xFF)
    # without g and u, and by the call that allocates them: the same values
    assert torch.equal(q4_0_glu_gemm(dx, dg, du, N, act=act), H)
    again = q4_0_glu_gemm(dx, dg, du, N, act=act, save=True)
    assert all(torch.equal(a, b) for a, b in zip(again, (H, G, U)))


def test_glu_gemm_extreme_gates():
    """Gates far out on both sides: exp over- and underflows, the block does not."""
    from moe_experts_amd import q4_0_glu_gemm
    K, N, M = 64, 64, 5
    Wg, Wu = weights(14, K, N), weights(15, K, N)
    x = datagen.to_f16(datagen.activations(16, M, K) * 200)
    for act in ("silu", "gelu"):
        H = q4_0_glu_gemm(to_dev(x), to_dev(Wg), to_dev(Wu), N, act=act)
        h, g, _ = ref.glu_gemm(x, Wg, Wu, act)
        assert np.abs(g[0]).max() > 100 and np.abs(h[0]).max() < 65504
        ref.check(host(H), h, act)


def test_rows_are_independent():
    """An infinity or NaN in one row of the input stays in that row."""
    from moe_experts_amd import q4_0_gemm_backward, q4_0_glu, q4_0_glu_backward, q4_0_glu_gemm
    K, N = 256, 128
    Wg, Wu = to_dev(weights(17, K, N)), to_dev(weights(18, K, N))
    for M in (8, 70, 300):
        x = datagen.activations(19, M, K)
        bad = x.copy()
        bad[2, 5], bad[5, 7] = np.inf, np.nan
        keep = [m for m in range(M) if m not in (2, 5)]
        def same(f, a, b):
            u, v = host(f(a)), host(f(b))
            assert np.array_equal(u[keep], v[keep]) and np.isfinite(u).all()
            assert np.isnan(v[5]).all() and not np.isfinite(v[2]).any()
        if M == 8:
            same(lambda t: q4_0_glu(t, Wg, Wu, N), to_dev(x), to_dev(bad))
        same(lambda t: q4_0_glu_gemm(t, Wg, Wu, N), to_dev(x).half(), to_dev(bad).half())
        dy = datagen.activations(20, M, N)
        bad = dy.copy()
        bad[2, 5], bad[5, 7] = np.inf, np.nan
        same(lambda t: q4_0_gemm_backward(t, Wg, K), bf16(dy), bf16(bad))
        G, U = (to_dev(datagen.to_f16(datagen.activations(s, M, N))) for s in (21, 22))
        same(lambda t: q4_0_glu_backward(t, G, U, Wg, Wu, K), bf16(dy), bf16(bad))


# ------------------------------------------------------------------ gradients
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
def test_glu_backward(M, N, K, act):
    from moe_experts_amd import q4_0_glu_backward, q4_0_glu_backward_workspace_bytes
    Wg, Wu = weights(31, K, N), weights(32, K, N)
    dH = gradient(33, M, N)
    r = datagen.rng(34)
    G, U = ((r.standard_normal((M, N)) * 2).astype(np.float16) for _ in range(2))
    need = q4_0_glu_backward_workspace_bytes(M, N, K)
    wfull, ws = nan_ws(need)
    full, dX = guarded(M * K, dtype=torch.bfloat16, fill=1232.0)
    q4_0_glu_backward(dH, to_dev(G), to_dev(U), to_dev(Wg), to_dev(Wu), K, act=act,
                      dX=dX.view(M, K), ws=ws)
    ref.check(host(dX).reshape(M, K), ref.glu_backward(values(dH), G, U, Wg, Wu, act))
    assert guards_intact(full, M * K, fill=1232.0) and ws_guards_intact(wfull, need, 0xFF)


@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
def test_gemm_backward(M, N, K):
    from moe_experts_amd import q4_0_gemm_backward, q4_0_gemm_backward_workspace_bytes
    B = weights(35, K, N)
    dY = gradient(36, M, N)
    need = q4_0_gemm_backward_workspace_bytes(M, N, K)
    wfull, ws = nan_ws(need)
    full, dX = guarded(M * K, dtype=torch.bfloat16, fill=1232.0)
    q4_0_gemm_backward(dY, to_dev(B), K, dX=dX.view(M, K), ws=ws)
    ref.check(host(dX).reshape(M, K), ref.gemm_backward(values(dY), B))
    assert guards_intact(full, M * K, fill=1232.0) and ws_guards_intact(wfull, need, 0xFF)


@pytest.mark.parametrize("N", [2048, 4096, 12288, 12352])
def test_gradient_rows_of_every_length(N):
    """Rows that a workgroup holds in one, two or six groups a lane, and longer ones."""
    from moe_experts_amd import q4_0_gemm_backward, q4_0_glu_backward
    M, K = 3, 64
    Wg, Wu = weights(46, K, N), weights(47, K, N)
    dH = gradient(48, M, N)
    r = datagen.rng(49)
    G, U = ((r.standard_normal((M, N)) * 2).astype(np.float16) for _ in range(2))
    dX = q4_0_glu_backward(dH, to_dev(G), to_dev(U), to_dev(Wg), to_dev(Wu), K)
    ref.check(host(dX), ref.glu_backward(values(dH), G, U, Wg, Wu, "silu"))
    ref.check(host(q4_0_gemm_backward(dH, to_dev(Wg), K)), ref.gemm_backward(values(dH), Wg))


def test_gradients_of_far_sizes():
    """Rows from 1e-30 to 1e30, and rows of zeros, in one call: each keeps its own precision."""
    from moe_experts_amd import q4_0_gemm_backward
    M, N, K = 61, 128, 192
    B = weights(37, K, N)
    dy = datagen.activations(38, M, N) * (10.0 ** np.linspace(-30, 30, M))[:, None]
    dy[7] = 0
    dY = bf16(dy)
    got = host(q4_0_gemm_backward(dY, to_dev(B), K))
    ref.check(got, ref.gemm_backward(values(dY), B))
    assert (got[7] == 0).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_against_differences(act):
    """The gradient of sum(c * H(x)) along a direction v, from the kernels' forward and backward
    calls, against a central difference of the 64-bit forward."""
    from moe_experts_amd import q4_0_glu_backward, q4_0_glu_gemm
    M, K, N = 37, 256, 192
    x = datagen.to_f16(datagen.activations(41, M, K) * 0.5)
    Wg, Wu = weights(42, K, N), weights(43, K, N)
    c = bf16(datagen.activations(44, M, N))
    _, G, U = q4_0_glu_gemm(to_dev(x), to_dev(Wg), to_dev(Wu), N, act=act, save=True)
    dX = host(q4_0_glu_backward(c, G, U, to_dev(Wg), to_dev(Wu), K, act=act))
    wg, wu, cv = ref.dequant(Wg), ref.dequant(Wu), values(c).astype(np.float64)
    x = x.astype(np.float64)
    f = lambda z: (cv * ref.act(z @ wg, act)[0] * (z @ wu)).sum(1)
    v = datagen.activations(45, M, K).astype(np.float64)
    eps = 1e-4
    num = (f(x + eps * v) - f(x - eps * v)) / (2 * eps)
    # G and U are rounded to fp16 (and carry the weights' rounding) before the slope: their
    # effect on dX, through the second derivatives (|act''| < 1.2), plus the product's own bound
    (_, _), (g, eg), (u, eu) = ref.glu_gemm(x.astype(np.float16), Wg, Wu, act)
    _, own = ref.glu_backward(cv, g, u, Wg, Wu, act)
    shift = (np.abs(cv) * (1.2 * eg * np.abs(u) + ref.SLOPE * eu)) @ np.abs(wg).T \
        + (np.abs(cv) * ref.SLOPE * eg) @ np.abs(wu).T
    tol = ((own + shift) * np.abs(v)).sum(1) + 1e-6 * np.abs(num)
    assert (np.abs((dX * v).sum(1) - num) <= tol).all()
    # and far inside it where the errors are independent: 1 % of the gradient's own size
    assert np.linalg.norm((dX * v).sum(1) - num) <= 0.01 * np.linalg.norm(num)


# ------------------------------------------------------------------ adapters
def row_ids(kind, M, L, seed=51):
    r = datagen.rng(seed)
    if kind == "mixed":      # any order, some rows without an adapter, some out of range
        ids = r.integers(-2, L + 2, M)
    elif kind == "none":
        ids = np.full(M, -1)
    elif kind == "one":
        ids = np.full(M, L - 1)
    else:                    # requests one after the other, of ragged lengths
        ids = np.sort(r.integers(0, M, M)) * L // max(M, 1)
    return ids.astype(np.int32)


@pytest.mark.parametrize("kind", ["mixed", "none", "one"])
@pytest.mark.parametrize("M,K,N,R,L", [
    (1, 8, 32, 8, 1), (1, 1024, 512, 16, 3), (2, 1000, 160, 24, 5), (3, 72, 32, 8, 2),
    (5, 2056, 544, 64, 9), (8, 1024, 1056, 128, 4), (8, 4096, 64, 40, 12),
])
def test_gemv_lora(M, K, N, R, L, kind):
    from moe_experts_amd import q4_0_gemv, q4_0_gemv_lora, q4_0_gemv_lora_workspace_bytes
    x, B = datagen.activations(52, M, K), weights(53, K, N)
    A, Bl, scale = adapters(54, L, R, K, N)
    ids = row_ids(kind, M, L)
    full, y = guarded(M * N)
    need = q4_0_gemv_lora_workspace_bytes(M, N, K, R)
    wfull, ws = nan_ws(need)
    q4_0_gemv_lora(to_dev(x), to_dev(B), N, to_dev(A), to_dev(Bl), to_dev(ids), to_dev(scale),
                   y=y.view(M, N), ws=ws)
    got = host(y).reshape(M, N)
    ref.check(got, ref.gemv_lora(x, B, A, Bl, ids, scale))
    assert guards_intact(full, M * N) and ws_guards_intact(wfull, need, 0xFF)
    if kind == "none":  # the plain product, whichever tiles form it
        want, bound = ref.product32(x, B)
        ref.check(host(q4_0_gemv(to_dev(x), to_dev(B), N)), (want, bound))
        ref.check(got, (want, bound))


@pytest.mark.parametrize("kind", ["mixed", "none", "one", "ragged"])
@pytest.mark.parametrize("M,K,N,R,L", [
    (1, 64, 64, 8, 1), (3, 1024, 192, 16, 40), (48, 512, 128, 32, 40), (64, 128, 64, 8, 3),
    (65, 256, 192, 24, 7), (129, 64, 64, 128, 2), (130, 2048, 128, 16, 5), (300, 192, 320, 40, 30),
    (515, 448, 64, 64, 3),
])
def test_gemm_lora(M, K, N, R, L, kind):
    from moe_experts_amd import q4_0_gemm_lora, q4_0_gemm_lora_workspace_bytes
    x, B = datagen.to_f16(datagen.activations(55, M, K)), weights(56, K, N)
    A, Bl, scale = adapters(57, L, R, K, N)
    ids = row_ids(kind, M, L)
    full, Y = guarded(M * N, dtype=torch.float16, fill=1232.0)
    need = q4_0_gemm_lora_workspace_bytes(M, N, K, R)
    wfull, ws = nan_ws(need)
    q4_0_gemm_lora(to_dev(x), to_dev(B), N, to_dev(A), to_dev(Bl), to_dev(ids), to_dev(scale),
                   Y=Y.view(M, N), ws=ws)
    ref.check(host(Y).reshape(M, N), ref.gemm_lora(x, B, A, Bl, ids, scale))
    assert guards_intact(full, M * N, fill=1232.0) and ws_guards_intact(wfull, need, 0xFF)


def test_adapter_products_beyond_half_range():
    """A narrow product over 65504 (a large A, a small B) keeps its precision."""
    from moe_experts_amd import q4_0_gemm_lora
    M, K, N, R, L = 200, 64, 64, 8, 2
    x, B = datagen.to_f16(datagen.activations(58, M, K)), weights(59, K, N)
    A, Bl, scale = adapters(60, L, R, K, N)
    A = (A.astype(np.float32) * 60000).astype(np.float16)
    Bl = (Bl.astype(np.float32) * 1e-4).astype(np.float16)
    ids = row_ids("ragged", M, L)
    got = q4_0_gemm_lora(to_dev(x), to_dev(B), N, to_dev(A), to_dev(Bl), to_dev(ids),
                         to_dev(scale))
    assert np.abs(x.astype(np.float64) @ A[0].astype(np.float64).T).max() > 65504
    ref.check(host(got), ref.gemm_lora(x, B, A, Bl, ids, scale))


def test_unused_adapters_are_not_read():
    """Adapters that no row uses may hold anything."""
    from moe_experts_amd import q4_0_gemm_lora, q4_0_gemv_lora
    K, N, R, L = 256, 128, 16, 5
    B = weights(61, K, N)
    A, Bl, scale = adapters(62, L, R, K, N)
    for M in (4, 40, 300):
        ids = np.where(np.arange(M) % 3 == 0, 1, np.where(np.arange(M) % 3 == 1, 4, -1))
        ids = ids.astype(np.int32)
        x = datagen.to_f16(datagen.activations(63, M, K))
        outs = []
        for poison in (False, True):
            a, b, s = A.copy(), Bl.copy(), scale.copy()
            if poison:
                a[[0, 2, 3]], b[[0, 2, 3]], s[[0, 2, 3]] = np.nan, np.inf, np.nan
            args = [to_dev(v) for v in (a, b, ids, s)]
            o = [host(q4_0_gemm_lora(to_dev(x), to_dev(B), N, *args))]
            if M <= 8:
                o.append(host(q4_0_gemv_lora(to_dev(x.astype(np.float32)), to_dev(B), N, *args)))
            outs.append(o)
        assert all(np.array_equal(u, v) and np.isfinite(u).all() for u, v in zip(*outs))


@pytest.mark.parametrize("M", [4, 8, 40, 64, 130, 520])
def test_an_adapter_with_infinities_stays_with_its_rows(M):
    """Infinities and NaN of one adapter reach the rows that use it, and no others."""
    from moe_experts_amd import q4_0_gemm_lora, q4_0_gemv_lora
    K, N, R, L = 256, 192, 24, 3
    B = weights(64, K, N)
    A, Bl, scale = adapters(65, L, R, K, N)
    ids = np.random.default_rng(66).integers(-1, L, M).astype(np.int32)
    ids[:3] = [0, 1, 2]
    x = datagen.to_f16(datagen.activations(67, M, K))
    others = ids != 1
    for broken in (0, 1, 2):
        a, b, s = A.copy(), Bl.copy(), scale.copy()
        if broken == 0:
            a[1, :, ::7] = np.inf
        elif broken == 1:
            b[1, ::5] = np.nan
        else:
            s[1] = np.inf
        calls = [(q4_0_gemm_lora, x)]
        if M <= 8:
            calls.append((q4_0_gemv_lora, x.astype(np.float32)))
        for f, v in calls:
            right = host(f(to_dev(v), to_dev(B), N, *[to_dev(t) for t in (A, Bl, ids, scale)]))
            got = host(f(to_dev(v), to_dev(B), N, *[to_dev(t) for t in (a, b, ids, s)]))
            assert np.array_equal(got[others], right[others])
            assert not np.isfinite(got[~others]).all()


@pytest.mark.parametrize("M", [1, 2, 3, 8])
def test_rows_of_any_size_and_a_row_with_an_infinity(M):
    """Decode rows from 1e-30 to 1e30 keep their own precision, and a row with an infinity or a
    NaN leaves the others as they are."""
    from moe_experts_amd import q4_0_gemv_lora, q4_0_glu
    K, N, R, L = 520, 96, 8, 2
    x = datagen.activations(81, M, K) * (10.0 ** np.linspace(-30, 30, M))[:, None]
    x = x.astype(np.float32)
    B = weights(82, K, N)
    A, Bl, scale = adapters(83, L, R, K, N)
    ids = row_ids("mixed", M, L)
    ad = [to_dev(v) for v in (A, Bl, ids, scale)]
    got = host(q4_0_gemv_lora(to_dev(x), to_dev(B), N, *ad))
    for m in range(M):  # a row by itself: the bound is relative to its own values
        ref.check(got[m:m + 1], ref.gemv_lora(x[m:m + 1], B, A, Bl, ids[m:m + 1], scale))
    if M == 1:
        return
    Wu = weights(84, K, N)
    x = datagen.activations(85, M, K)
    right = host(q4_0_glu(to_dev(x), to_dev(B), to_dev(Wu), N))
    right_l = host(q4_0_gemv_lora(to_dev(x), to_dev(B), N, *ad))
    for bad in (np.inf, -np.inf, np.nan):
        y = x.copy()
        y[1, 77] = bad
        got = host(q4_0_glu(to_dev(y), to_dev(B), to_dev(Wu), N))
        got_l = host(q4_0_gemv_lora(to_dev(y), to_dev(B), N, *ad))
        keep = np.arange(M) != 1
        assert np.array_equal(got[keep], right[keep])
        assert np.array_equal(got_l[keep], right_l[keep])
        assert not np.isfinite(got_l[1]).any()


@pytest.mark.parametrize("shift", [2, 4, 6, 14])
@pytest.mark.parametrize("M,K,N", [(1, 72, 96), (4, 72, 96), (8, 1000, 544), (5, 40, 288)])
def test_decode_over_matrices_at_any_even_address(M, K, N, shift):
    """Q4_0 blocks are 2-byte aligned; rows of an odd number of blocks start in turn at and
    inside a dword. The bytes before and behind a matrix are not weights."""
    from moe_experts_amd import q4_0_gemv_lora, q4_0_glu
    def place(w):
        flat = np.ascontiguousarray(w).reshape(-1).view(np.uint8)
        buf = torch.full((flat.size + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        buf[shift:shift + flat.size] = torch.from_numpy(flat.copy()).cuda()
        return buf[shift:shift + flat.size]
    x = datagen.activations(86, M, K)
    Wg, Wu = weights(87, K, N), weights(88, K, N)
    ref.check(host(q4_0_glu(to_dev(x), place(Wg), place(Wu), N)), ref.glu(x, Wg, Wu, "silu"))
    A, Bl, scale = adapters(89, 2, 8, K, N)
    ids = row_ids("mixed", M, 2)
    got = q4_0_gemv_lora(to_dev(x), place(Wg), N, to_dev(A), to_dev(Bl), to_dev(ids),
                         to_dev(scale))
    ref.check(host(got), ref.gemv_lora(x, Wg, A, Bl, ids, scale))


@pytest.mark.parametrize("M", [40, 70, 300])
@pytest.mark.parametrize("shift", [2, 8, 10])
def test_prompt_and_gradient_over_matrices_at_any_even_address(M, shift):
    from moe_experts_amd import q4_0_gemm_backward, q4_0_glu_gemm
    K, N = 192, 320
    Wg, Wu = weights(90, K, N), weights(91, K, N)
    bufs = []
    for w in (Wg, Wu):
        flat = np.ascontiguousarray(w).reshape(-1).view(np.uint8)
        buf = torch.full((flat.size + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        buf[shift:shift + flat.size] = torch.from_numpy(flat.copy()).cuda()
        bufs.append(buf[shift:shift + flat.size])
    x = datagen.to_f16(datagen.activations(92, M, K))
    got = q4_0_glu_gemm(to_dev(x), bufs[0], bufs[1], N, save=True)
    for g, want, what in zip(got, ref.glu_gemm(x, Wg, Wu, "silu"), "HGU"):
        ref.check(host(g), want, what)
    dY = gradient(93, M, N)
    ref.check(host(q4_0_gemm_backward(dY, bufs[0], K)), ref.gemm_backward(values(dY), Wg))


@pytest.mark.parametrize("M", [2, 40, 130])
def test_adapter_tables_past_four_gigabytes(M):
    """Rows that use the last adapter of a table whose offsets pass 32 bits."""
    from moe_experts_amd import q4_0_gemm_lora, q4_0_gemv_lora
    K, N, R, L = 90112, 64, 128, 190
    B = weights(94, K, N)
    A, Bl, scale = adapters(95, 1, R, K, N)
    table = torch.zeros((L, R, K), dtype=torch.float16, device="cuda")
    assert table.numel() * 2 > 1 << 32
    table[L - 1] = to_dev(A)[0]
    wide = torch.zeros((L, N, R), dtype=torch.float16, device="cuda")
    wide[L - 1] = to_dev(Bl)[0]
    factors = torch.zeros(L, dtype=torch.float32, device="cuda")
    factors[L - 1] = float(scale[0])
    last = np.where(np.arange(M) % 3 == 1, -1, 0).astype(np.int32)
    ids = to_dev(np.where(last == 0, L - 1, -1).astype(np.int32))
    x = datagen.to_f16(datagen.activations(96, M, K))
    got = q4_0_gemm_lora(to_dev(x), to_dev(B), N, table, wide, ids, factors)
    ref.check(host(got), ref.gemm_lora(x, B, A, Bl, last, scale))
    if M <= 8:
        x = x.astype(np.float32)
        got = q4_0_gemv_lora(to_dev(x), to_dev(B), N, table, wide, ids, factors)
        ref.check(host(got), ref.gemv_lora(x, B, A, Bl, last, scale))


@pytest.mark.parametrize("M", [1, 5])
def test_decode_arrays_at_any_dword(M):
    """x and h of the gated block, and y, are 4-byte aligned."""
    from moe_experts_amd import q4_0_gemv_lora, q4_0_glu
    K, N = 333, 160
    x = datagen.activations(97, M, K)
    Wg, Wu = weights(98, K, N), weights(99, K, N)
    at = torch.zeros(M * K + 8, dtype=torch.float32, device="cuda")
    for o in (1, 2, 3):
        at[o:o + M * K] = to_dev(x).reshape(-1)
        h = torch.full((M * N + 8,), 7.0, dtype=torch.float32, device="cuda")
        q4_0_glu(at[o:o + M * K].view(M, K), to_dev(Wg), to_dev(Wu), N,
                 h=h[o:o + M * N].view(M, N))
        ref.check(host(h[o:o + M * N]).reshape(M, N), ref.glu(x, Wg, Wu, "silu"))
        assert (h[:o] == 7).all() and (h[o + M * N:] == 7).all()
        A, Bl, scale = adapters(100, 2, 8, 328, N)
        ids = row_ids("mixed", M, 2)
        B = weights(101, 328, N)
        v = datagen.activations(102, M, 328)
        q4_0_gemv_lora(to_dev(v), to_dev(B), N, to_dev(A), to_dev(Bl), to_dev(ids), to_dev(scale),
                       y=h[o:o + M * N].view(M, N))
        ref.check(host(h[o:o + M * N]).reshape(M, N), ref.gemv_lora(v, B, A, Bl, ids, scale))


@pytest.mark.parametrize("M", [2, 5, 40, 130])
def test_weights_of_any_scale(M):
    """Block scales from the smallest half to ones whose weights reach 65504, beside each other."""
    from moe_experts_amd import q4_0_gemm_lora, q4_0_glu, q4_0_glu_gemm
    K, N = 128, 128
    W = [weights(s, K, N).reshape(K, N // 32, 18).copy() for s in (103, 104)]
    for i, w in enumerate(W):
        d = 2.0 ** np.random.default_rng(105 + i).uniform(-24, 12.9, (K, N // 32))
        w[..., :2] = d.astype(np.float16)[..., None].view(np.uint8)
    x = datagen.to_f16(datagen.activations(107, M, K) * 2.0 ** -12)
    if M <= 8:
        got = q4_0_glu(to_dev(x.astype(np.float32)), to_dev(W[0]), to_dev(W[1]), N)
        ref.check(host(got), ref.glu(x.astype(np.float32), W[0], W[1], "silu"))
    else:
        _, G, U = q4_0_glu_gemm(to_dev(x), to_dev(W[0]), to_dev(W[1]), N, save=True)
        _, g, u = ref.glu_gemm(x, W[0], W[1], "silu")
        ref.check(host(G), g, "G")
        ref.check(host(U), u, "U")
    A, Bl, scale = adapters(108, 2, 8, K, N)
    ids = np.full(M, -1, np.int32)
    got = q4_0_gemm_lora(to_dev(x), to_dev(W[0]), N, to_dev(A), to_dev(Bl), to_dev(ids),
                         to_dev(scale))
    ref.check(host(got), ref.gemm_lora(x, W[0], A, Bl, ids, scale))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("M", [3, 40, 300])
def test_block_with_adapters_and_its_gradient(M):
    """The feed-forward of a layer as it is used: the gated block, the down projection with the
    requests' adapters, and, for training through the frozen block, the gradients back to x."""
    from moe_experts_amd import (q4_0_gemm_backward, q4_0_gemm_lora, q4_0_gemv_lora, q4_0_glu,
                                 q4_0_glu_backward, q4_0_glu_gemm)
    K, I, R, L = 256, 320, 16, 4
    Wg, Wu, Wd = weights(71, K, I), weights(72, K, I), weights(73, I, K)
    dg, du, dd = (to_dev(w) for w in (Wg, Wu, Wd))
    A, Bl, scale = adapters(74, L, R, I, K)
    ids = row_ids("mixed", M, L)
    ad = [to_dev(v) for v in (A, Bl, ids, scale)]
    x = datagen.to_f16(datagen.activations(75, M, K) * 0.5)
    if M <= 8:
        h = q4_0_glu(to_dev(x.astype(np.float32)), dg, du, I)
        y = host(q4_0_gemv_lora(h, dd, K, *ad))
        ref.check(y, ref.gemv_lora(host(h), Wd, A, Bl, ids, scale))
    H, G, U = q4_0_glu_gemm(to_dev(x), dg, du, I, save=True)
    y = q4_0_gemm_lora(H, dd, K, *ad)
    ref.check(host(y), ref.gemm_lora(host(H), Wd, A, Bl, ids, scale))
    dY = gradient(76, M, K)
    dH = q4_0_gemm_backward(dY, dd, I)
    dX = q4_0_glu_backward(dH, G, U, dg, du, K)
    ref.check(host(dH), ref.gemm_backward(values(dY), Wd))
    ref.check(host(dX), ref.glu_backward(values(dH), host(G), host(U), Wg, Wu, "silu"))


@pytest.mark.parametrize("M,K,N", [(1930, 64, 4160), (1100, 4352, 64)])
def test_many_tiles(M, K, N):
    """More tiles than the GPU takes at once, a last row of tiles with few rows, and columns that
    are left over for lower tiles."""
    from moe_experts_amd import q4_0_gemm_backward, q4_0_gemm_lora, q4_0_glu_gemm
    x = datagen.to_f16(datagen.activations(110, M, K))
    Wg, Wu = weights(111, K, N), weights(112, K, N)
    got = q4_0_glu_gemm(to_dev(x), to_dev(Wg), to_dev(Wu), N, save=True)
    for g, want, what in zip(got, ref.glu_gemm(x, Wg, Wu, "silu"), "HGU"):
        ref.check(host(g), want, what)
    dY = gradient(113, M, N)
    ref.check(host(q4_0_gemm_backward(dY, to_dev(Wg), K)), ref.gemm_backward(values(dY), Wg))
    A, Bl, scale = adapters(114, 3, 8, K, N)
    ids = row_ids("ragged", M, 3)
    got = q4_0_gemm_lora(to_dev(x), to_dev(Wg), N, to_dev(A), to_dev(Bl), to_dev(ids),
                         to_dev(scale))
    ref.check(host(got), ref.gemm_lora(x, Wg, A, Bl, ids, scale))


def test_gradient_whose_left_operand_passes_two_gigabytes():
    """Two matrices and millions of columns: the scaled gradients of a tile that lacks rows pass
    2 GiB. Only a few values of dH are not zero, so that the result is known from a few weights."""
    from moe_experts_amd import q4_0_glu_backward
    M, N, K = 50, 12000000, 64  # one tile, whatever its height
    assert M * 2 * N * 2 > 1 << 31 and M * N * 2 < 1 << 31
    r = datagen.rng(120)
    at = r.integers(0, N, (M, 3))  # the columns of each row that carry a gradient
    at[:, 0] = N - 1 - np.arange(M)
    dh = (r.standard_normal((M, 3)) * 1e-3).astype(np.float32)
    g, u = (r.standard_normal((M, 3)).astype(np.float16) for _ in range(2))
    rows = torch.arange(M, device=dev())[:, None]
    cols = to_dev(at)
    dH = torch.zeros((M, N), dtype=torch.bfloat16, device=dev())
    dH[rows, cols] = to_dev(dh).bfloat16()
    G, U = (torch.full((M, N), 0.5, dtype=torch.float16, device=dev()) for _ in range(2))
    G[rows, cols], U[rows, cols] = to_dev(g), to_dev(u)
    gen = torch.Generator(device="cuda").manual_seed(121)
    mats = []
    for _ in range(2):
        w = torch.randint(0, 256, (K, N // 32, 18), dtype=torch.uint8, device=dev(), generator=gen)
        d = torch.rand((K, N // 32, 1), device=dev(), generator=gen) * 0.05
        w[..., :2] = d.half().view(torch.uint8)
        mats.append(w)
    dX = host(q4_0_glu_backward(dH, G, U, mats[0], mats[1], K))
    uniq = np.unique(at)
    # the weights of the columns in use, as blocks of their own: column c of block c // 32
    few = []
    for w in mats:
        blocks = w[:, to_dev(uniq // 32)].cpu().numpy()
        few.append(ref.dequant(blocks).reshape(K, uniq.size, 32)[:, np.arange(uniq.size),
                                                                 uniq % 32])
    where = np.searchsorted(uniq, at)
    full = lambda v: values_at(M, uniq.size, where, v)
    dhv, gv, uv = full(values(dH[rows, cols])), full(g), full(u)
    a, slope = ref.act(gv, "silu")
    few_steps = 64 * ref.E32 * (1 + np.abs(gv))
    want = ref._through([dhv * uv * slope, dhv * a], [np.abs(dhv * uv) * few_steps,
                                                      np.abs(dhv) * few_steps], few)
    ref.check(dX, want)


def values_at(M, n, where, v):
    """A matrix of zeros with row m's values v[m] at where[m]."""
    out = np.zeros((M, n))
    out[np.arange(M)[:, None], where] = v
    return out


@pytest.mark.parametrize("M", [40, 300])
def test_block_in_an_autograd_function(M):
    """The calls as a training program makes them: forward and backward of a
    torch.autograd.Function, between bfloat16 tensors. Outside one, an input that requires a
    gradient is refused."""
    from moe_experts_amd import q4_0_glu_backward, q4_0_glu_gemm
    K, N = 256, 192
    Wg, Wu = weights(131, K, N), weights(132, K, N)
    dg, du = to_dev(Wg), to_dev(Wu)

    class Block(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            H, G, U = q4_0_glu_gemm(x.half(), dg, du, N, save=True)
            ctx.save_for_backward(G, U)
            return H.bfloat16()

        @staticmethod
        def backward(ctx, dh):
            return q4_0_glu_backward(dh.contiguous(), *ctx.saved_tensors, dg, du, K)

    x = to_dev(datagen.activations(133, M, K) * 0.5).bfloat16().requires_grad_()
    c = gradient(134, M, N)
    Block.apply(x).backward(c)
    _, G, U = q4_0_glu_gemm(x.detach().half(), dg, du, N, save=True)
    assert torch.equal(x.grad, q4_0_glu_backward(c, G, U, dg, du, K))
    ref.check(host(x.grad), ref.glu_backward(values(c), host(G), host(U), Wg, Wu, "silu"))
    with pytest.raises(ValueError, match="requires a gradient"):
        q4_0_glu_gemm(x.detach().half().requires_grad_(), dg, du, N)


@pytest.mark.parametrize("K,M", [(8, 1), (16, 2)])
def test_projection_of_the_widest_matrices(K, M):
    """A matrix of nearly 2 GiB with fewer rows than a strip's step of 32: the offsets of the rows
    that it lacks pass 32 bits. Every byte that is not a scale reads as NaN in a scale's place."""
    from moe_experts_amd import q4_0_gemv_lora
    nb = min(((1 << 31) - 1) // (18 * K), ((1 << 31) - 1) // (128 * M))
    N, P = 32 * nb, 64
    assert K > 8 or 24 * nb * 18 > 1 << 32
    r = datagen.rng(140)
    d = r.uniform(0.01, 0.02, (K, P)).astype(np.float16)
    some = np.full((K, P, 18), 0xFF, np.uint8)
    some[..., :2] = d[..., None].view(np.uint8)
    of = torch.arange(nb, device=dev()) % P
    B = to_dev(some)[:, of].contiguous()
    x = datagen.activations(141, M, K)
    A = torch.zeros((1, 8, K), dtype=torch.float16, device=dev())
    Bl = torch.zeros((1, N, 8), dtype=torch.float16, device=dev())
    ids = torch.full((M,), -1, dtype=torch.int32, device=dev())
    y = q4_0_gemv_lora(to_dev(x), B, N, A, Bl, ids, torch.ones(1, device=dev()))
    want, bound = ref.product32(x, some)  # weights 15 - 8 = 7 times d, block by block
    want, bound = (to_dev(v.reshape(M, P, 32)[:, :, 0]) for v in (want, bound))
    for m in range(M):
        got = y[m].view(nb, 32)
        off = (got.double() - want[m][of][:, None]).abs()
        assert bool((off <= bound[m][of][:, None]).all()), (m, float(got.sum()))
