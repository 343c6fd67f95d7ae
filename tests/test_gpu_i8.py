"""8-bit operators against 64-bit references, element by element within bounds counted
from the roundings (tests/i8_ref.py); whole numbers exactly."""
import numpy as np
import pytest
import torch

from moe_experts_amd import datagen
from tests import i8_ref as ref
from tests.gpu_util import dev, guarded, guarded_ws, guards_intact, to_dev, ws_guards_intact

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def host(t):
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy()


def whole(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def typed(a, kind):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(TYPES[kind]).to(dev())


def int8(seed, *shape, low=-127):
    return datagen.rng(seed).integers(low, 128, shape).astype(np.int8)


def scales(seed, n):
    return np.exp(datagen.rng(seed).standard_normal(n) - 4).astype(np.float32)


def gradient(seed, M, N):
    r = datagen.rng(seed)
    return typed(r.standard_normal((M, N)) * np.exp(r.standard_normal((M, 1)) * 2 - 9), "bf16")


def same_rows(got, want):
    q, s = whole(got[0]), whole(got[1])
    assert np.array_equal(s, want[1], equal_nan=True)
    assert np.array_equal(q, want[0])


# ------------------------------------------------------------------ rows
ROW_SHAPES = [(1, 1), (3, 7), (8, 16), (70, 33), (5, 511), (5, 513), (2, 2047), (2, 2049),
              (3, 4096), (3, 4097), (2, 8193), (2, 16384), (2, 16391), (1, 40000), (600, 24)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,K", ROW_SHAPES)
def test_quantize(M, K, kind):
    from moe_experts_amd import i8_quantize
    x = typed(datagen.activations(1, M, K) * np.exp(datagen.rng(2).standard_normal((M, 1)) * 4),
              kind)
    fq, q = guarded(M * K, torch.int8, fill=77)
    fs, s = guarded(M)
    i8_quantize(x, Q=q.view(M, K), scale=s)
    same_rows((q.view(M, K), s), ref.rows(host(x)))
    assert guards_intact(fq, M * K, fill=77) and guards_intact(fs, M)


@pytest.mark.parametrize("kind", TYPES)
def test_quantize_every_short_row(kind):
    from moe_experts_amd import i8_quantize
    for K in range(1, 40):
        x = typed(datagen.activations(K, 5, K), kind)
        same_rows(i8_quantize(x), ref.rows(host(x)))


@pytest.mark.parametrize("size", [1.0, 2.0 ** -60, 2.0 ** -66, 2.0 ** -120, 2.0 ** -140, 2.0 ** 119])
@pytest.mark.parametrize("K", [200, 5000, 20000])
def test_quantize_ties_and_their_neighbours(K, size):
    """Values at the halves of their scale, and one fp32 step beside them, at every size of scale
    that fp32 has, below the normal range too."""
    from moe_experts_amd import i8_quantize
    r = datagen.rng(11)
    x = (r.uniform(-1, 1, (4, K)) * size).astype(np.float32)
    x[:, 0] = np.float32([1, 127, 0.7, 3]) * np.float32(size)  # row 1: the scale is a power of two
    s = (np.abs(x).max(1) / np.float32(127)).astype(np.float32)[:, None]
    half = np.round(r.uniform(-126, 126, (4, K - 1))) + 0.5
    x[:, 1:] = (half * s).astype(np.float32)
    x[:, 1::3] = np.nextafter(x[:, 1::3], np.float32(0))
    x[:, 2::3] = np.nextafter(x[:, 2::3], np.float32(np.inf))
    x = np.where(np.abs(x) > np.abs(x[:, :1]), 0, x)
    same_rows(i8_quantize(to_dev(x)), ref.rows(x))


def test_quantize_odd_rows():
    """Zeros, an infinity, a NaN (of either sign, in any place), the smallest and the largest
    numbers: each row by itself."""
    from moe_experts_amd import i8_quantize
    for K in (9, 700, 5000, 17000):
        x = datagen.activations(12, 9, K)
        x[0] = 0
        x[1, K // 2] = np.inf
        x[2, K - 1] = -np.inf
        x[3, 0] = np.nan
        x[4, K - 1] = -np.nan
        x[5] = np.where(np.arange(K) == K // 3, np.float32(1e-45), 0)
        x[6] = np.float32(3.4e38) * np.sign(x[6])
        x[7] = np.float32(1e-45) * np.round(x[7] * 100)
        same_rows(i8_quantize(to_dev(x)), ref.rows(x))
    for kind in ("fp16", "bf16"):
        x = typed(datagen.activations(13, 4, 300), kind)
        x[1, 299], x[2, 0], x[3] = float("inf"), float("nan"), 0
        same_rows(i8_quantize(x), ref.rows(host(x)))


@pytest.mark.parametrize("kind", TYPES)
def test_rows_at_any_address(kind):
    """Arrays that begin at any value of a larger one."""
    from moe_experts_amd import i8_dequantize, i8_quantize
    M, K = 3, 1000
    store = typed(datagen.activations(14, 1, M * K + 8), kind).view(-1)
    for off in (1, 2, 3, 5):
        x = store[off:off + M * K].view(M, K)
        fq = torch.zeros(M * K + 8, dtype=torch.int8, device=dev())
        q = fq[off:off + M * K].view(M, K)
        s = torch.zeros(M + 8, device=dev())[off:off + M]
        i8_quantize(x, Q=q, scale=s)
        want = ref.rows(host(x))
        same_rows((q, s), want)
        assert not whole(fq)[:off].any() and not whole(fq)[off + M * K:].any()
        back = torch.zeros(M * K + 8, dtype=TYPES[kind], device=dev())
        i8_dequantize(q, s, X=back[off:off + M * K].view(M, K))
        v = torch.from_numpy(want[0].astype(np.float32) * want[1][:, None]).to(TYPES[kind])
        assert torch.equal(back[off:off + M * K].cpu().view(M, K), v)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,K", ROW_SHAPES)
def test_dequantize(M, K, kind):
    from moe_experts_amd import i8_dequantize
    q, s = int8(21, M, K, low=-128), scales(22, M)
    full, x = guarded(M * K, TYPES[kind], fill=7.0)
    i8_dequantize(to_dev(q), to_dev(s), X=x.view(M, K))
    want = torch.from_numpy(q.astype(np.float32) * s[:, None]).to(TYPES[kind])
    assert torch.equal(x.view(M, K).cpu(), want) and guards_intact(full, M * K, fill=7.0)
    assert torch.equal(i8_dequantize(to_dev(q), to_dev(s), dtype=TYPES[kind]).cpu(), want)


def test_broken_rows_stay_broken():
    """What i8_quantize makes of a row with an infinity or a NaN comes back as NaN, and its
    neighbours come back whole."""
    from moe_experts_amd import i8_dequantize, i8_quantize
    for K in (5, 300, 5000):
        x = to_dev(datagen.activations(23, 4, K))
        x[1, 0], x[2, K - 1] = float("inf"), float("nan")
        back = i8_dequantize(*i8_quantize(x), dtype=torch.bfloat16)
        assert torch.isnan(back[1:3].float()).all() and torch.isfinite(back[0::3].float()).all()


# ------------------------------------------------------------------ products
#: few rows in every grouping, tiles of every height, ragged ends, with and without splits
GEMM_SHAPES = [(1, 16, 8), (1, 4096, 256), (5, 80, 24), (8, 11008, 72), (16, 1040, 136),
               (17, 64, 8), (32, 528, 1000), (33, 4096, 200), (48, 48, 520), (50, 2064, 72),
               (64, 640, 128), (65, 16, 8), (65, 4112, 264), (100, 128, 128), (130, 144, 1032),
               (200, 8208, 520), (300, 272, 136), (777, 5120, 264), (1100, 400, 4104),
               (1300, 2064, 4160), (1030, 16, 4096)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,K,N", GEMM_SHAPES)
def test_gemm(M, K, N, kind):
    from moe_experts_amd import i8_gemm, i8_gemm_workspace_bytes
    X, W, sx, sw = int8(31, M, K, low=-128), int8(32, N, K, low=-128), scales(33, M), scales(34, N)
    if kind == "fp16":
        sx = sx / 64
    full, y = guarded(M * N, TYPES[kind], guard=128, fill=7.0)
    need = i8_gemm_workspace_bytes(M, N, K)
    wfull, ws = guarded_ws(need, fill=0xFF)
    i8_gemm(to_dev(X), to_dev(sx), to_dev(W), to_dev(sw), Y=y.view(M, N), ws=ws)
    ref.check(host(y.view(M, N)), ref.gemm(X, sx, W, sw, kind))
    assert guards_intact(full, M * N, guard=128, fill=7.0)
    assert ws_guards_intact(wfull, need, fill=0xFF)


@pytest.mark.parametrize("M,K,N", GEMM_SHAPES)
def test_gemm_is_exact(M, K, N):
    """Scales of one: the whole numbers themselves, rounded to fp32 once."""
    from moe_experts_amd import i8_gemm
    X, W = int8(35, M, K, low=-128), int8(36, N, K, low=-128)
    ones = lambda n: torch.ones(n, device=dev())
    y = i8_gemm(to_dev(X), ones(M), to_dev(W), ones(N), dtype=torch.float32)
    assert np.array_equal(host(y), ref.product(X, W).astype(np.float32))


@pytest.mark.parametrize("M", [1, 40, 70, 300])
def test_gemm_largest_sums(M):
    """The longest rows of -128: sums just below 2^31."""
    from moe_experts_amd import i8_gemm
    K, N = 131056, 16
    full = lambda *s: torch.full(s, -128, dtype=torch.int8, device=dev())
    ones = lambda n: torch.ones(n, device=dev())
    X, W = full(M, K), full(N, K)
    W[3] = 127
    y = host(i8_gemm(X, ones(M), W, ones(N), dtype=torch.float32))
    want = np.full((M, N), K * 16384.0)
    want[:, 3] = -128.0 * 127 * K
    assert np.array_equal(y, want.astype(np.float32))


@pytest.mark.parametrize("M", [2, 40, 130])
def test_scales_of_every_kind(M):
    """A NaN stays with its row or column, zero and negative scales are taken as they are."""
    from moe_experts_amd import i8_gemm
    K, N = 256, 64
    X, W, sx, sw = int8(37, M, K), int8(38, N, K), scales(39, M), scales(40, N)
    sx[1], sw[5], sw[6], sw[7] = np.nan, np.nan, 0, -0.5
    y = host(i8_gemm(to_dev(X), to_dev(sx), to_dev(W), to_dev(sw), dtype=torch.float32))
    bad = np.zeros((M, N), dtype=bool)
    bad[1] = bad[:, 5] = True
    assert np.isnan(y[bad]).all() and np.isfinite(y[~bad]).all()
    want, e = ref.gemm(X, sx, W, sw, "fp32")
    assert (np.abs(y - want) <= e)[~bad].all() and not y[~bad[:, 6], 6].any()


@pytest.mark.parametrize("M,K,N", [(1, 16, 8), (1, 4096, 256), (1, 16384, 24), (1, 16400, 24),
                                   (2, 8192, 40), (2, 8208, 40), (3, 528, 1000), (5, 3280, 72),
                                   (7, 48, 16), (8, 2048, 520), (8, 2064, 8), (8, 11008, 72),
                                   (4, 131056, 16)])
def test_gemv(M, K, N):
    """Quantized as by i8_quantize, multiplied as by i8_gemm: bitwise."""
    from moe_experts_amd import i8_gemm, i8_gemv, i8_gemv_workspace_bytes, i8_quantize
    x = datagen.activations(41, M, K) * np.exp(datagen.rng(42).standard_normal((M, 1)) * 3)
    x = x.astype(np.float32)
    x[:, -1] = 0.5 * np.abs(x).max(1) / 127  # a value close to a half of the scale
    W, sw = to_dev(int8(43, N, K)), to_dev(scales(44, N))
    full, y = guarded(M * N)
    need = i8_gemv_workspace_bytes(M, N, K)
    wfull, ws = guarded_ws(need, fill=0xFF)
    i8_gemv(to_dev(x), W, sw, y=y.view(M, N), ws=ws)
    q, s = i8_quantize(to_dev(x))
    assert torch.equal(y.view(M, N), i8_gemm(q, s, W, sw, dtype=torch.float32))
    qr, sr = ref.rows(x)
    ref.check(host(y.view(M, N)), ref.gemm(qr, sr, whole(W), whole(sw), "fp32"))
    assert guards_intact(full, M * N) and ws_guards_intact(wfull, need, fill=0xFF)


@pytest.mark.parametrize("K", [512, 4096])
def test_gemv_rows_are_independent(K):
    """A row of zeros, one with an infinity, one with a NaN among eight: the others are what they
    are alone, bitwise."""
    from moe_experts_amd import i8_gemv
    N = 72
    x = to_dev(datagen.activations(45, 8, K))
    W, sw = to_dev(int8(46, N, K)), to_dev(scales(47, N))
    x[2] = 0
    x[4, K // 2], x[6, K - 1] = float("inf"), float("nan")
    y = i8_gemv(x, W, sw)
    for m in range(8):
        alone = i8_gemv(x[m:m + 1].clone(), W, sw)
        if m in (4, 6):
            assert torch.isnan(y[m]).all() and torch.isnan(alone).all()
        else:
            assert torch.equal(y[m:m + 1], alone)
    assert not y[2].any()


def test_gemv_at_any_dword():
    from moe_experts_amd import i8_gemv
    M, K, N = 3, 528, 40
    W, sw = to_dev(int8(48, N, K)), scales(49, N + 4)
    store = to_dev(datagen.activations(50, 1, M * K + 4)).view(-1)
    for off in (1, 2, 3):
        x, s = store[off:off + M * K].view(M, K), to_dev(sw)[off:off + N]
        assert torch.equal(i8_gemv(x, W, s), i8_gemv(x.clone(), W, s.clone()))


# ------------------------------------------------------------------ gradients
#: tiles of 32, 64, 128 and 256 rows, ragged ends, with and without splits
GRAD_SHAPES = [(1, 8, 16), (1, 4096, 272), (7, 24, 48), (30, 520, 272), (33, 72, 528),
               (64, 1032, 256), (65, 8, 16), (100, 4104, 272), (130, 136, 1040), (150, 2048, 512),
               (300, 520, 4112), (777, 1536, 272), (2100, 72, 8208), (4200, 136, 4112)]


@pytest.mark.parametrize("M,N,K", GRAD_SHAPES)
def test_backward(M, N, K):
    from moe_experts_amd import i8_gemm_backward, i8_gemm_backward_workspace_bytes
    dY, W, sw = gradient(51, M, N), int8(52, N, K, low=-128), scales(53, N)
    full, dX = guarded(M * K, torch.bfloat16, fill=7.0)
    need = i8_gemm_backward_workspace_bytes(M, N, K)
    wfull, ws = guarded_ws(need, fill=0xFF)
    i8_gemm_backward(dY, to_dev(W), to_dev(sw), dX=dX.view(M, K), ws=ws)
    want = ref.backward(host(dY), W, sw)
    ref.check(host(dX.view(M, K)), want)
    ref.check_norm(host(dX.view(M, K)), want[0])
    assert guards_intact(full, M * K, fill=7.0) and ws_guards_intact(wfull, need, fill=0xFF)


@pytest.mark.parametrize("N,M,K", GRAD_SHAPES[:1] + [(n + (-n) % 8, m, k) for n, m, k in GRAD_SHAPES])
def test_backward_weight(M, N, K):
    from moe_experts_amd import (i8_gemm_backward_weight,
                                 i8_gemm_backward_weight_workspace_bytes)
    N += (-N) % 8
    dY, X, sx = gradient(54, M, N), int8(55, M, K, low=-128), scales(56, M)
    full, dW = guarded(N * K, torch.bfloat16, fill=7.0)
    need = i8_gemm_backward_weight_workspace_bytes(M, N, K)
    wfull, ws = guarded_ws(need, fill=0xFF)
    i8_gemm_backward_weight(dY, to_dev(X), to_dev(sx), dW=dW.view(N, K), ws=ws)
    want = ref.backward_weight(host(dY), X, sx)
    ref.check(host(dW.view(N, K)), want)
    ref.check_norm(host(dW.view(N, K)), want[0])
    assert guards_intact(full, N * K, fill=7.0) and ws_guards_intact(wfull, need, fill=0xFF)


@pytest.mark.parametrize("M", [1, 2, 63, 64, 65, 129, 255, 257, 300, 513])
def test_backward_weight_of_every_length(M):
    """Tokens that end anywhere in a step and in a chunk of the transposition."""
    from moe_experts_amd import i8_gemm_backward_weight
    N, K = 72, 48
    dY, X, sx = gradient(57, M, N), int8(58, M, K), scales(59, M)
    got = host(i8_gemm_backward_weight(dY, to_dev(X), to_dev(sx)))
    want = ref.backward_weight(host(dY), X, sx)
    ref.check(got, want)
    ref.check_norm(got, want[0])


def test_backward_weight_of_many_tokens():
    """More rows than 64 chunks of 256, so that a chunk of the search for the largest is longer."""
    from moe_experts_amd import i8_gemm_backward_weight
    M, N, K = 64 * 256 * 3 + 5, 8, 16
    dY, X, sx = gradient(59, M, N), int8(58, M, K), scales(57, M)
    got = host(i8_gemm_backward_weight(dY, to_dev(X), to_dev(sx)))
    want = ref.backward_weight(host(dY), X, sx)
    ref.check(got, want)
    ref.check_norm(got, want[0])


#: lengths around a pair, a step, what a wave, a lane and a workgroup take, and splits
FEW_TOKENS = [1, 2, 31, 32, 33, 255, 257, 511, 512, 513, 1023, 1025, 1999, 2047, 2048, 2049, 4095,
              4096, 4097, 6001, 32769]


@pytest.mark.parametrize("N", [8, 16])
@pytest.mark.parametrize("M", FEW_TOKENS)
def test_backward_weight_of_few_channels(M, N):
    from moe_experts_amd import (i8_gemm_backward_weight,
                                 i8_gemm_backward_weight_workspace_bytes)
    K = (16, 48, 64, 80, 208)[M % 5]
    dY, X, sx = gradient(90, M, N), int8(91, M, K, low=-128), scales(92, M)
    full, dW = guarded(N * K, torch.bfloat16, fill=7.0)
    need = i8_gemm_backward_weight_workspace_bytes(M, N, K)
    wfull, ws = guarded_ws(need, fill=0xFF)
    i8_gemm_backward_weight(dY, to_dev(X), to_dev(sx), dW=dW.view(N, K), ws=ws)
    want = ref.backward_weight(host(dY), X, sx)
    ref.check(host(dW.view(N, K)), want)
    ref.check_norm(host(dW.view(N, K)), want[0])
    assert guards_intact(full, N * K, fill=7.0) and ws_guards_intact(wfull, need, fill=0xFF)


@pytest.mark.parametrize("N", [8, 16])
@pytest.mark.parametrize("M", [70, 9000])
def test_few_channels_of_far_sizes(M, N):
    """Channels of any size beside one another; tokens whose size falls by 2^40 on the way, so that
    splits scale by powers of their own; a channel of zeros."""
    from moe_experts_amd import i8_gemm_backward_weight
    K = 80
    r = datagen.rng(93)
    X, sx = int8(94, M, K), scales(95, M)
    size = 2.0 ** np.linspace(-60, 90, N)
    size[5] = 0
    fall = 2.0 ** np.linspace(0, -40, M)[:, None]
    dY = typed(r.standard_normal((M, N)) * size * fall, "bf16")
    got = host(i8_gemm_backward_weight(dY, to_dev(X), to_dev(sx)))
    ref.check(got, ref.backward_weight(host(dY), X, sx))
    assert not got[5].any()


@pytest.mark.parametrize("N", [8, 16])
@pytest.mark.parametrize("M", [70, 9000])
def test_few_broken_channels_stay_alone(M, N):
    from moe_experts_amd import i8_gemm_backward_weight
    K = 272
    dY, X, sx = gradient(96, M, N), to_dev(int8(97, M, K)), scales(98, M)
    was = i8_gemm_backward_weight(dY, X, to_dev(sx))
    broken = dY.clone()
    broken[3, 6], broken[M - 1, 1] = float("inf"), float("nan")
    got = i8_gemm_backward_weight(broken, X, to_dev(sx))
    keep = [n for n in range(N) if n not in (1, 6)]
    assert not torch.isfinite(got[[1, 6]].float()).any()
    assert torch.equal(got[keep], was[keep])
    sx[M - 2] = np.nan
    assert torch.isnan(i8_gemm_backward_weight(dY, X, to_dev(sx)).float()).all()


@pytest.mark.parametrize("N", [8, 24, 64, 1000, 2040, 2048, 2056, 4096, 4104, 6008, 16392])
@pytest.mark.parametrize("M", [1, 7, 8, 9, 15, 16])
def test_backward_of_few_rows(M, N):
    from moe_experts_amd import i8_gemm_backward, i8_gemm_backward_workspace_bytes
    K = (16, 48, 64, 80, 208)[(M + N // 8) % 5]
    dY, W, sw = gradient(100, M, N), int8(101, N, K, low=-128), scales(102, N)
    full, dX = guarded(M * K, torch.bfloat16, fill=7.0)
    need = i8_gemm_backward_workspace_bytes(M, N, K)
    wfull, ws = guarded_ws(need, fill=0xFF)
    i8_gemm_backward(dY, to_dev(W), to_dev(sw), dX=dX.view(M, K), ws=ws)
    want = ref.backward(host(dY), W, sw)
    ref.check(host(dX.view(M, K)), want)
    ref.check_norm(host(dX.view(M, K)), want[0])
    assert guards_intact(full, M * K, fill=7.0) and ws_guards_intact(wfull, need, fill=0xFF)


@pytest.mark.parametrize("M", [5, 8, 13, 16])
@pytest.mark.parametrize("N", [72, 9000])
def test_few_rows_of_far_sizes(M, N):
    """Rows of any size beside one another, whose values fall by 2^40 on the way; a row of zeros."""
    from moe_experts_amd import i8_gemm_backward
    K = 80
    r = datagen.rng(103)
    W, sw = int8(104, N, K), scales(105, N)
    size = 2.0 ** np.linspace(-60, 90, M)[:, None]
    size[4] = 0
    dY = typed(r.standard_normal((M, N)) * size * 2.0 ** np.linspace(0, -40, N), "bf16")
    got = host(i8_gemm_backward(dY, to_dev(W), to_dev(sw)))
    ref.check(got, ref.backward(host(dY), W, sw))
    assert not got[4].any()


@pytest.mark.parametrize("M", [5, 8, 13, 16])
@pytest.mark.parametrize("N", [72, 9000])
def test_few_broken_rows_stay_alone(M, N):
    from moe_experts_amd import i8_gemm_backward
    K = 272
    dY, W, sw = gradient(106, M, N), to_dev(int8(107, N, K)), scales(108, N)
    was = i8_gemm_backward(dY, W, to_dev(sw))
    broken = dY.clone()
    broken[3, 6], broken[1, N - 1] = float("inf"), float("nan")
    got = i8_gemm_backward(broken, W, to_dev(sw))
    keep = [m for m in range(M) if m not in (1, 3)]
    assert not torch.isfinite(got[[1, 3]].float()).any()
    assert torch.equal(got[keep], was[keep])
    sw[N - 2] = np.nan
    assert torch.isnan(i8_gemm_backward(dY, W, to_dev(sw)).float()).all()


@pytest.mark.parametrize("rows", [17, 23, 24, 31, 32, 33, 40, 104])
@pytest.mark.parametrize("depth", [8, 264, 2040, 2048])
def test_gradients_by_groups_of_rows(rows, depth):
    """Results of more rows than a workgroup makes, the last group of any height."""
    from moe_experts_amd import i8_gemm_backward, i8_gemm_backward_weight
    K = (16, 80, 208)[rows % 3]
    dY, B, s = gradient(110, rows, depth), int8(111, depth, K, low=-128), scales(112, depth)
    full, out = guarded(rows * K, torch.bfloat16, fill=7.0)
    i8_gemm_backward(dY, to_dev(B), to_dev(s), dX=out.view(rows, K))
    want = ref.backward(host(dY), B, s)
    ref.check(host(out.view(rows, K)), want)
    ref.check_norm(host(out.view(rows, K)), want[0])
    assert guards_intact(full, rows * K, fill=7.0)
    rows += -rows % 8
    depth -= depth // 16  # any length
    dY, B, s = gradient(113, depth, rows), int8(114, depth, K, low=-128), scales(115, depth)
    full, out = guarded(rows * K, torch.bfloat16, fill=7.0)
    i8_gemm_backward_weight(dY, to_dev(B), to_dev(s), dW=out.view(rows, K))
    want = ref.backward_weight(host(dY), B, s)
    ref.check(host(out.view(rows, K)), want)
    ref.check_norm(host(out.view(rows, K)), want[0])
    assert guards_intact(full, rows * K, fill=7.0)


@pytest.mark.parametrize("M,N,K", [(7, 24, 48), (64, 1032, 272), (150, 2048, 512), (300, 520, 4112),
                                   (4200, 136, 4112)])
def test_gradients_pick_single_values(M, N, K):
    """One value in each row (column) of dY: rows of W (X) come out times a power of two, exactly."""
    from moe_experts_amd import i8_gemm_backward, i8_gemm_backward_weight
    r = datagen.rng(60)
    W, X = int8(61, N, K, low=-128), int8(62, M, K, low=-128)
    at = r.integers(0, N, M)
    dY = np.zeros((M, N), dtype=np.float32)
    dY[np.arange(M), at] = 2.0 ** r.integers(-30, 10, M)
    sw = (2.0 ** r.integers(-8, 3, N)).astype(np.float32)
    got = host(i8_gemm_backward(typed(dY, "bf16"), to_dev(W), to_dev(sw)))
    size = dY[np.arange(M), at] * sw[at]
    assert np.array_equal(got, W[at].astype(np.float32) * size[:, None])
    at = r.integers(0, M, N)
    dY = np.zeros((M, N), dtype=np.float32)
    dY[at, np.arange(N)] = 2.0 ** r.integers(-30, 10, N)
    sx = (2.0 ** r.integers(-8, 3, M)).astype(np.float32)
    got = host(i8_gemm_backward_weight(typed(dY, "bf16"), to_dev(X), to_dev(sx)))
    size = dY[at, np.arange(N)] * sx[at]
    assert np.array_equal(got, X[at].astype(np.float32) * size[:, None])


def test_gradients_of_far_sizes():
    """Rows (columns) of dY of any size of fp32 beside one another, and rows of zeros."""
    from moe_experts_amd import i8_gemm_backward, i8_gemm_backward_weight
    M, N, K = 96, 64, 48
    r = datagen.rng(63)
    W, X, sw, sx = int8(64, N, K), int8(65, M, K), scales(66, N), scales(67, M)
    size = 2.0 ** np.linspace(-110, 100, M)
    size[5] = 0
    dY = typed(r.standard_normal((M, N)) * size[:, None], "bf16")
    got = host(i8_gemm_backward(dY, to_dev(W), to_dev(sw)))
    ref.check(got, ref.backward(host(dY), W, sw))
    assert not got[5].any()
    size = 2.0 ** np.linspace(-110, 100, N)
    size[5] = 0
    dY = typed(r.standard_normal((M, N)) * size, "bf16")
    got = host(i8_gemm_backward_weight(dY, to_dev(X), to_dev(sx)))
    ref.check(got, ref.backward_weight(host(dY), X, sx))
    assert not got[5].any()


@pytest.mark.parametrize("M", [40, 300])
def test_broken_gradients_stay_with_their_rows(M):
    from moe_experts_amd import i8_gemm_backward, i8_gemm_backward_weight
    N, K = 136, 272
    dY, W, X = gradient(68, M, N), int8(69, N, K), int8(70, M, K)
    sw, sx = scales(71, N), scales(72, M)
    clean = (i8_gemm_backward(dY, to_dev(W), to_dev(sw)),
             i8_gemm_backward_weight(dY, to_dev(X), to_dev(sx)))
    broken = dY.clone()
    broken[3, 7], broken[9, 60] = float("inf"), float("nan")
    for got, was, rows in ((i8_gemm_backward(broken, to_dev(W), to_dev(sw)), clean[0], (3, 9)),
                           (i8_gemm_backward_weight(broken, to_dev(X), to_dev(sx)), clean[1],
                            (7, 60))):
        keep = torch.ones(got.shape[0], dtype=torch.bool, device=dev())
        for i in rows:
            keep[i] = False
            assert not torch.isfinite(got[i].float()).any()
        assert torch.equal(got[keep], was[keep])
    sx[5] = np.nan
    assert torch.isnan(i8_gemm_backward_weight(dY, to_dev(X), to_dev(sx)).float()).all()


@pytest.mark.parametrize("M", [40, 150])
def test_gradients_against_differences(M):
    """The product is linear in either operand's values: the change of sum(c * Y) under whole
    steps of X or W, from Y in fp32, is what the gradients say. Bounds: Y's of i8_ref.gemm, the
    gradients' of i8_ref, each added up over what it multiplies."""
    from moe_experts_amd import i8_gemm, i8_gemm_backward, i8_gemm_backward_weight
    N, K = 72, 528
    r = datagen.rng(73)
    X, W, sx, sw = int8(74, M, K) // 2, int8(75, N, K) // 2, scales(76, M), scales(77, N)
    c = typed(r.standard_normal((M, N)), "bf16")
    ch = host(c).astype(np.float64)
    y = lambda X, W: host(i8_gemm(to_dev(X), to_dev(sx), to_dev(W), to_dev(sw),
                                  dtype=torch.float32)).astype(np.float64)
    for which in ("X", "W"):
        E = r.integers(-3, 4, (M if which == "X" else N, K)).astype(np.int8)
        X1, W1 = (X + E, W) if which == "X" else (X, W + E)
        change = (ch * (y(X1, W1) - y(X, W))).sum()
        e = sum((np.abs(ch) * ref.gemm(a, sx, b, sw, "fp32")[1]).sum()
                for a, b in ((X, W), (X1, W1)))
        if which == "X":
            g = host(i8_gemm_backward(c, to_dev(W), to_dev(sw)))
            step, bound = E * sx.astype(np.float64)[:, None], ref.backward(ch, W, sw)[1]
        else:
            g = host(i8_gemm_backward_weight(c, to_dev(X), to_dev(sx)))
            step, bound = E * sw.astype(np.float64)[:, None], ref.backward_weight(ch, X, sx)[1]
        assert abs((g.astype(np.float64) * step).sum() - change) <= e + (bound * np.abs(step)).sum()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("M", [3, 40, 300])
def test_training_step(M):
    """A linear in 8 bits as a training program runs it: the rows that the forward pass quantized
    are all that it keeps, and both gradients come from them."""
    from moe_experts_amd import (i8_dequantize, i8_gemm, i8_gemm_backward,
                                 i8_gemm_backward_weight, i8_quantize)
    K, N = 272, 136

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            kept = (*i8_quantize(x), *i8_quantize(w))
            ctx.save_for_backward(*kept)
            return i8_gemm(*kept, dtype=torch.bfloat16)

        @staticmethod
        def backward(ctx, dy):
            qx, sx, qw, sw = ctx.saved_tensors
            dy = dy.contiguous()
            return i8_gemm_backward(dy, qw, sw), i8_gemm_backward_weight(dy, qx, sx)

    x = typed(datagen.activations(81, M, K), "bf16").requires_grad_()
    w = typed(datagen.activations(82, N, K) / 16, "bf16").requires_grad_()
    c = gradient(83, M, N)
    y = Linear.apply(x, w)
    y.backward(c)
    (qx, sx), (qw, sw) = ref.rows(host(x)), ref.rows(host(w))
    ref.check(host(y), ref.gemm(qx, sx, qw, sw, "bf16"))
    for g, want in ((x.grad, ref.backward(host(c), qw, sw)),
                    (w.grad, ref.backward_weight(host(c), qx, sx))):
        ref.check(host(g), want)
        ref.check_norm(host(g), want[0])
    kept = i8_quantize(x.detach())
    # half a step of the scale, and the roundings of the product and the result
    near = host(i8_dequantize(*kept, dtype=torch.bfloat16))
    size = np.abs(host(x))
    assert (np.abs(near - host(x)) <= 0.5001 * sx[:, None] + ref.EBF * (size + sx[:, None])).all()
    with pytest.raises(ValueError, match="requires a gradient"):
        i8_quantize(x)


def test_adapter_beside_a_frozen_projection():
    """The narrow half of an adapter trained from the rows that a frozen projection kept: its
    gradient is that of weights of as many rows as the adapter's rank."""
    from moe_experts_amd import i8_gemm_backward_weight, i8_quantize
    M, K, R, N = 130, 528, 8, 72
    x = typed(datagen.activations(84, M, K), "fp16")
    up = typed(datagen.activations(85, N, R), "bf16")
    dy = gradient(86, M, N)
    dt = (dy.float() @ up.float()).bfloat16()
    q, s = i8_quantize(x)
    got = host(i8_gemm_backward_weight(dt, q, s))
    want = ref.backward_weight(host(dt), *ref.rows(host(x)))
    ref.check(got, want)
    ref.check_norm(got, want[0])


def test_prompt_then_tokens():
    """Weights stored in 8 bits once; the prompt by i8_gemm, the tokens behind it by i8_gemv, one
    at a time and eight together: rows of one result, bitwise."""
    from moe_experts_amd import i8_gemm, i8_gemv, i8_quantize
    K, N = 1040, 264
    W, sw = i8_quantize(typed(datagen.activations(87, N, K) / 32, "bf16"))
    x = to_dev(datagen.activations(88, 100, K))
    y = i8_gemm(*i8_quantize(x), W, sw, dtype=torch.float32)
    for m in (0, 57, 99):
        assert torch.equal(i8_gemv(x[m:m + 1].clone(), W, sw), y[m:m + 1])
    assert torch.equal(i8_gemv(x[20:28].clone(), W, sw), y[20:28])
    assert torch.equal(i8_gemm(*i8_quantize(x[:40].clone()), W, sw, dtype=torch.float32), y[:40])


# ------------------------------------------------------------------ sizes at the limits
def test_products_of_nearly_two_gigabytes():
    """Operands and results whose offsets need all of 31 bits, in every place: their last rows."""
    from moe_experts_amd import i8_gemm, i8_gemm_backward, i8_gemm_backward_weight, i8_gemv
    n, K = ((1 << 31) - 1) // 16, 16
    n -= n % 8
    g = torch.Generator(device="cuda").manual_seed(91)
    big = torch.randint(-128, 128, (n, K), dtype=torch.int8, device=dev(), generator=g)
    s = torch.rand((n,), device=dev(), generator=g)
    few = to_dev(int8(92, 8, K))
    sf = to_dev(scales(93, 8))
    tail = slice(n - 300, n)
    for rows, scale, name in ((big, s, "X"), (few, sf, "W")):
        assert rows.is_contiguous()
    y = i8_gemm(big, s, few, sf, dtype=torch.float16)          # many tokens
    ref.check(host(y[tail]), ref.gemm(whole(big[tail]), whole(s[tail]), whole(few), whole(sf), "fp16"))
    del y
    x = to_dev(datagen.activations(94, 1, K))
    y = i8_gemv(x, big, s)                                      # many channels
    q, sq = ref.rows(whole(x))
    ref.check(host(y[:, tail]), ref.gemm(q, sq, whole(big[tail]), whole(s[tail]), "fp32"))
    del y
    y = i8_gemm(few[:4].contiguous(), sf[:4].contiguous(), big, s, dtype=torch.float16)
    ref.check(host(y[:, tail]),
              ref.gemm(whole(few[:4]), whole(sf[:4]), whole(big[tail]), whole(s[tail]), "fp16"))
    del y
    # gradients: a contraction over all of them, of which a few count
    at = torch.tensor([0, 1, n // 2, n - 2, n - 1], device=dev())
    dY = torch.zeros((4, n), dtype=torch.bfloat16, device=dev())
    dY[:, at] = gradient(95, 4, 5)
    got = host(i8_gemm_backward(dY, big, s))
    ref.check(got, ref.backward(host(dY[:, at]), whole(big[at]), whole(s[at])))
    del dY
    dY = torch.zeros((n, 8), dtype=torch.bfloat16, device=dev())
    dY[at] = gradient(96, 5, 8)
    got = host(i8_gemm_backward_weight(dY, big, s))
    ref.check(got, ref.backward_weight(host(dY[at]), whole(big[at]), whole(s[at])))


def test_rows_of_nearly_two_gigabytes():
    from moe_experts_amd import i8_dequantize, i8_quantize
    for M, K in (((1 << 29) - 1, 2), (3, (1 << 30) // 3), (70000, 15339)):
        assert (1 << 31) - M * K * 2 < 1 << 17
        x = torch.zeros((M, K), dtype=torch.float16, device=dev())
        x[-1] = typed(datagen.activations(97, 1, K), "fp16")
        x[0] = 3
        q, s = i8_quantize(x)
        want = ref.rows(host(x[-1:]))
        same_rows((q[-1:], s[-1:]), want)
        assert bool((q[0] == 127).all()) and bool((q[1:-1] == 0).all()) and not s[1:-1].any()
        back = i8_dequantize(q, s, dtype=torch.float16)
        v = torch.from_numpy(want[0].astype(np.float32) * want[1][:, None]).half()
        assert torch.equal(back[-1:].cpu(), v) and not back[1:-1].any()
        del x, q, s, back
