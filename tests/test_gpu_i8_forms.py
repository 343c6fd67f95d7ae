"""The 8-bit operators' row kernels in every form that a shape can choose, and the gradients'
tiles behind each of them: lengths around every form's end, sizes far apart, values that are not
finite. Against 64-bit references as in test_gpu_i8.py."""
import numpy as np
import pytest
import torch

from moe_experts_amd import datagen
from tests import i8_ref as ref
from tests.gpu_util import dev, guarded, guards_intact, to_dev

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


def int8(seed, *shape):
    return datagen.rng(seed).integers(-128, 128, shape).astype(np.int8)


def scales(seed, n):
    return np.exp(datagen.rng(seed).standard_normal(n) - 4).astype(np.float32)


def gradient(seed, M, N):
    r = datagen.rng(seed)
    return typed(r.standard_normal((M, N)) * np.exp(r.standard_normal((M, 1)) * 2 - 9), "bf16")


def tiled(form, M, N, K):
    from moe_experts_amd import i8_gemm_plan
    return i8_gemm_plan(form, M, N, K)[0] > 0


# ------------------------------------------------------------------ quantizing
MANY = 257  # rows: more than the wider workgroups take
LONG = [2049, 4095, 4096, 4097, 8191, 8192, 8193, 11008, 12287, 12289, 16383, 16384, 16385, 20001]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("K", LONG)
def test_quantize_many_rows(K, kind):
    from moe_experts_amd import i8_dequantize, i8_quantize
    x = typed(datagen.activations(1, MANY, K) * np.exp(datagen.rng(2).standard_normal((MANY, 1)) * 4),
              kind)
    fq, q = guarded(MANY * K, torch.int8, fill=77)
    fs, s = guarded(MANY)
    i8_quantize(x, Q=q.view(MANY, K), scale=s)
    want = ref.rows(host(x))
    assert np.array_equal(whole(s), want[1], equal_nan=True)  # a row past fp16 has infinities
    assert np.array_equal(whole(q).reshape(MANY, K), want[0])
    assert guards_intact(fq, MANY * K, fill=77) and guards_intact(fs, MANY)
    back = i8_dequantize(q.view(MANY, K), s, dtype=TYPES[kind])
    value = torch.from_numpy(want[0].astype(np.float32) * want[1][:, None]).to(TYPES[kind])
    assert np.array_equal(host(back), value.float().numpy(), equal_nan=True)


def odd_rows(K):
    """Ties and their neighbours at scales of every size, zeros, infinities and NaN, the smallest
    and the largest numbers."""
    r = datagen.rng(11)
    sizes = np.float32([1.0, 2.0 ** -60, 2.0 ** -66, 2.0 ** -120, 2.0 ** -140, 2.0 ** 119])
    ties = (r.uniform(-1, 1, (6, K)) * sizes[:, None]).astype(np.float32)
    ties[:, 0] = np.float32([1, 127, 0.7, 3, 1, 1.5]) * sizes
    s = (np.abs(ties).max(1) / np.float32(127)).astype(np.float32)[:, None]
    half = np.round(r.uniform(-126, 126, (6, K - 1))) + 0.5
    ties[:, 1:] = (half * s).astype(np.float32)
    ties[:, 1::3] = np.nextafter(ties[:, 1::3], np.float32(0))
    ties[:, 2::3] = np.nextafter(ties[:, 2::3], np.float32(np.inf))
    ties = np.where(np.abs(ties) > np.abs(ties[:, :1]), 0, ties)
    x = datagen.activations(12, 8, K)
    x[0] = 0
    x[1, K // 2] = np.inf
    x[2, K - 1] = -np.inf
    x[3, 0] = np.nan
    x[4, K - 1] = -np.nan
    x[5] = np.where(np.arange(K) == K // 3, np.float32(1e-45), 0)
    x[6] = np.float32(3.4e38) * np.sign(x[6])
    x[7] = np.float32(1e-45) * np.round(x[7] * 100)
    return np.concatenate([ties, x])


@pytest.mark.parametrize("K", [3001, 6001, 10001, 14001, 17001])
def test_quantize_odd_rows_among_many(K):
    from moe_experts_amd import i8_quantize
    few = odd_rows(K)
    many = np.concatenate([few] * 19)
    assert len(many) > 256
    for x in (few, many):
        q, s = i8_quantize(to_dev(x))
        want = ref.rows(x)
        assert np.array_equal(whole(s), want[1], equal_nan=True)
        assert np.array_equal(whole(q), want[0])


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("K", [3001, 6001, 10001, 14001, 17001])
def test_quantize_broken_rows_among_many(K, kind):
    from moe_experts_amd import i8_quantize
    x = typed(datagen.activations(13, MANY, K), kind)
    x[1, K - 1], x[2, 0], x[3], x[MANY - 1, K // 2] = float("inf"), float("nan"), 0, float("nan")
    q, s = i8_quantize(x)
    want = ref.rows(host(x))
    assert np.array_equal(whole(s), want[1], equal_nan=True) and np.array_equal(whole(q), want[0])


# ------------------------------------------------------------------ left operands
#: M, N, K by tiles: lengths of a row of dY around each form of the row kernel
ROWS = [(300, 8, 1040), (300, 72, 1040), (300, 504, 1040), (300, 512, 1040), (300, 520, 1040),
        (300, 2040, 1040), (40, 2056, 272), (40, 4088, 272), (40, 4096, 272), (40, 4104, 272),
        (40, 8192, 80), (40, 8200, 80), (40, 12280, 80), (40, 12296, 80), (40, 16384, 80),
        (40, 16392, 80), (17, 20008, 48)]
#: M, N, K by tiles: tokens around each form of the transposition in one kernel, and in two
COLUMNS = [(1, 264, 1040), (63, 264, 1040), (65, 264, 1040), (127, 264, 1040), (129, 264, 1040),
           (255, 264, 1040), (511, 264, 1040), (513, 264, 1040), (1023, 264, 1040),
           (1025, 264, 1040), (2047, 264, 1040), (2049, 264, 1040), (4095, 72, 48), (4097, 24, 48),
           (8191, 72, 48), (300, 4096, 80),
           (8193, 24, 48), (1, 4104, 80), (65, 4104, 80), (129, 4104, 80), (255, 4104, 80),
           (257, 4104, 80), (300, 4160, 272), (513, 4104, 80), (20001, 72, 16),
           (64 * 256 * 3 + 5, 24, 16)]


@pytest.mark.parametrize("M,N,K", ROWS)
def test_input(M, N, K):
    from moe_experts_amd import i8_gemm_backward
    assert tiled("i8_gemm_backward", M, N, K)
    dY, W, sw = gradient(51, M, N), int8(52, N, K), scales(53, N)
    got = host(i8_gemm_backward(dY, to_dev(W), to_dev(sw)))
    want = ref.backward(host(dY), W, sw)
    ref.check(got, want)
    ref.check_norm(got, want[0])


@pytest.mark.parametrize("M,N,K", COLUMNS)
def test_weights(M, N, K):
    from moe_experts_amd import i8_gemm_backward_weight
    assert tiled("i8_gemm_backward_weight", M, N, K)
    dY, X, sx = gradient(54, M, N), int8(55, M, K), scales(56, M)
    got = host(i8_gemm_backward_weight(dY, to_dev(X), to_dev(sx)))
    want = ref.backward_weight(host(dY), X, sx)
    ref.check(got, want)
    ref.check_norm(got, want[0])


#: by tiles, with and without splits, the weights' by either transposition
BROKEN = [("i8_gemm_backward", 300, 136, 1040), ("i8_gemm_backward", 40, 4104, 272),
          ("i8_gemm_backward_weight", 300, 264, 1040), ("i8_gemm_backward_weight", 2500, 72, 272),
          ("i8_gemm_backward_weight", 300, 4104, 272), ("i8_gemm_backward_weight", 9001, 72, 272)]


def call(form, dY, B, s):
    import moe_experts_amd as q4
    return getattr(q4, form)(dY, B, to_dev(s))


@pytest.mark.parametrize("form,M,N,K", BROKEN)
def test_broken_values_stay_with_their_rows(form, M, N, K):
    assert tiled(form, M, N, K)
    weight = form.endswith("weight")
    depth = M if weight else N
    dY, B, s = gradient(68, M, N), to_dev(int8(69, depth, K)), scales(70, depth)
    was = call(form, dY, B, s)
    broken = dY.clone()
    broken[3, 7], broken[M - 1, 60], broken[9, N - 1] = float("inf"), float("nan"), float("-inf")
    got = call(form, broken, B, s)
    rows = (7, 60, N - 1) if weight else (3, M - 1, 9)
    keep = [i for i in range(got.shape[0]) if i not in rows]
    assert not torch.isfinite(got[list(rows)].float()).any()
    assert torch.equal(got[keep], was[keep])
    s[depth - 3] = np.nan
    assert torch.isnan(call(form, dY, B, s).float()).all()


@pytest.mark.parametrize("form,M,N,K", BROKEN)
def test_far_sizes(form, M, N, K):
    """Rows of the result of any size of fp32 beside one another, and a row of zeros."""
    assert tiled(form, M, N, K)
    weight = form.endswith("weight")
    depth, rows = (M, N) if weight else (N, M)
    r = datagen.rng(63)
    size = 2.0 ** np.linspace(-110, 100, rows)
    size[5] = 0
    v = r.standard_normal((rows, depth)) * size[:, None]
    dY, B, s = typed(v.T if weight else v, "bf16"), int8(64, depth, K), scales(65, depth)
    got = host(call(form, dY, to_dev(B), s))
    ref.check(got, (ref.backward_weight if weight else ref.backward)(host(dY), B, s))
    assert not got[5].any()


@pytest.mark.parametrize("M,N,K", [(300, 264, 1040), (2100, 72, 528)])
def test_gradients_against_differences(M, N, K):
    """By tiles: the change of sum(c * Y) under whole steps of X or W is what the gradients say."""
    from moe_experts_amd import i8_gemm, i8_gemm_backward, i8_gemm_backward_weight
    assert tiled("i8_gemm_backward", M, N, K) and tiled("i8_gemm_backward_weight", M, N, K)
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
