"""How exactly the dense feed-forward forms its products (ffn_precision.py)."""
import numpy as np
import pytest
import torch

from moe_experts_amd import datagen
from tests import ffn_precision as fp
from tests import ffn_ref as ref
from tests.gpu_util import to_dev
from tests.test_gpu_ffn import adapters, host, row_ids, weights

pytestmark = pytest.mark.gpu

# few rows (1 to 4 groups of 16, exact weights) and tiles
FEW = (1, 16, 17, 33, 49, 64)
MANY = (65, 100, 150, 300, 777)


@pytest.mark.parametrize("K,N", [(64, 64), (576, 192), (1088, 320)])
@pytest.mark.parametrize("M", FEW + MANY)
def test_gated_block_differences(M, K, N):
    """Weights that differ by less than fp16 holds of them."""
    from moe_experts_amd import q4_0_glu_gemm
    Wg, Wu = fp.near_rows(1, K, N), fp.near_rows(2, K, N)
    for at in (0, 37):
        x = fp.differences(M, K, at)
        _, G, U = q4_0_glu_gemm(to_dev(x), to_dev(Wg), to_dev(Wu), N, save=True)
        assert np.array_equal(host(G), fp.exact_differences(x, Wg))
        assert np.array_equal(host(U), fp.exact_differences(x, Wu))


@pytest.mark.parametrize("place", [-24, -21, -14, -6, 2])
@pytest.mark.parametrize("M", (16, 100, 150, 777))
def test_gated_block_differences_at_every_scale(M, place):
    """Scales from the smallest normal ones of fp16 to those whose weights are its largest."""
    from moe_experts_amd import q4_0_glu_gemm
    K, N = 576, 192
    Wg, Wu = fp.near_rows(1, K, N, place), fp.near_rows(2, K, N, -18)
    x = fp.differences(M, K)
    _, G, U = q4_0_glu_gemm(to_dev(x), to_dev(Wg), to_dev(Wu), N, save=True)
    assert np.array_equal(host(G), fp.exact_differences(x, Wg))
    assert np.array_equal(host(U), fp.exact_differences(x, Wu))


@pytest.mark.parametrize("K,N", [(576, 192), (4096, 256), (1088, 1088)])
@pytest.mark.parametrize("M", FEW + MANY)
def test_gated_block_norms(M, K, N):
    from moe_experts_amd import q4_0_glu_gemm
    x = datagen.to_f16(datagen.activations(3, M, K))
    Wg, Wu = weights(4, K, N), weights(5, K, N)
    left = 0.0 if M <= 64 else fp.LEFT
    H, G, U = (host(t) for t in q4_0_glu_gemm(to_dev(x), to_dev(Wg), to_dev(Wu), N, save=True))
    g, eg = fp.norm_bound(x, Wg, left, True)
    u, eu = fp.norm_bound(x, Wu, left, True)
    fp.check_norm(G, g, eg, "g")
    fp.check_norm(U, u, eu, "u")
    # h: its own rounding, and the errors of the unrounded g and u through the product, element
    # by element of the size the norms give them
    a, slope = ref.act(g, "silu")
    h = a * u
    per = lambda x_, B: fp.norm_bound(x_, B, left, False)[1] / np.sqrt(g.size)
    through = np.sqrt(np.square(slope * u).sum() * per(x, Wg) ** 2
                      + np.square(a).sum() * per(x, Wu) ** 2)
    fp.check_norm(H, h, np.hypot(np.linalg.norm(h - fp.rounded16(h)), 2 * through), "h")


@pytest.mark.parametrize("M", [3, 5, 8])
def test_decode_differences_and_norms(M):
    """fp32 rows over exact weights."""
    from moe_experts_amd import q4_0_gemv_lora, q4_0_glu
    K, N, R, L = 1000, 288, 8, 2
    Wg, Wu = fp.near_rows(6, K, N), fp.near_rows(7, K, N)
    A, Bl, scale = adapters(8, L, R, K, N)
    none = to_dev(np.full(M, -1, np.int32))
    ad = [to_dev(A), to_dev(Bl), none, to_dev(scale)]
    for at in range(0, K, 97):
        x = fp.differences(M, K, at).astype(np.float32)
        y = host(q4_0_gemv_lora(to_dev(x), to_dev(Wg), N, *ad))
        g, u = fp.exact_differences(x, Wg), fp.exact_differences(x, Wu)
        assert np.array_equal(y, g)
        h = host(q4_0_glu(to_dev(x), to_dev(Wg), to_dev(Wu), N))
        want = ref.act(g, "silu")[0] * u
        assert (np.abs(h - want) <= 16 * ref.E32 * np.abs(want)).all()
    x = datagen.activations(9, M, K)
    B = weights(10, K, N)
    y = host(q4_0_gemv_lora(to_dev(x), to_dev(B), N, *ad))
    fp.check_norm(y, *fp.norm_bound(x, B, 0.0, False))


@pytest.mark.parametrize("M", FEW)
def test_projection_of_few_rows(M):
    """fp16 rows over exact weights, without and with adapters."""
    from moe_experts_amd import q4_0_gemm_lora
    K, N, R, L = 1088, 320, 16, 3
    A, Bl, scale = adapters(11, L, R, K, N)
    ad = [to_dev(A), to_dev(Bl)]
    none, s = to_dev(np.full(M, -1, np.int32)), to_dev(scale)
    B = fp.near_rows(12, K, N)
    for at in range(0, K, 113):
        x = fp.differences(M, K, at)
        y = host(q4_0_gemm_lora(to_dev(x), to_dev(B), N, *ad, none, s))
        assert np.array_equal(y, fp.exact_differences(x, B))
    x, B = datagen.to_f16(datagen.activations(13, M, K)), weights(14, K, N)
    y = host(q4_0_gemm_lora(to_dev(x), to_dev(B), N, *ad, none, s))
    fp.check_norm(y, *fp.norm_bound(x, B, 0.0, True))
    # with adapters: two more fp32 sums, of K and of R terms
    ids = row_ids("mixed", M, L)
    y = host(q4_0_gemm_lora(to_dev(x), to_dev(B), N, *ad, to_dev(ids), s))
    value = x.astype(np.float64) @ ref.dequant(B) + ref.adapters(x, A, Bl, ids, scale, False)[0]
    own = np.linalg.norm(value - fp.rounded16(value))
    sums = 2 * (np.sqrt(K) + np.sqrt(R)) * ref.E32 * np.linalg.norm(value) * 2
    fp.check_norm(y, value, np.hypot(own, sums))


@pytest.mark.parametrize("K", [1, 5, 8, 31, 33, 40])
@pytest.mark.parametrize("M", [2, 3, 8])
def test_decode_of_short_rows_reads_none_of_the_next(M, K):
    """Rows shorter than a step of 32: an infinity at the start of each other row, which stands
    right behind, does not reach them."""
    from moe_experts_amd import q4_0_gemv_lora, q4_0_glu
    N = 96
    Wg, Wu = weights(15, K, N), weights(16, K, N)
    x = datagen.activations(17, M, K)
    bad = x.copy()
    bad[1::2, 0] = np.inf
    calls = [lambda v: q4_0_glu(to_dev(v), to_dev(Wg), to_dev(Wu), N)]
    if K % 8 == 0:
        A, Bl, scale = adapters(18, 2, 8, K, N)
        rest = [to_dev(t) for t in (A, Bl, row_ids("mixed", M, 2), scale)]
        calls.append(lambda v: q4_0_gemv_lora(to_dev(v), to_dev(Wg), N, *rest))
    for call in calls:
        right, got = host(call(x)), host(call(bad))
        assert np.array_equal(got[0::2], right[0::2])
        assert not np.isfinite(got[1::2]).any()
