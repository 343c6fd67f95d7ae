"""Every tile GEMM of the dense feed-forward, with and without splits of the
contraction, odd and even numbers of K steps, a last row of tiles with few rows and
a last column of tiles that is half full. Each shape says which kernel it is for,
and that is asked of the plan."""
import numpy as np
import pytest

import tests.built  # noqa: F401  (the plan is the library's)
from moe_experts_amd import datagen, q4_0_ffn_plan
from tests import ffn_precision as fp
from tests import ffn_ref as ref
from tests.gpu_util import guarded, guards_intact, to_dev, ws_guards_intact
from tests.test_gpu_ffn import adapters, gradient, host, nan_ws, row_ids, values, weights

# form, rows of a tile, splits, K steps of a split, M, N, K
SHAPES = [
    ("q4_0_glu_gemm", 64, 1, 6, 65, 64, 384),
    ("q4_0_glu_gemm", 64, 1, 5, 65, 64, 320),
    ("q4_0_glu_gemm", 64, 3, 6, 65, 2112, 1024),
    ("q4_0_glu_gemm", 64, 16, 5, 65, 64, 5120),
    ("q4_0_glu_gemm", 128, 1, 6, 129, 6464, 384),
    ("q4_0_glu_gemm", 128, 1, 5, 129, 6464, 320),
    ("q4_0_glu_gemm", 128, 4, 6, 65, 3264, 1536),
    ("q4_0_glu_gemm", 128, 4, 5, 65, 3264, 1280),
    ("q4_0_glu_gemm", 256, 1, 6, 257, 6464, 384),
    ("q4_0_glu_gemm", 256, 1, 5, 257, 6464, 320),
    ("q4_0_glu_gemm", 256, 5, 8, 129, 2112, 2560),
    ("q4_0_glu_gemm", 256, 6, 11, 129, 2112, 4096),
    ("q4_0_glu_backward", 64, 1, 10, 65, 320, 64),
    ("q4_0_glu_backward", 64, 16, 8, 65, 4096, 64),
    ("q4_0_glu_backward", 64, 14, 5, 65, 2112, 64),      # a split takes from both matrices
    ("q4_0_glu_backward", 128, 1, 10, 777, 320, 2496),
    ("q4_0_glu_backward", 128, 14, 6, 65, 2560, 2112),   # here too
    ("q4_0_glu_backward", 128, 7, 5, 65, 1088, 4544),    # and here
    ("q4_0_glu_backward", 256, 1, 10, 1030, 320, 3904),
    ("q4_0_glu_backward", 256, 5, 16, 129, 2560, 4544),  # and here
    ("q4_0_glu_backward", 256, 12, 17, 129, 6400, 2112),
    ("q4_0_gemm_backward", 64, 1, 6, 65, 384, 64),
    ("q4_0_gemm_backward", 64, 1, 5, 65, 320, 64),
    ("q4_0_gemm_backward", 64, 4, 6, 65, 1536, 3264),
    ("q4_0_gemm_backward", 64, 16, 5, 65, 5120, 64),
    ("q4_0_gemm_backward", 128, 1, 6, 777, 384, 2496),
    ("q4_0_gemm_backward", 128, 1, 5, 777, 320, 2496),
    ("q4_0_gemm_backward", 128, 4, 6, 65, 1536, 6464),
    ("q4_0_gemm_backward", 128, 15, 7, 2000, 6400, 64),
    ("q4_0_gemm_backward", 256, 1, 6, 1030, 384, 3904),
    ("q4_0_gemm_backward", 256, 1, 5, 1030, 320, 3904),
    ("q4_0_gemm_backward", 256, 4, 10, 129, 2560, 6464),
    ("q4_0_gemm_backward", 256, 5, 13, 129, 4096, 4544),
    ("q4_0_gemm_lora", 64, 1, 6, 65, 64, 384),
    ("q4_0_gemm_lora", 64, 1, 5, 65, 64, 320),
    ("q4_0_gemm_lora", 64, 4, 6, 65, 3264, 1536),
    ("q4_0_gemm_lora", 64, 16, 5, 65, 64, 5120),
    ("q4_0_gemm_lora", 128, 1, 6, 777, 2496, 384),
    ("q4_0_gemm_lora", 128, 1, 5, 777, 2496, 320),
    ("q4_0_gemm_lora", 128, 4, 6, 65, 6464, 1536),
    ("q4_0_gemm_lora", 128, 15, 7, 2000, 64, 6400),
    ("q4_0_gemm_lora", 256, 1, 6, 1030, 3904, 384),
    ("q4_0_gemm_lora", 256, 1, 5, 1030, 3904, 320),
    ("q4_0_gemm_lora", 256, 4, 10, 129, 6464, 2560),
    ("q4_0_gemm_lora", 256, 5, 13, 129, 4544, 4096),
]


def of(form):
    return [s[1:] for s in SHAPES if s[0] == form]


def planned(form, rows, splits, steps, M, N, K):
    assert q4_0_ffn_plan(form, M, N, K) == (rows, splits, steps)
    assert M % rows


# ---------------------------------------------------------------- without a GPU
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_shapes_take_the_kernels_they_are_for(shape):
    planned(*shape)


def test_every_kernel_has_its_shapes():
    """Heights, with and without splits, of every form; of splits and of one workgroup a tile odd
    and even numbers of steps, more than the four that go before the loop's own."""
    forms = {s[0] for s in SHAPES}
    assert len(forms) == 4
    have = {(f, rows, splits > 1, steps % 2) for f, rows, splits, steps, *_ in SHAPES}
    assert all(s[3] >= 5 for s in SHAPES)
    for f in forms:
        for rows in (64, 128, 256):
            for split in (False, True):
                for odd in (0, 1):
                    if f == "q4_0_glu_backward" and odd and not split:
                        continue  # two matrices of whole steps: always even
                    assert (f, rows, split, odd) in have, (f, rows, split, odd)


def test_plan_refuses():
    from moe_experts_amd import Q4Error
    with pytest.raises(ValueError, match="form must be"):
        q4_0_ffn_plan("q4_0_gemm", 65, 64, 64)
    for shape in ((0, 64, 64), (65, 96, 64), (65, 64, 32), (1 << 30, 64, 64)):
        with pytest.raises(Q4Error):
            q4_0_ffn_plan("q4_0_glu_gemm", *shape)
    assert q4_0_ffn_plan("q4_0_glu_gemm", 64, 64, 64)[0] == 0  # few rows: the strips
    assert q4_0_ffn_plan("q4_0_gemm_backward", 64, 64, 64)[0] == 64


# ---------------------------------------------------------------- on the GPU
def buffers(M, C, need, dtype, n=1):
    outs = [guarded(M * C, dtype=dtype, fill=1232.0) for _ in range(n)]
    wfull, ws = nan_ws(max(need, 256))
    def intact():
        return all(guards_intact(f, M * C, fill=1232.0) for f, _ in outs) and \
            ws_guards_intact(wfull, max(need, 256), 0xFF)
    return [v.view(M, C) for _, v in outs], ws, intact


@pytest.mark.gpu
@pytest.mark.parametrize("rows,splits,steps,M,N,K", of("q4_0_glu_gemm"))
def test_gated_block(rows, splits, steps, M, N, K):
    import torch
    from moe_experts_amd import q4_0_glu_gemm, q4_0_glu_gemm_workspace_bytes
    planned("q4_0_glu_gemm", rows, splits, steps, M, N, K)
    x = datagen.to_f16(datagen.activations(1, M, K))
    Wg, Wu = weights(2, K, N), weights(3, K, N)
    outs, ws, intact = buffers(M, N, q4_0_glu_gemm_workspace_bytes(M, N, K), torch.float16, 3)
    dg, du = to_dev(Wg), to_dev(Wu)
    q4_0_glu_gemm(to_dev(x), dg, du, N, act="gelu", H=outs[0], G=outs[1], U=outs[2], ws=ws)
    for got, want, what in zip(outs, ref.glu_gemm(x, Wg, Wu, "gelu"), "HGU"):
        ref.check(host(got), want, what)
    assert intact()
    for got, W in ((outs[1], Wg), (outs[2], Wu)):
        fp.check_norm(host(got), *fp.norm_bound(x, W, fp.LEFT, True))
    assert torch.equal(q4_0_glu_gemm(to_dev(x), dg, du, N, act="gelu"), outs[0])
    # every k of every step, in every row of a tile
    Wg = fp.near_rows(4, K, N)
    for at in (0, K // 2 + 5):
        x = fp.differences(M, K, at)
        G = q4_0_glu_gemm(to_dev(x), to_dev(Wg), du, N, save=True)[1]
        assert np.array_equal(host(G), fp.exact_differences(x, Wg))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,splits,steps,M,N,K", of("q4_0_glu_backward"))
def test_gradient_of_the_block(rows, splits, steps, M, N, K):
    import torch
    from moe_experts_amd import q4_0_glu_backward, q4_0_glu_backward_workspace_bytes
    planned("q4_0_glu_backward", rows, splits, steps, M, N, K)
    Wg, Wu = weights(5, K, N), weights(6, K, N)
    dH = gradient(7, M, N)
    r = datagen.rng(8)
    G, U = ((r.standard_normal((M, N)) * 2).astype(np.float16) for _ in range(2))
    outs, ws, intact = buffers(M, K, q4_0_glu_backward_workspace_bytes(M, N, K), torch.bfloat16)
    q4_0_glu_backward(dH, to_dev(G), to_dev(U), to_dev(Wg), to_dev(Wu), K, dX=outs[0], ws=ws)
    got = host(outs[0])
    ref.check(got, ref.glu_backward(values(dH), G, U, Wg, Wu, "silu"))
    assert intact()
    dh, g, u = (v.astype(np.float64) for v in (values(dH), G, U))
    a, slope = ref.act(g, "silu")
    # rows from 1e-8 to 1 times one another: each row to its own size
    size = np.abs(dh).max(1, keepdims=True)
    value, bound = fp.gradient_bound([dh * u * slope / size, dh * a / size],
                                     [ref.dequant(Wg), ref.dequant(Wu)])
    fp.check_norm(got / size, value, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,splits,steps,M,N,K", of("q4_0_gemm_backward"))
def test_gradient_of_a_projection(rows, splits, steps, M, N, K):
    import torch
    from moe_experts_amd import q4_0_gemm_backward, q4_0_gemm_backward_workspace_bytes
    planned("q4_0_gemm_backward", rows, splits, steps, M, N, K)
    B = weights(9, K, N)
    dY = gradient(10, M, N)
    outs, ws, intact = buffers(M, K, q4_0_gemm_backward_workspace_bytes(M, N, K), torch.bfloat16)
    q4_0_gemm_backward(dY, to_dev(B), K, dX=outs[0], ws=ws)
    got = host(outs[0])
    ref.check(got, ref.gemm_backward(values(dY), B))
    assert intact()
    dy = values(dY).astype(np.float64)
    size = np.abs(dy).max(1, keepdims=True)
    fp.check_norm(got / size, *fp.gradient_bound([dy / size], [ref.dequant(B)]))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,splits,steps,M,N,K", of("q4_0_gemm_lora"))
@pytest.mark.parametrize("kind", ["mixed", "ragged"])
def test_projection_with_adapters(rows, splits, steps, M, N, K, kind):
    import torch
    from moe_experts_amd import q4_0_gemm_lora, q4_0_gemm_lora_workspace_bytes
    planned("q4_0_gemm_lora", rows, splits, steps, M, N, K)
    R, L = 24, 3
    x, B = datagen.to_f16(datagen.activations(11, M, K)), weights(12, K, N)
    A, Bl, scale = adapters(13, L, R, K, N)
    ids = row_ids(kind, M, L)
    outs, ws, intact = buffers(M, N, q4_0_gemm_lora_workspace_bytes(M, N, K, R), torch.float16)
    ad = [to_dev(v) for v in (A, Bl, ids, scale)]
    q4_0_gemm_lora(to_dev(x), to_dev(B), N, *ad, Y=outs[0], ws=ws)
    ref.check(host(outs[0]), ref.gemm_lora(x, B, A, Bl, ids, scale))
    assert intact()
    none = to_dev(np.full(M, -1, np.int32))
    y = host(q4_0_gemm_lora(to_dev(x), to_dev(B), N, ad[0], ad[1], none, ad[3]))
    value, bound = fp.norm_bound(x, B, 1.0, True)
    fp.check_norm(y, value, 1.05 * bound)  # all of the weights' roundings: parts known exactly
