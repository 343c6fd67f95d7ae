"""Every tile of the 8-bit products and gradients by i8_gemm_plan, and the kernel of few rows
in a gradient: with and without splits, odd
and even numbers of K steps, fewer steps than stages, half-full last tiles. Products exactly;
gradients exactly where one term makes a value, and by their norm where all do."""
import numpy as np
import pytest
import torch

import tests.built  # noqa: F401
from tests import i8_ref as ref
from tests.gpu_util import dev

#: M, K, N
GEMM = [(17, 16, 8), (17, 144, 8), (17, 272, 72), (33, 400, 136), (17, 528, 8), (17, 8208, 8),
        (100, 8208, 136), (130, 8208, 200),
        (4200, 16, 72), (2050, 144, 200), (2050, 272, 200), (2050, 400, 200), (1700, 528, 264),
        (520, 8208, 8), (257, 11008, 72), (257, 8208, 136), (257, 8208, 200),
        (65, 16, 8200), (200, 144, 4104), (1030, 272, 1000), (1030, 400, 1000), (1030, 528, 1000),
        (65, 11008, 2056), (130, 11008, 2056),
        (130, 16, 11008), (1300, 144, 1544), (1300, 272, 1544), (1300, 400, 1544), (1300, 528, 1544),
        (2050, 11008, 200), (1030, 8208, 1000),
        (257, 16, 11008), (257, 144, 11008), (257, 272, 11008), (2500, 400, 1544), (2500, 528, 1544),
        (65, 11008, 8200), (200, 11008, 6008),
        (2500, 16, 3080), (2500, 144, 3080), (2500, 272, 3080), (2500, 400, 3080), (2500, 528, 3080),
        (130, 11008, 11008), (2050, 32784, 520)]
BACKWARD = [(17, 16, 8), (17, 16, 72), (17, 16, 136), (17, 16, 200), (17, 16, 264), (17, 16, 1000),
            (17, 16, 2056), (17, 16, 8200), (17, 16, 11008), (200, 144, 3080),
            (4200, 144, 8), (4200, 144, 72), (4200, 144, 136), (4200, 144, 200), (2050, 400, 264),
            (777, 16, 2056), (520, 16, 6008), (400, 16, 8200), (400, 16, 11008),
            (130, 11008, 8), (4200, 400, 72), (4200, 400, 136), (4200, 400, 200), (4200, 400, 264),
            (1700, 16, 2056), (1030, 16, 6008), (777, 16, 8200), (777, 16, 11008),
            (17, 32784, 8), (257, 11008, 72), (1300, 3088, 136), (1300, 3088, 200),
            (1300, 3088, 264), (3100, 400, 11008), (65, 11008, 8200),
            (1, 16, 8), (16, 16, 8), (9, 144, 72), (16, 16, 2048), (16, 16, 2056), (8, 80, 4096),
            (8, 80, 4104), (3, 272, 11008), (16, 272, 11008), (16, 16, 70000), (8, 16, 140000),
            (4200, 16, 24), (4200, 16, 72), (31, 80, 2048), (500, 512, 24)]
WEIGHT = [(17, 16, 8), (65, 16, 8), (130, 16, 8), (200, 16, 8), (257, 16, 8), (1700, 16, 8),
          (2500, 16, 8), (2500, 144, 200), (2050, 272, 200),
          (17, 16, 8200), (65, 16, 8200), (130, 16, 8200), (200, 16, 8200), (257, 16, 8200),
          (2050, 16, 1000), (2500, 16, 520), (3100, 16, 1544),
          (17, 144, 8200), (65, 144, 8200), (130, 144, 8200), (200, 144, 8200), (257, 144, 8200),
          (2050, 16, 1544), (2050, 16, 3080), (4200, 16, 2056),
          (17, 32784, 8), (65, 11008, 264), (130, 272, 11008), (200, 272, 11008), (257, 400, 8200),
          (64, 16, 24), (65, 16, 24), (400, 16, 24), (1700, 16, 24), (2500, 16, 24), (17, 32784, 24),
          (4097, 144, 8), (4200, 144, 8), (2048, 4096, 16), (2049, 4096, 16), (9000, 1040, 16),
          (40000, 80, 16), (40000, 80, 8), (140000, 16, 8), (66000, 144, 16),
          (17, 16, 4104), (96, 16, 4104), (2048, 80, 40), (31, 512, 488)]
SHAPES = {"i8_gemm": GEMM, "i8_gemm_backward": BACKWARD, "i8_gemm_backward_weight": WEIGHT}


def plan(form, M, K, N):
    from moe_experts_amd import i8_gemm_plan
    return i8_gemm_plan(form, M, N, K)


@pytest.mark.parametrize("form", SHAPES)
def test_the_shapes_reach_every_tile(form):
    got = {(r, c, s > 1, steps % 2) for r, c, s, steps in (plan(form, *m) for m in SHAPES[form])}
    tiles = {(r, c) for r, c, _, _ in got}
    gradient = {(32, 128), (64, 128), (128, 128), (128, 256)}
    want = {"i8_gemm": {(32, 64), (64, 64), (64, 128), (128, 128), (128, 256), (256, 192)},
            "i8_gemm_backward": gradient | {(0, 0)},
            "i8_gemm_backward_weight": gradient | {(0, 0)}}[form]
    assert tiles == want
    for tile in tiles:
        for split in (False, True):
            if (form, tile, split) == ("i8_gemm_backward", (0, 0), True):
                continue  # by tiles
            if (form, tile, split) == ("i8_gemm_backward_weight", (128, 256), True):
                continue  # never: so many results leave nothing to split for
            for odd in (0, 1):
                assert (*tile, split, odd) in got, (tile, split, odd)


def int8(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, device=dev(), dtype=torch.int8)


def gen(*shape):
    return torch.Generator(device="cuda").manual_seed(sum(shape))


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", GEMM)
def test_gemm(M, K, N):
    from moe_experts_amd import i8_gemm
    g = gen(M, K, N)
    X, W = int8(g, M, K), int8(g, N, K)
    ones = lambda n: torch.ones(n, device=dev())
    y = i8_gemm(X, ones(M), W, ones(N), dtype=torch.float32)
    assert torch.equal(y, (X.double() @ W.double().T).float())


def picks(g, rows, cols):
    """A column for each row, and powers of two."""
    at = torch.randint(0, cols, (rows,), generator=g, device=dev())
    e = torch.randint(-20, 10, (rows,), generator=g, device=dev())
    return at, torch.exp2(e.float())


def dense(g, rows, cols):
    return (torch.randn((rows, cols), generator=g, device=dev()) * 1e-3).bfloat16()


def close(got, want):
    ref.check_norm(got.double().cpu().numpy(), want.cpu().numpy())


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", BACKWARD)
def test_backward(M, K, N):
    from moe_experts_amd import i8_gemm_backward
    g = gen(M, K, N)
    W = int8(g, N, K)
    sw = torch.exp2(torch.randint(-8, 3, (N,), generator=g, device=dev()).float())
    at, size = picks(g, M, N)
    dY = torch.zeros((M, N), device=dev()).scatter_(1, at[:, None], size[:, None])
    got = i8_gemm_backward(dY.bfloat16(), W, sw)
    assert torch.equal(got.float(), W[at].float() * (size * sw[at])[:, None])
    dY, sw = dense(g, M, N), torch.rand((N,), generator=g, device=dev()) + 0.5
    close(i8_gemm_backward(dY, W, sw), (dY.double() * sw.double()) @ W.double())


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", WEIGHT)
def test_backward_weight(M, K, N):
    from moe_experts_amd import i8_gemm_backward_weight
    g = gen(M, K, N)
    X = int8(g, M, K)
    sx = torch.exp2(torch.randint(-8, 3, (M,), generator=g, device=dev()).float())
    at, size = picks(g, N, M)
    dY = torch.zeros((N, M), device=dev()).scatter_(1, at[:, None], size[:, None]).T.contiguous()
    got = i8_gemm_backward_weight(dY.bfloat16(), X, sx)
    assert torch.equal(got.float(), X[at].float() * (size * sx[at])[:, None])
    dY, sx = dense(g, M, N), torch.rand((M,), generator=g, device=dev()) + 0.5
    left = (dY.double() * sx.double()[:, None]).T.contiguous()
    close(i8_gemm_backward_weight(dY, X, sx), left @ X.double())
