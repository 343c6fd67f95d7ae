"""Gradients of the 8-bit product whose terms lie far apart: results that rest on terms far below
their row's largest, because the largest meet zeros, are as near as any other.

The bound holds no part of a row's largest value: each term within half a step of fp16 of itself;
what fp16 loses of terms below 2^-27 of their row's largest (its normal range ends there at the
latest) either left out, where it is as little of a result's terms together, or within half a step
of bf16 of itself, which is at most that of the term; sums in fp32 and the result's rounding to
bf16. Terms stay above 2^-139 of a row's largest, the documented limit."""
import numpy as np
import pytest
import torch

from moe_experts_amd import datagen
from tests import i8_ref as ref
from tests.gpu_util import (dev, guarded, guarded_ws, guards_intact, to_dev,
                            ws_guards_intact)

pytestmark = pytest.mark.gpu


def host(t):
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16().to(dev())


def near(t, b):
    """sum_c t[i][c] * b[c][j] and its bound."""
    b = b.astype(np.float64)
    v, size = t @ b, np.abs(t) @ np.abs(b)
    # the product dY * scale in fp32, the rounding to fp16, what falls below it, fp32 sums
    small = np.where(np.abs(t) < 2.0 ** -27 * np.abs(t).max(axis=1, keepdims=True), np.abs(t), 0)
    e = (ref.E32 + 2 * ref.E16 * (1 + ref.E32) + (t.shape[1] + 16) * ref.E32 * (1 + 2 * ref.E16)) * size
    e += ref.EBF * (1 + ref.E32) * (small @ np.abs(b))
    rel, sub = ref.HALF_STEP["bf16"]
    return v, e + rel * (np.abs(v) + e) + sub


def spread(seed, rows, depth, gap):
    """Values [rows][depth]: a few of each row 2^gap above the rest, and which columns those are;
    "all": every size from 1 to 2^-110."""
    r = datagen.rng(seed)
    v = r.standard_normal((rows, depth))
    v = np.where(np.abs(v) < 0.05, 0.5, v)
    large = np.zeros(depth, dtype=bool)
    large[r.choice(depth, max(1, depth // 40), replace=False)] = True
    if gap == "all":
        return v * 2.0 ** r.permutation(np.linspace(0, -110, depth)), large
    return np.where(large, v, v * 2.0 ** -gap), large


def operand(seed, depth, cols, large):
    """int8 [depth][cols] that has zeros for the large terms in two of three columns, and is sparse
    in one."""
    r = datagen.rng(seed)
    b = r.integers(-128, 128, (depth, cols)).astype(np.int8)
    b[np.ix_(large, np.arange(cols) % 3 != 0)] = 0
    thin = np.flatnonzero(np.arange(cols) % 3 == 2)
    b[:, thin] *= r.random((depth, len(thin))) < 0.01
    return b


GAPS = [20, 27, 30, 34, 40, 60, 110, "all"]
#: rows, depth, cols and whether tiles serve the input's and the weights' gradient: few rows, groups
#: of rows, tiles with and without splits, transposed by one kernel and by two
SHAPES = [(1, 64, 48, False, None), (5, 200, 80, False, None), (8, 4096, 272, False, False),
          (16, 2048, 144, False, False), (40, 1000, 272, False, False),
          (40, 4104, 272, True, True), (72, 2056, 4112, True, True), (264, 512, 1040, True, True),
          (264, 136, 4112, True, True), (136, 8200, 272, True, True), (4112, 264, 144, True, True),
          (2104, 72, 8208, True, True), (1032, 200, 6032, True, True)]


def tiled(form, M, N, K):
    from moe_experts_amd import i8_gemm_plan
    return i8_gemm_plan(form, M, N, K)[0] > 0


@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("rows,depth,cols,tiles", [s[:4] for s in SHAPES])
def test_input(rows, depth, cols, tiles, gap):
    from moe_experts_amd import i8_gemm_backward
    assert tiled("i8_gemm_backward", rows, depth, cols) == tiles
    v, large = spread(1, rows, depth, gap)
    W = operand(2, depth, cols, large)
    sw = np.exp(datagen.rng(3).standard_normal(depth) - 4).astype(np.float32)
    dY = bf16(v * 2.0 ** datagen.rng(4).integers(-30, 30, (rows, 1)))
    got = i8_gemm_backward(dY, to_dev(W), to_dev(sw))
    ref.check(host(got), near(host(dY).astype(np.float64) * sw.astype(np.float64), W))


@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("rows,depth,cols,tiles", [(*s[:3], s[4]) for s in SHAPES if s[4] is not None]
                         + [(8, 777, 80, False), (16, 9001, 80, False), (16, 70000, 16, True),
                            (8, 33, 48, False), (264, 1, 16, False), (264, 131, 4112, True)])
def test_weights(rows, depth, cols, tiles, gap):
    from moe_experts_amd import i8_gemm_backward_weight
    assert tiled("i8_gemm_backward_weight", depth, rows, cols) == tiles
    v, large = spread(5, rows, depth, gap)
    X = operand(6, depth, cols, large)
    sx = np.exp(datagen.rng(7).standard_normal(depth) - 4).astype(np.float32)
    dY = bf16((v * 2.0 ** datagen.rng(8).integers(-30, 30, (rows, 1))).T)
    got = i8_gemm_backward_weight(dY, to_dev(X), to_dev(sx))
    t = np.ascontiguousarray((host(dY).astype(np.float64) * sx.astype(np.float64)[:, None]).T)
    ref.check(host(got), near(t, X))


@pytest.mark.parametrize("rows,depth,cols", [s[:3] for s in SHAPES if s[0] > 1])
def test_far_terms_stay_with_their_row(rows, depth, cols):
    """One row with far terms among rows without: those are what they are beside any other, and
    a call is what it is when it is repeated, bitwise."""
    from moe_experts_amd import i8_gemm_backward, i8_gemm_backward_weight
    r = datagen.rng(9)
    v, large = spread(10, rows, depth, 40)
    B = to_dev(operand(11, depth, cols, large))
    s = to_dev(np.exp(r.standard_normal(depth) - 4).astype(np.float32))
    plain = np.where(np.abs(v) < 2.0 ** -20, v * 2.0 ** 40, v)
    mixed = plain.copy()
    mixed[rows // 2] = v[rows // 2]
    keep = [i for i in range(rows) if i != rows // 2]
    was, got = (i8_gemm_backward(bf16(a), B, s) for a in (plain, mixed))
    assert torch.equal(was[keep], got[keep]) and not torch.equal(was, got)
    assert torch.equal(got, i8_gemm_backward(bf16(mixed), B, s))
    if rows % 8 == 0:
        was, got = (i8_gemm_backward_weight(bf16(a.T), B, s) for a in (plain, mixed))
        assert torch.equal(was[keep], got[keep]) and not torch.equal(was, got)
        assert torch.equal(got, i8_gemm_backward_weight(bf16(mixed.T), B, s))


@pytest.mark.parametrize("gap", [40, "all"])
@pytest.mark.parametrize("rows,depth,cols", [(16, 2048, 144), (40, 4104, 272), (72, 2056, 4112),
                                             (264, 512, 1040), (136, 8200, 272)])
def test_dead_channels(rows, depth, cols, gap):
    """Columns of zeros beside others, under rows with far terms: exact zeros, and their neighbours
    within the bound."""
    from moe_experts_amd import i8_gemm_backward, i8_gemm_backward_weight
    v, large = spread(12, rows, depth, gap)
    B = operand(13, depth, cols, large)
    dead = datagen.rng(14).random(cols) < 0.3
    dead[[0, cols - 1]] = True
    B[:, dead] = 0
    s = np.exp(datagen.rng(15).standard_normal(depth) - 4).astype(np.float32)
    dY = bf16(v)
    want = near(host(dY).astype(np.float64) * s.astype(np.float64), B)
    results = [i8_gemm_backward(dY, to_dev(B), to_dev(s))]
    if rows % 8 == 0:
        results.append(i8_gemm_backward_weight(dY.T.contiguous(), to_dev(B), to_dev(s)))
    for got in map(host, results):
        ref.check(got, want)
        assert not got[:, dead].any()


def test_all_results_rest_on_far_terms():
    """A token whose row is zeros, 2^40 above the rest in the gradient: every result of both kernels
    rests on what fp16 loses, and takes the contraction twice, not more."""
    from moe_experts_amd import i8_gemm_backward_weight
    for M, N, K in ((777, 1536, 1040), (1999, 16, 272), (9001, 72, 272)):
        r = datagen.rng(16)
        X = r.integers(-127, 128, (M, K)).astype(np.int8)
        X[M // 2] = 0
        v = r.standard_normal((M, N))
        v[M // 2] *= 2.0 ** 40
        sx = np.exp(r.standard_normal(M) - 4).astype(np.float32)
        dY = bf16(v)
        got = host(i8_gemm_backward_weight(dY, to_dev(X), to_dev(sx)))
        t = np.ascontiguousarray((host(dY).astype(np.float64) * sx.astype(np.float64)[:, None]).T)
        ref.check(got, near(t, X))


@pytest.mark.parametrize("rows,depth,cols", [(8, 4096, 272), (40, 1000, 272), (40, 4104, 272),
                                             (72, 2056, 4112), (136, 8200, 272), (4112, 264, 144),
                                             (2104, 72, 8208), (264, 131, 4112)])
def test_memory_around_is_left_alone(rows, depth, cols):
    """The second left operand is written and read within the workspace, whatever that holds before;
    results are bitwise those of another."""
    import moe_experts_amd as q4
    v, large = spread(17, rows, depth, "all")
    B = to_dev(operand(18, depth, cols, large))
    s = to_dev(np.exp(datagen.rng(19).standard_normal(depth) - 4).astype(np.float32))
    forms = [("i8_gemm_backward", bf16(v), (rows, depth, cols), "dX")] if depth % 8 == 0 else []
    forms.append(("i8_gemm_backward_weight", bf16(v.T), (depth, rows, cols), "dW"))
    for form, dY, (M, N, K), out in forms:
        if N % 8:
            continue
        need = getattr(q4, form + "_workspace_bytes")(M, N, K)
        seen = []
        for fill in (0xFF, 0x00):
            full, y = guarded(rows * cols, torch.bfloat16, fill=7.0)
            wfull, ws = guarded_ws(need, fill=fill)
            getattr(q4, form)(dY, B, s, **{out: y.view(rows, cols)}, ws=ws)
            seen.append(y.clone())
            assert guards_intact(full, rows * cols, fill=7.0)
            assert ws_guards_intact(wfull, need, fill=fill)
        assert torch.equal(*seen)


@pytest.mark.parametrize("rows,depth,cols", [(8, 4096, 272), (40, 4104, 272), (264, 512, 1040),
                                             (136, 8200, 272)])
def test_replays_with_and_without_far_terms(rows, depth, cols):
    """A captured call whose inputs come to have far terms, lose them and have them again: every
    replay is the eager call, bitwise."""
    from moe_experts_amd import i8_gemm_backward, i8_gemm_backward_weight
    v, large = spread(20, rows, depth, 40)
    plain = np.where(np.abs(v) < 2.0 ** -20, v * 2.0 ** 40, v)
    B = to_dev(operand(21, depth, cols, large))
    s = to_dev(np.exp(datagen.rng(22).standard_normal(depth) - 4).astype(np.float32))
    inputs = [bf16(plain), bf16(v)]
    dY = inputs[0].clone()
    dYt = dY.T.contiguous()
    dX = torch.zeros((rows, cols), dtype=torch.bfloat16, device=dev())
    dW = torch.zeros_like(dX)

    def call():
        i8_gemm_backward(dY, B, s, dX=dX)
        i8_gemm_backward_weight(dYt, B, s, dW=dW)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for which in (1, 0, 1, 1, 0):
        dY.copy_(inputs[which])
        dYt.copy_(inputs[which].T)
        dX.fill_(77)
        dW.fill_(77)
        g.replay()
        got = dX.clone(), dW.clone()
        call()
        assert torch.equal(got[0], dX) and torch.equal(got[1], dW)


@pytest.mark.parametrize("rows,depth,cols", [(8, 4096, 272), (40, 1000, 272), (40, 4104, 272),
                                             (264, 512, 1040), (136, 8200, 272)])
def test_broken_rows_beside_far_terms(rows, depth, cols):
    """Rows with an infinity or a NaN among rows with far terms: none of their results is finite, and
    the others are what they were."""
    from moe_experts_amd import i8_gemm_backward, i8_gemm_backward_weight
    v, large = spread(23, rows, depth, "all")
    B = to_dev(operand(24, depth, cols, large))
    s = to_dev(np.exp(datagen.rng(25).standard_normal(depth) - 4).astype(np.float32))
    broken = v.copy()
    broken[2, depth // 2], broken[5, 0] = np.inf, np.nan
    keep = [i for i in range(rows) if i not in (2, 5)]
    for call in (lambda a: i8_gemm_backward(bf16(a), B, s),
                 lambda a: i8_gemm_backward_weight(bf16(a.T), B, s)):
        was, got = call(v), call(broken)
        assert torch.equal(got[keep], was[keep])
        assert not torch.isfinite(got[[2, 5]].float()).any()
