"""What the bounds of ffn_precision.py see, without a GPU: mistakes planted in the
products are outside them, right products inside."""
import numpy as np
import pytest

from moe_experts_amd import datagen
from tests import ffn_precision as fp
from tests import ffn_ref as ref

M, K, N = 96, 576, 128


def product(x, B, plant):
    """x . deq(B) as the tiles form it, in 64 bits, with a mistake."""
    x, w = x.astype(np.float64), ref.dequant(B)
    hi = fp.rounded16(w)
    rest = w - hi
    x8 = (x.astype(np.float16).view(np.uint16) & 0xff00).view(np.float16).astype(np.float64)
    k = np.arange(x.shape[1])
    if plant == "none":
        return x @ w
    if plant == "cut":                       # as the tiles do it: x cut to 3 bits
        return x @ hi + x8 @ rest
    if plant == "missing":
        return x @ hi
    if plant == "sign":
        return x @ hi - x8 @ rest
    if plant == "quarter":                   # the roundings of a quarter of k only
        return x @ hi + (x8 * (k % 64 < 16)) @ rest
    if plant == "quarters swapped":
        return x @ hi + x8[:, (k // 64) * 64 + (k + 16) % 64] @ rest
    if plant == "column":
        return x @ hi + x8 @ np.roll(rest, 1, axis=1)
    if plant == "scale":
        return x @ hi + 2 * (x8 @ rest)
    if plant == "row":
        return x @ hi + np.roll(x8, 1, axis=0) @ rest
    raise ValueError(plant)


RIGHT = ("none", "cut")
WRONG = ("missing", "sign", "quarter", "quarters swapped", "column", "scale", "row")


@pytest.mark.parametrize("plant", RIGHT + WRONG)
def test_norms(plant):
    x = datagen.to_f16(datagen.activations(1, M, K))
    B = datagen.q4_0_random(2, K, N)
    value, bound = fp.norm_bound(x, B, fp.LEFT, True)
    got = fp.rounded16(product(x, B, plant))
    if plant in RIGHT:
        fp.check_norm(got, value, bound)
    else:
        with pytest.raises(AssertionError, match="of the bound"):
            fp.check_norm(got, value, bound)


@pytest.mark.parametrize("place", [-24, -18, 2])
@pytest.mark.parametrize("plant", RIGHT + WRONG)
def test_differences(plant, place):
    x, B = fp.differences(M, K), fp.near_rows(3, K, N, place)
    got = fp.rounded16(product(x, B, plant))
    assert (got == fp.exact_differences(x, B)).all() == (plant in RIGHT)


def test_differences_take_every_k():
    x = fp.differences(64, 64)
    assert (x == 1).any(0).all() and (np.abs(x.astype(np.int32)).sum(1) == 2).all()


def test_every_rounding_is_held_by_an_eight_bit_float():
    """(q - 8) * d - fp16((q - 8) * d), times 2^8, is its own upper byte, for every nibble and
    every scale whose weights are finite."""
    d = np.arange(1 << 16, dtype=np.uint16).view(np.float16)
    d = d[np.isfinite(d)]
    for a in range(-8, 8):
        exact = a * d.astype(np.float64)
        with np.errstate(over="ignore"):
            w = np.float16(a) * d
        fine = np.isfinite(w)
        rest = (exact[fine] - w[fine].astype(np.float64)) * 256
        held = (rest.astype(np.float16).view(np.uint16) & 0xff00).view(np.float16)
        assert (held.astype(np.float64) == rest).all()


@pytest.mark.parametrize("plant,right", [("none", True), ("half operand", True),
                                         ("weights cut", False), ("operand cut", False),
                                         ("columns of the other", False), ("matrices swapped", False)])
def test_gradient_norms(plant, right):
    """Gradients through two matrices, against what may be rounded on the way."""
    r = datagen.rng(4)
    rows = [r.standard_normal((M, N)) * np.exp(r.standard_normal((M, 1))) for _ in range(2)]
    mats = [ref.dequant(datagen.q4_0_random(s, K, N)) for s in (5, 6)]
    value, bound = fp.gradient_bound(rows, mats)
    cut = lambda v: (v.astype(np.float16).view(np.uint16) & 0xfff0).view(np.float16).astype(float)
    got = [v.copy() for v in rows], [fp.rounded16(m) for m in mats]
    if plant == "half operand":
        got[0][:] = [fp.rounded16(v) for v in rows]
    elif plant == "weights cut":
        got[1][:] = [cut(m) for m in mats]
    elif plant == "operand cut":
        got[0][:] = [cut(v) for v in rows]
    elif plant == "columns of the other":
        got[0][1][:, 64:] = rows[0][:, 64:]
    elif plant == "matrices swapped":
        got[1].reverse()
    dx = fp._bf16(sum(a @ w.T for a, w in zip(*got)))
    if right:
        fp.check_norm(dx, value, bound)
    else:
        with pytest.raises(AssertionError, match="of the bound"):
            fp.check_norm(dx, value, bound)
