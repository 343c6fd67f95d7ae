"""The 8-bit operators' references against what is known without them (CPU)."""
from fractions import Fraction

import numpy as np
import pytest

from moe_experts_amd import datagen
from tests import i8_ref as ref


def test_rows_by_hand():
    # largest 127 * 2^-3: scale 2^-3; halves go to the even neighbour
    x = np.float32([[15.875, 0.0625, 0.1875, 0.3125, -0.0625, -0.1875, 0.0624, 0.0626]])
    q, s = ref.rows(x)
    assert s[0] == 0.125 and q.tolist() == [[127, 0, 2, 2, 0, -2, 0, 1]]
    q, s = ref.rows(np.float32([[0, -0.0], [1, np.inf], [np.nan, 2], [-127, 64]]))
    assert s[0] == 0 and np.isnan(s[1]) and np.isnan(s[2]) and s[3] == 1
    assert q.tolist() == [[0, 0], [0, 0], [0, 0], [-127, 64]]


@pytest.mark.parametrize("size", [1.0, 1e-30, 1e-40, 1e38])
def test_rows_against_whole_fractions(size):
    """The rounding decided in rational numbers, over values close to halves of their scale."""
    r = datagen.rng(3)
    x = (r.standard_normal((6, 200)) * size).astype(np.float32)
    s = np.abs(x).max(1) / np.float32(127)
    near = np.round(r.uniform(-126, 126, (6, 100))) + 0.5
    x[:, 1:101] = near * s[:, None]
    x[:, 1:101:3] = np.nextafter(x[:, 1:101:3], np.float32(0))
    q, s = ref.rows(x)
    for m in range(6):
        sm = Fraction(float(s[m]))
        for k in range(200):
            t = Fraction(float(x[m, k])) / sm
            assert q[m, k] == max(-127, min(127, round(t)))  # Fraction rounds halves to even


def test_product_is_whole():
    r = datagen.rng(4)
    X, W = (r.integers(-128, 128, (n, 70000)).astype(np.int8) for n in (2, 3))
    want = [[sum(int(a) * int(b) for a, b in zip(x, w)) for w in W] for x in X]
    assert (ref.product(X, W) == np.array(want, dtype=np.float64)).all()


@pytest.mark.parametrize("M,N,K", [(40, 64, 96), (300, 64, 512)])
def test_mistakes_are_seen(M, N, K):
    """One token's term left out of a weight gradient, two exchanged columns, a scale forgotten:
    each is outside what the checks allow."""
    r = datagen.rng(5)
    X, sx = ref.rows(datagen.activations(6, M, K))
    dY = r.standard_normal((M, N))
    want = ref.backward_weight(dY, X, sx)
    ref.check(want[0], want)
    ref.check_norm(want[0], want[0])
    wrong = [ref.backward_weight(dY[:-1], X[:-1], sx[:-1])[0],
             ref.backward_weight(dY[:, np.r_[1, 0, 2:N]], X, sx)[0],
             ref.backward_weight(dY, X, np.where(np.arange(M) == 7, 1, sx).astype(np.float32))[0]]
    for v in wrong:
        with pytest.raises(AssertionError):
            ref.check_norm(v, want[0])
