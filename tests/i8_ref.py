"""64-bit references and error bounds of the 8-bit operators.

Each function returns (value, bound): the result in float64 and how far a right
implementation may be from it, element by element, counted from the roundings the
operator documents (half a step: 2^-11 of the value in fp16, 2^-8 in bf16, 2^-24 in
fp32; below the normal range half the smallest subnormal). `rows` is exact."""
import numpy as np

E16, EBF, E32 = 2.0 ** -11, 2.0 ** -8, 2.0 ** -24
HALF_STEP = {"fp32": (E32, 2.0 ** -150), "fp16": (E16, 2.0 ** -25), "bf16": (EBF, 2.0 ** -134)}


def rows(x):
    """(int8, fp32 scale) of the rows of x: the fp32 quotient of two fp32 numbers is correctly
    rounded in numpy, and so is the float64 one. A quotient of two 24-bit numbers that is not
    itself a half differs from every half below 128 by at least 2^-26, so that rounding it to 53
    bits does not make it one."""
    x = np.asarray(x, dtype=np.float32)
    ok = np.isfinite(x).all(axis=1)
    amax = np.abs(np.where(ok[:, None], x, 0)).max(axis=1)
    s = (amax / np.float32(127)).astype(np.float32)
    safe = np.where(s > 0, s, 1).astype(np.float64)
    q = np.rint(np.where(ok[:, None], x, 0).astype(np.float64) / safe[:, None])
    q = np.where((s > 0)[:, None], np.clip(q, -127, 127), 0).astype(np.int8)
    return q, np.where(ok, s, np.float32(np.nan)).astype(np.float32)


def product(X, W):
    """Whole numbers, exact: partial sums of 64 values of k stay below 2^21, so float32 products
    of them are exact, and float64 adds them exactly."""
    X, W = np.asarray(X), np.asarray(W)
    out = np.zeros((X.shape[0], W.shape[0]))
    if X.shape[1] <= 1 << 16:  # |sum| < 2^30 < 2^53
        return X.astype(np.float64) @ W.astype(np.float64).T
    for k in range(0, X.shape[1], 1 << 16):
        out += X[:, k:k + (1 << 16)].astype(np.float64) @ W[:, k:k + (1 << 16)].astype(np.float64).T
    return out


def gemm(X, sx, W, sw, kind):
    """(sum * sx) * sw, each step rounded to fp32, then to the result's type."""
    sx, sw = sx.astype(np.float64)[:, None], sw.astype(np.float64)
    v = product(X, W) * sx * sw
    rel, sub = HALF_STEP[kind]
    few = 3 * E32 * (1 + 4 * E32)
    tiny = 2.0 ** -150 * (1 + np.abs(sw))  # the two fp32 products below the normal range
    e = few * np.abs(v) + tiny
    return v, e + rel * (np.abs(v) + e) + sub


def _contract(t, e_t, big, b, depth):
    """sum_c t[i][c] * b[c][j]: t, known to fp32 steps (e_t), is rounded to fp16 after a power of
    two has taken its rows' largest (big) to 2^13 or more; fp32 sums; bf16 results."""
    ab, at = np.abs(b), np.abs(t)
    e16 = e_t + E16 * (at + e_t) + 2.0 ** -25 * 2.0 ** -13 * big
    v = t @ b
    e = e16 @ ab + (depth + 16) * E32 * ((at + e16) @ ab)
    rel, sub = HALF_STEP["bf16"]
    return v, e + rel * (np.abs(v) + e) + sub


def backward(dY, W, sw):
    t = dY.astype(np.float64) * sw.astype(np.float64)
    big = np.abs(t).max(axis=1, keepdims=True)
    return _contract(t, E32 * np.abs(t) + 2.0 ** -150, big, W.astype(np.float64), t.shape[1])


def backward_weight(dY, X, sx):
    t = (dY.astype(np.float64) * sx.astype(np.float64)[:, None]).T
    big = np.abs(t).max(axis=1, keepdims=True)
    return _contract(np.ascontiguousarray(t), E32 * np.abs(t) + 2.0 ** -150, big,
                     X.astype(np.float64), t.shape[1])


def check(got, ref, what=""):
    """Every element finite and within its bound."""
    value, bound = ref
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == value.shape, f"{what}: shape {got.shape}"
    assert np.isfinite(got).all(), f"{what}: not finite"
    share = np.abs(got - value) / bound
    worst = float(share.max()) if share.size else 0.0
    at = np.unravel_index(share.argmax(), share.shape) if share.size else ()
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound at {at}"
    return worst


def check_norm(got, value, what=""):
    """A gradient's error as a whole. The bf16 rounding of the result is at most 2^-8 of every
    element, and so of the norm; the fp16 roundings of the terms are independent of one another
    and of mean zero, so that together they add far less than 2^-11 of the norm. One of 4096 equal
    terms left out would be 2^-6."""
    err = np.linalg.norm(np.asarray(got, dtype=np.float64) - value)
    norm = np.linalg.norm(value)
    assert err <= (EBF + E16) * norm, f"{what}: error {err / norm:.3g} of the norm"
