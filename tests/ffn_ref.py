"""64-bit references and error bounds of the dense feed-forward operators.

Each function returns (value, bound): the result in float64 and how far a right
implementation may be from it, element by element, counted from the roundings
the operator documents (a rounding is off by at most half a step: 2^-11 of the
value in fp16, 2^-8 in bf16, 2^-24 in fp32; below the normal range by half the
smallest subnormal)."""
import numpy as np

E16, E16_SUB = 2.0 ** -11, 2.0 ** -25
EBF, E32 = 2.0 ** -8, 2.0 ** -24
SLOPE = 1.13  # |act'| <= 1.1 (SiLU), 1.129 (GELU)


def dequant(B):
    """Q4_0 bytes [K, N/32, 18] -> float64 [K, N]."""
    B = np.ascontiguousarray(B)
    K, nb, _ = B.shape
    d = B[..., :2].copy().view(np.float16).astype(np.float64)
    q = np.empty((K, nb, 32))
    q[..., 0::2] = B[..., 2:] & 15
    q[..., 1::2] = B[..., 2:] >> 4
    return ((q - 8) * d).reshape(K, nb * 32)


def scales(B):
    """|d| of every weight, float64 [K, N]."""
    return np.repeat(np.abs(B[..., :2].copy().view(np.float16).astype(np.float64))[..., 0], 32, 1)


def act(z, kind):
    """(value, slope)."""
    c = np.sqrt(2 / np.pi)
    if kind == "silu":
        s = 1 / (1 + np.exp(-z))
        return z * s, s + z * s * (1 - s)
    t = np.tanh(c * (z + 0.044715 * z ** 3))
    return z / 2 * (1 + t), (1 + t) / 2 + z / 2 * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def product32(x, B):
    """x . deq(B) with fp32 products and sums. The nibbles 0..15 are summed unsigned and
    8 * sum(x * d) is taken off, so every partial sum stays under sum |x| * d * 24."""
    x = x.astype(np.float64)
    K = x.shape[1]
    return x @ dequant(B), (K + 64) * E32 * 24 * (np.abs(x) @ scales(B)) + 1e-30


def product16(x, B):
    """x . deq(B) with each weight rounded to fp16 and fp32 sums."""
    x = x.astype(np.float64)
    w = dequant(B)
    s = np.abs(x) @ np.abs(w)
    return x @ w, (E16 + (x.shape[1] + 8) * E32) * s * (1 + E16) + \
        E16_SUB * np.abs(x).sum(1, keepdims=True)


def gate(g, eg, u, eu, kind):
    """act(g) * u and its error from those of g and u; the activation itself costs a few fp32
    roundings, of its argument too (its slope times the argument's size is below 4 |z|)."""
    a, _ = act(g, kind)
    ea = SLOPE * eg + 32 * E32 * (np.abs(a) + np.abs(g))
    return a * u, ea * (np.abs(u) + eu) + np.abs(a) * eu + 4 * E32 * np.abs(a * u)


def round16(v, e):
    return v, e + E16 * (np.abs(v) + e) + E16_SUB


def glu(x, Wg, Wu, kind):
    return gate(*product32(x, Wg), *product32(x, Wu), kind)


def glu_gemm(x, Wg, Wu, kind):
    """((h, bound), (g, bound), (u, bound))."""
    g, u = product16(x, Wg), product16(x, Wu)
    return round16(*gate(*g, *u, kind)), round16(*g), round16(*u)


def _through(rows, e_rows, mats):
    """sum_i rows[i] . mats[i]^T, the rows scaled together by a power of two that takes their
    largest value to 2^13..2^14 and rounded to fp16."""
    big = np.max([np.abs(r).max(1) for r in rows], axis=0)[:, None]
    value, bound = 0.0, 0.0
    terms = sum(m.shape[1] for m in mats)
    for r, e, w in zip(rows, e_rows, mats):
        aw = np.abs(w).T
        value = value + r @ w.T
        e16 = e + E16 * (np.abs(r) + e) + E16_SUB * big * 2.0 ** -12
        bound = bound + (np.abs(r) + e16) @ aw * (E16 + (terms + 8) * E32) + e16 @ aw \
            + E16_SUB * np.abs(r).sum(1, keepdims=True)
    return value, bound + EBF * (np.abs(value) + bound) + 1e-38


def glu_backward(dh, g, u, Wg, Wu, kind):
    dh, g, u = (v.astype(np.float64) for v in (dh, g, u))
    a, slope = act(g, kind)
    # value and slope in fp32: relative steps of terms that are below (1 + |z|) * 4
    few = 64 * E32 * (1 + np.abs(g))
    return _through([dh * u * slope, dh * a], [np.abs(dh * u) * few, np.abs(dh) * few],
                    [dequant(Wg), dequant(Wu)])


def gemm_backward(dy, B):
    dy = dy.astype(np.float64)
    return _through([dy], [np.zeros_like(dy)], [dequant(B)])


def adapters(x, A, Bl, ids, scale, half):
    """scale * (x . A^T) . B^T of each row's adapter. half: the narrow product may be rounded to
    fp16 relative to its row's largest value."""
    x, A, Bl, scale = (v.astype(np.float64) for v in (x, A, Bl, scale))
    M, K = x.shape
    R, N = A.shape[1], Bl.shape[1]
    value, bound = np.zeros((M, N)), np.zeros((M, N))
    for i in range(A.shape[0]):
        m = np.nonzero(ids == i)[0]
        if not m.size:
            continue
        t = x[m] @ A[i].T
        et = (K + 8) * E32 * (np.abs(x[m]) @ np.abs(A[i]).T)
        if half:
            et = et + E16 * (np.abs(t) + et) + E16_SUB * np.abs(t).max(1, keepdims=True) * 2
        s = abs(scale[i])
        value[m] = scale[i] * (t @ Bl[i].T)
        bound[m] = s * (et @ np.abs(Bl[i]).T) + \
            s * (R + 8) * E32 * ((np.abs(t) + et) @ np.abs(Bl[i]).T)
    return value, bound


def gemv_lora(x, B, A, Bl, ids, scale):
    y, e = product32(x, B)
    a, ea = adapters(x, A, Bl, ids, scale, False)
    return y + a, e + ea + 4 * E32 * (np.abs(y) + np.abs(a))


def gemm_lora(x, B, A, Bl, ids, scale):
    y, e = product16(x, B)
    a, ea = adapters(x, A, Bl, ids, scale, True)
    return round16(y + a, e + ea + 4 * E32 * (np.abs(y) + np.abs(a)))


def check(got, ref, what=""):
    """Every element finite and within its bound; returns the largest share of a bound used."""
    value, bound = ref
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == value.shape, f"{what}: shape {got.shape}"
    assert np.isfinite(got).all(), f"{what}: not finite"
    share = np.abs(got - value) / bound
    worst = float(share.max()) if share.size else 0.0
    at = np.unravel_index(share.argmax(), share.shape) if share.size else ()
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound at {at}"
    return worst
