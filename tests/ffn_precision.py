"""Bounds that see how exactly the dense feed-forward forms its products, where the
element-by-element bounds of ffn_ref.py (worst cases over the contraction) do not.

Norms: independent roundings add up in their squares. Against the value in 64 bits
a result in fp16 is off by its own rounding, known exactly, by what is left of the
weights' roundings, and by the fp32 sums: K additions, each off by 2^-24 of a
partial sum that is on the whole no larger than the result.

Differences: rows of x that hold 1 and -1 and a matrix whose rows differ by a few
last places of their scales, so that the products cancel but for what rounding a
weight to fp16 would take. Every result is a small whole number of those places,
held exactly by fp16, and has to be met bit by bit."""
import numpy as np

from tests import ffn_ref as ref

#: Share of the weights' roundings that a tile GEMM of the forward forms may leave: their
#: products take x cut to 3 significant bits, off by less than a quarter of x (a tenth on the
#: whole).
LEFT = 0.25


def rounded16(w):
    return w.astype(np.float16).astype(np.float64)


def norm_bound(x, B, left, own):
    """How far (2-norm) x . deq(B) may be from its value: (value, norm). left: share of the
    weights' roundings that may be left; own: whether the result is rounded to fp16."""
    x, w = x.astype(np.float64), ref.dequant(B)
    y = x @ w
    parts = [left * np.linalg.norm(x @ (w - rounded16(w))),
             2 * np.sqrt(x.shape[1]) * ref.E32 * np.linalg.norm(y)]
    if own:
        parts.append(np.linalg.norm(y - rounded16(y)))
    return y, float(np.sqrt(np.sum(np.square(parts))))


def check_norm(got, value, bound, what=""):
    off = float(np.linalg.norm(np.asarray(got, dtype=np.float64) - value))
    assert off <= bound, f"{what}: off by {off:.4g}, {off / bound:.3g} of the bound"


def near_rows(seed, K, N, place=-18):
    """A Q4_0 matrix whose rows have the same nibbles and, column block by column block, scales
    that differ by a few last places, of 2^place (-24 to 2: the normal scales of fp16 whose
    weights it holds)."""
    r = np.random.default_rng(seed)
    nb = N // 32
    q = r.integers(0, 256, (1, nb, 16), dtype=np.uint8)
    d = (r.integers(1100, 1900, (1, nb)) + r.integers(0, 7, (K, nb))) * 2.0 ** place
    B = np.empty((K, nb, 18), dtype=np.uint8)
    B[..., 2:] = q
    B[..., :2] = d.astype(np.float16)[..., None].view(np.uint8)
    return B


def differences(M, K, at=0):
    """Rows of x with 1 and -1 at two places, which over the rows take every k: those of row m
    begin at m + at."""
    x = np.zeros((M, K), dtype=np.float16)
    m = np.arange(M)
    a = (m + at) % K
    x[m, a] = 1
    x[m, (a + 1 + m % (K - 1)) % K] = -1
    return x


def exact_differences(x, B):
    y = x.astype(np.float64) @ ref.dequant(B)
    assert (rounded16(y) == y).all()
    return y


def _bf16(v):
    """v rounded to bf16, to nearest, ties to even."""
    u = np.ascontiguousarray(v, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def gradient_bound(rows, mats):
    """How far (2-norm) sum_i rows[i] . mats[i]^T may be from its value, as a gradient: the rows
    scaled together to 2^13..2^14 and rounded to fp16, the weights rounded to fp16, the result to
    bf16. The parts are known exactly and do not depend on one another; their squares add up to
    within a few hundredths (of M * K products of them)."""
    big = np.max([np.abs(r).max(1) for r in rows], axis=0)
    scale = 2.0 ** (13 - np.floor(np.log2(np.where(big > 0, big, 1.0))))[:, None]
    value = sum(r @ w.T for r, w in zip(rows, mats))
    weights = sum(r @ (w - rounded16(w)).T for r, w in zip(rows, mats))
    operand = sum((r - rounded16(r * scale) / scale) @ w.T for r, w in zip(rows, mats))
    terms = sum(w.shape[1] for w in mats)
    parts = [np.linalg.norm(v) for v in (value - _bf16(value), weights, operand)]
    parts.append(2 * np.sqrt(terms) * ref.E32 * np.linalg.norm(value))
    return value, 1.05 * float(np.sqrt(np.sum(np.square(parts))))
