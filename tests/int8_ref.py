"""Plain forms of the products in 8-bit integers, in NumPy.

The quantiser and the scaling are a handful of fp32 operations, each rounded once as
IEEE 754 says; the sums are whole numbers, exact in 64 bits. Results are therefore
compared bit for bit.
"""

import numpy as np

from oracle import bf16_bits_from_f64


def quantise(x):
    """x float32 [rows][cols] -> int8 codes, float32 scales."""
    x = np.asarray(x, np.float32)
    top = np.max(np.abs(np.where(np.isnan(x), np.float32(np.inf), x)), axis=1)
    live = np.isfinite(top) & (top >= np.float32(2.0 ** -120))
    safe = np.where(live, top, np.float32(1))
    inv = np.float32(127) / safe
    q = np.zeros(x.shape, np.int8)
    q[live] = np.rint(x[live] * inv[live, None]).astype(np.int8)
    scale = np.where(live, safe / np.float32(127), np.float32(0))
    return q, np.where(np.isfinite(top), scale, np.float32(np.nan)).astype(np.float32)


def product(a, sa, b, sb):
    """bf16 bits of (fl32(a b^T) sa) sb; a [M][K], b [N][K] int8."""
    acc = a.astype(np.float64) @ b.astype(np.float64).T      # (whole numbers below 2^53)
    with np.errstate(invalid="ignore", over="ignore"):
        v = acc.astype(np.float32) * np.asarray(sa, np.float32)[:, None] * np.asarray(sb, np.float32)[None, :]
    return bf16_bits_from_f64(v.astype(np.float64))


def contiguous(a, sa, b, sb, offsets, before):
    """before: d's bits [M_total][N]; rows of no expert keep them."""
    d = before.copy()
    for g, (i, j) in enumerate(zip(offsets, offsets[1:])):
        if j > i:
            d[i:j] = product(a[i:j], sa[i:j], b[g], sb[g])
    return d


def masked(a, sa, b, sb, counts, before):
    d = before.copy()
    for g, n in enumerate(counts):
        n = min(max(int(n), 0), a.shape[1])
        if n:
            d[g, :n] = product(a[g, :n], sa[g, :n], b[g], sb[g])
    return d
