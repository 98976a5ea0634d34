"""The AdamW step in NumPy: states as the fp32 operations of the definition, each rounded once
(compared bit for bit), parameters in fp64, 8-bit states by the definition of their rounding."""

import math

import numpy as np

F = np.float32
BLOCK = 128


def mix(h):
    h = np.asarray(h, np.uint64)
    low = np.uint64(0xFFFFFFFF)
    h = ((h ^ (h >> np.uint64(16))) * np.uint64(0x7FEB352D)) & low
    h = ((h ^ (h >> np.uint64(15))) * np.uint64(0x846CA68B)) & low
    return h ^ (h >> np.uint64(16))


def random_bits(seed, step, index, n):
    low = np.uint64(0xFFFFFFFF)
    key = mix(np.uint64((seed + int(mix(step & 0xFFFFFFFF))) & 0xFFFFFFFF))
    i = np.arange(n, dtype=np.uint64)
    key = mix((key + np.uint64(index)) & low)
    base = mix((key + i // np.uint64(BLOCK)) & low)
    return mix((base + (i % np.uint64(BLOCK)) * np.uint64(0x9E3779B9)) & low)


def decode(codes, scales):
    """e4m3 codes and scale bytes -> fp64 values."""
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8.0 + m) * 2.0 ** (e - 10.0))
    v = np.where(c & 127 == 127, np.nan, v)
    s = np.repeat(2.0 ** (scales.astype(np.float64) - 127), BLOCK)[: len(c)]
    s = np.where(np.repeat(scales == 0, BLOCK)[: len(c)], 0.0, s)
    return np.where(c & 128, -v, v) * s


def encode(x, cut, root):
    """fp32 values -> codes, scale bytes; cut: 16 random bits an element."""
    n = len(x)
    pad = -n % BLOCK
    a = np.abs(x.astype(np.float64))
    fin = np.where(np.isfinite(a), a, 0.0)
    top = np.pad(fin, (0, pad)).reshape(-1, BLOCK).max(1)
    e = np.zeros(len(top))
    for i, t in enumerate(top):
        if t > 0:
            k = math.frexp(t)[1] - 10
            while t > 448.0 * 2.0 ** k:
                k += 1
            e[i] = max(k, -126)
    sc = np.repeat(2.0 ** -e, BLOCK)[:n]
    y = (fin.astype(F) * sc.astype(F)).astype(F).astype(np.float64)
    small = y < 2.0 ** -6
    # (below 2^-6 the sum with 2^-6 is rounded to fp32 first)
    y = np.where(small, (y.astype(F) + F(2.0 ** -6)).astype(np.float64) - 2.0 ** -6, y)
    ex = np.where(small, -6, np.frexp(np.where(small, 1.0, y))[1] - 1)
    unit = 2.0 ** (ex - 3.0)
    low = np.floor(y / unit)
    k = low + (y / unit - low + cut / 65536.0 >= 1.0)
    v = k * unit
    # the code of a value of the format
    ev = np.maximum(np.frexp(np.where(v > 0, v, 1.0))[1] - 1, -6)
    ev = np.where(v < 2.0 ** -6, -6, ev)
    man = v / 2.0 ** (ev - 3.0)
    code = np.where(v < 2.0 ** -6, man, (ev + 7) * 8 + man - 8).astype(np.int64)
    if root:
        code = np.where((x > 0) & (code < 1), 1, code)
    code = np.where(np.isfinite(a), code, 127) + np.where(np.signbit(x), 128, 0)
    return code.astype(np.uint8), (e + 127).astype(np.uint8)


def factor(sumsq, max_norm):
    with np.errstate(over="ignore"):
        return F(min(1.0, float(F(max_norm)) / (math.sqrt(sumsq) + 1e-6)))       # (max_norm is a float)


def states(g, m, v, clip, b1, b2):
    """fp32 arrays -> m', v', sqrt(v'), each operation rounded once."""
    with np.errstate(all="ignore"):
        if clip is not None:
            g = (g * clip).astype(F)
        m = (m * F(b1) + g * F(1 - b1)).astype(F)
        v = (v * F(b2) + (g * g).astype(F) * F(1 - b2)).astype(F)
        return m, v, np.sqrt(v).astype(F)


def params(p, m, r, step, lr, b1, b2, eps, decay):
    """fp64 parameters and the size of the update."""
    with np.errstate(all="ignore"):
        u = lr / (1 - b1 ** step) * m.astype(np.float64) / (r.astype(np.float64) / math.sqrt(1 - b2 ** step) + eps)
        return p.astype(np.float64) * (1 - lr * decay) - u, np.abs(u)
