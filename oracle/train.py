"""Oracle of a mixture-of-experts layer's training step, in float64.

Routing (softmax, the k largest logits, balance loss, row of every pair) and
its gradient, the weight gradient in 8-bit floating point with power-of-two
scales along the tokens, and gradient clipping. Plain definitions with loops
where a loop says it best; nothing here is shared with the HIP sources.
"""

import numpy as np

from .formats import FORMATS


def softmax(x):
    """Row softmax in float64; a row of -inf alone has no probability, a row
    that holds NaN or +inf has NaN."""
    x = np.asarray(x, np.float64)
    p = np.zeros_like(x)
    for t in range(x.shape[0]):
        if np.isnan(x[t]).any() or (x[t] == np.inf).any():
            p[t] = np.nan
        elif (x[t] > -np.inf).any():
            e = np.exp(x[t] - x[t].max())
            p[t] = e / e.sum()
    return p


def route(x, k, mask=None, renormalise=False, coef=1.0, align=128, max_m=0):
    """x [T][E] -> dict of expert_ids, weights, counts, routed, prob_sum, loss,
    group_offsets, slots (see the C header for the definitions)."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    mask = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    p = softmax(x)
    p[~mask] = 0.0
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        if not mask[t]:
            continue
        may = [e for e in range(E) if x[t, e] > -np.inf]        # (neither -inf nor NaN)
        best = sorted(may, key=lambda e: (-x[t, e], e))[:k]
        ids[t, :len(best)] = best
        if np.isnan(p[t]).any():
            w[t] = np.nan
        elif best:
            w[t, :len(best)] = p[t, best]
            if renormalise:
                w[t] /= w[t].sum()
    counts = np.bincount(ids[ids >= 0], minlength=E).astype(np.int32)
    routed = int((ids[:, 0] >= 0).sum()) if T else 0
    psum = p.sum(0)
    n = max(routed, 1)
    loss = coef * float((E * counts / (k * n) * (psum / n)).sum())
    if max_m:
        offsets = np.arange(E + 1, dtype=np.int64) * max_m
    else:
        offsets = np.concatenate([[0], np.cumsum(-(-counts.astype(np.int64) // align) * align)])
    slots = np.full((T, k), -1, np.int32)
    seen = np.zeros(E, np.int64)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e >= 0:
                if not max_m or seen[e] < max_m:
                    slots[t, j] = offsets[e] + seen[e]
                seen[e] += 1
    return dict(expert_ids=ids, weights=w, counts=counts, routed=routed, prob_sum=psum, loss=loss,
                group_offsets=offsets.astype(np.int32), slots=slots)


def route_backward(x, ids, d_weights, d_loss, counts, routed, renormalise=False, coef=1.0):
    """-> (d_logits, size): the gradient in float64, and for each element the
    sum of the magnitudes that it is a sum of (what rounding errors go by)."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    k = ids.shape[1]
    p = softmax(x)
    dx, size = np.zeros((T, E)), np.zeros((T, E))
    n = max(int(routed), 1)
    f = d_loss * coef * E * np.asarray(counts, np.float64) / (k * n * n)
    for t in range(T):
        if ids[t, 0] < 0:
            continue
        dp, mag = f.copy(), np.abs(f)
        live = [j for j in range(k) if ids[t, j] >= 0]
        pc = p[t, ids[t, live]]
        dw = np.asarray(d_weights[t], np.float64)[live]
        m = np.abs(dw)
        if renormalise:
            s = pc.sum()
            m = (m + (m * pc).sum() / s) / s
            dw = (dw - (dw * pc).sum() / s) / s
        for i, j in enumerate(live):
            dp[ids[t, j]] += dw[i]
            mag[ids[t, j]] += m[i]
        dx[t] = p[t] * (dp - (p[t] * dp).sum())
        size[t] = p[t] * (mag + (p[t] * mag).sum())
    return dx, size


def quantize_transpose(x, fmt):
    """x [rows][cols] float32 -> (codes [cols][R], exponent bytes [R/128][cols]),
    R = rows rounded up to 128: one power-of-two scale for each column and 128
    rows, the smallest that brings the finite elements to FP8max or below."""
    top, _, encode = FORMATS[fmt]
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    R = -(-rows // 128) * 128
    q = np.zeros((cols, R), np.uint8)
    s = np.zeros((R // 128, cols), np.uint8)
    for i in range(R // 128):
        blk = x[i * 128:(i + 1) * 128].astype(np.float64)
        amax = np.where(np.isfinite(blk), np.abs(blk), 0.0).max(0)
        mant, e = np.frexp(np.where(amax > 0, amax, 1.0) / top)  # amax / top = mant 2^e, mant in [0.5, 1)
        e = np.where(mant == 0.5, e - 1, e)
        e = np.where(amax > 0, np.clip(e, -126, 126), 0)
        with np.errstate(invalid="ignore"):
            y = np.ldexp(blk, -e).astype(np.float32)              # exact, or below every code
        q[:, i * 128:i * 128 + blk.shape[0]] = encode(y).T
        s[i] = e + 127
    return q, s


def wgrad(qa, fa, sa, qb, fb, sb, offsets):
    """-> (d [G][M][N] float64, size): size is the sum of the products'
    magnitudes."""
    ta, tb = FORMATS[fa][1], FORMATS[fb][1]
    G = len(offsets) - 1
    a = ta[qa] * np.repeat(np.ldexp(1.0, sa.astype(int).T - 127), 128, axis=1)
    b = tb[qb] * np.repeat(np.ldexp(1.0, sb.astype(int).T - 127), 128, axis=1)
    d = np.zeros((G, a.shape[0], b.shape[0]))
    size = np.zeros_like(d)
    for g in range(G):
        lo, hi = int(offsets[g]), int(offsets[g + 1])
        if hi > lo:
            d[g] = a[:, lo:hi] @ b[:, lo:hi].T
            size[g] = np.abs(a[:, lo:hi]) @ np.abs(b[:, lo:hi]).T
    return d, size


def grad_clip(grads, max_norm):
    """-> (sum of squares, norm, clipped gradients), all in float64."""
    total = float(sum((np.asarray(g, np.float64) ** 2).sum() for g in grads))
    norm = np.sqrt(total)
    coef = min(1.0, max_norm / (norm + 1e-6)) if not np.isnan(norm) else np.nan
    return total, norm, [np.asarray(g, np.float64) * coef for g in grads]
