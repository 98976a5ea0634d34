"""Routing and its gradient in float64 for many rows at once (NumPy), for sizes
that the oracle's loops are too slow for. Finite logits or -inf."""

import numpy as np


def probabilities(x):
    top = x.max(1, keepdims=True)
    e = np.exp(x - np.where(top > -np.inf, top, 0.0))
    s = e.sum(1, keepdims=True)
    return e / np.where(s > 0, s, 1.0)


def route(x, k, mask=None, renormalise=False, coef=1.0, align=128, max_m=0):
    x = np.asarray(x, np.float64)
    T, E = x.shape
    on = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]           # ties to the lower expert
    value = np.take_along_axis(x, order, 1)
    ids = np.where((value > -np.inf) & on[:, None], order, -1).astype(np.int32)
    live = ids >= 0
    p = probabilities(x) * on[:, None]
    w = np.where(live, np.take_along_axis(p, order, 1), 0.0)
    if renormalise:
        s = w.sum(1, keepdims=True)
        w = w / np.where(s > 0, s, 1.0)
    counts = np.bincount(ids[live], minlength=E)
    routed, psum = int(live[:, 0].sum()), p.sum(0)
    n = max(routed, 1)
    loss = coef * float((E * counts / (k * n) * (psum / n)).sum())
    offsets = np.arange(E + 1) * max_m if max_m else np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    # a pair's rank: its place among the pairs of its expert, in their order
    flat = ids.reshape(-1)
    at = np.flatnonzero(flat >= 0)
    by = at[np.argsort(flat[at], kind="stable")]
    rank = np.zeros(flat.size, np.int64)
    rank[by] = np.arange(by.size) - np.repeat(np.cumsum(counts) - counts, counts)
    fits = (flat >= 0) & ((rank < max_m) if max_m else True)
    slots = np.where(fits, offsets[np.maximum(flat, 0)] + rank, -1).reshape(T, k)
    return dict(expert_ids=ids, weights=w, counts=counts.astype(np.int32), routed=routed, prob_sum=psum, loss=loss,
                group_offsets=offsets.astype(np.int32), slots=slots.astype(np.int32))


def route_backward(x, ids, d_weights, d_loss, counts, routed, renormalise=False, coef=1.0):
    """-> (d_logits, the sum of the magnitudes that each element is a sum of)"""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    k, n = ids.shape[1], max(int(routed), 1)
    p = probabilities(x)
    live, at = ids >= 0, np.maximum(ids, 0)
    dw = np.where(live, np.asarray(d_weights, np.float64), 0.0)
    mag = np.abs(dw)
    if renormalise:
        pc = np.where(live, np.take_along_axis(p, at, 1), 0.0)
        s = pc.sum(1, keepdims=True)
        s = np.where(s > 0, s, 1.0)
        mag = np.where(live, (mag + (mag * pc).sum(1, keepdims=True) / s) / s, 0.0)
        dw = np.where(live, (dw - (dw * pc).sum(1, keepdims=True) / s) / s, 0.0)
    f = d_loss * coef * E * np.asarray(counts, np.float64) / (k * n * n)
    dp, size = np.tile(f, (T, 1)), np.tile(np.abs(f), (T, 1))
    rows = np.broadcast_to(np.arange(T)[:, None], ids.shape)
    np.add.at(dp, (rows[live], ids[live]), dw[live])
    np.add.at(size, (rows[live], ids[live]), mag[live])
    on = live[:, :1]
    dx = p * (dp - (p * dp).sum(1, keepdims=True))
    size = p * (size + (p * size).sum(1, keepdims=True))
    return np.where(on, dx, 0.0), np.where(on, size, 0.0)
