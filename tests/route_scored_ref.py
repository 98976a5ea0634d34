"""Routing by scores in NumPy, in 64 bits, row by row from the definition."""

import numpy as np


def scores(x, score):
    """[T][E] fp64 logits -> fp64 scores."""
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        top = np.max(x, 1, keepdims=True)
        p = np.exp(x - np.where(top > -np.inf, top, 0.0))
        z = p.sum(1, keepdims=True)
        return np.where(z == 0, 0.0, p / np.where(z == 0, 1.0, z))


def select(x, s, bias, groups, opened, best, k, on):
    """The chosen experts of each row, -1 past the last."""
    T, E = x.shape
    size = E // groups
    ids = np.full((T, k), -1, np.int32)
    for t in range(T):
        if not on[t]:
            continue
        v = s[t] + (0.0 if bias is None else bias.astype(np.float64))
        may = (x[t] > -np.inf) & (v > -np.inf)         # (NaN: neither)
        by_value = bias is not None or opened < groups
        if not by_value:
            may = x[t] > -np.inf
        if opened < groups:
            value = np.full(groups, -np.inf)
            for g in range(groups):
                inside = np.sort(v[g * size:(g + 1) * size][may[g * size:(g + 1) * size]])[::-1]
                if len(inside):
                    value[g] = inside[:best].sum()
            order = sorted(range(groups), key=lambda g: (-value[g], g))[:opened]
            shut = np.ones(E, bool)
            for g in order:
                if value[g] > -np.inf:
                    shut[g * size:(g + 1) * size] = False
            may = may & ~shut
        by = v if bias is not None else x[t]
        live = np.flatnonzero(may)
        order = live[np.lexsort((live, -by[live]))][:k]
        ids[t, :len(order)] = order
    return ids


def route(x, bias, score, groups, opened, best, k, renorm, scale, coef, align, max_m, mask=None):
    """x fp64 [T][E] -> everything moe_route_scored writes, as a dict."""
    T, E = x.shape
    on = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    s = scores(x, score)
    ids = select(x, s, bias, groups, opened, best, k, on)
    live = ids >= 0
    poison = on & (np.isnan(x).any(1) | ((score == "softmax") & (x == np.inf).any(1)))
    w = np.where(live, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    with np.errstate(all="ignore"):
        if renorm:
            z = w.sum(1, keepdims=True)
            w = np.where(z > 0, w / np.where(z > 0, z, 1.0), 0.0)
        w = np.where(poison[:, None], np.nan, w * scale)
        z = s.sum(1, keepdims=True)
        share = np.where(z == 0, 0.0, s / np.where(z == 0, 1.0, z))
    routed = live[:, 0]
    n = int(routed.sum())
    psum = share[routed & ~poison].sum(0)
    if poison.any():
        psum = psum * np.nan
    counts = np.bincount(ids[live], minlength=E)[:E]
    loss = coef * (E * counts / (k * max(n, 1)) * (psum / max(n, 1))).sum()
    off = np.arange(E + 1) * max_m if max_m else np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    seen = np.zeros(E, np.int64)
    slots = np.full((T, k), -1, np.int64)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e >= 0:
                if not max_m or seen[e] < max_m:
                    slots[t, j] = off[e] + seen[e]
                seen[e] += 1
    return dict(expert_ids=ids, weights=w, counts=counts, routed=n, prob_sum=psum, loss=loss, group_offsets=off,
                slots=slots)


def backward(x, ids, dw, dloss, counts, n, score, renorm, scale, coef):
    """The formula in 64 bits -> gradient [T][E] and, for each element, the sum of the
    magnitudes of what it is made of."""
    T, E = x.shape
    k = ids.shape[1]
    s = scores(x, score)
    f = np.broadcast_to(dloss * coef * E * counts / (k * max(n, 1) ** 2), (T, E)).astype(np.float64)
    live = ids >= 0
    at = np.maximum(ids, 0)
    p = np.where(live, np.take_along_axis(s, at, 1), 0.0)
    d = np.where(live, dw * scale, 0.0)
    size = np.abs(d)
    with np.errstate(all="ignore"):
        if renorm:
            z = p.sum(1, keepdims=True)
            u = np.where(z > 0, p / np.where(z > 0, z, 1.0), 0.0)
            size = np.where(live & (z > 0), (np.abs(d) + (np.abs(d) * u).sum(1, keepdims=True)) / z, 0.0)
            d = np.where(live & (z > 0), (d - (d * u).sum(1, keepdims=True)) / z, 0.0)
        chosen, big = np.zeros((T, E)), np.zeros((T, E))
        for j in range(k):
            np.add.at(chosen, (np.arange(T), at[:, j]), np.where(live[:, j], d[:, j], 0.0))
            np.add.at(big, (np.arange(T), at[:, j]), np.where(live[:, j], size[:, j], 0.0))
        if score == "softmax":
            g = f + chosen
            dx = s * (g - (s * g).sum(1, keepdims=True))
            size = s * (np.abs(f) + big + (s * (np.abs(f) + big)).sum(1, keepdims=True))
        else:
            z = s.sum(1, keepdims=True)
            z = np.where(z > 0, z, 1.0)
            dot = (f * s).sum(1, keepdims=True) / z
            t = np.exp(-np.abs(x))
            slope = t / (1 + t) ** 2
            dx = slope * ((f - dot) / z + chosen)
            size = slope * ((np.abs(f) + np.abs(f * s).sum(1, keepdims=True) / z) / z + big)
    on = live[:, :1]
    return np.where(on, dx, 0.0), np.where(on, size, 0.0)
