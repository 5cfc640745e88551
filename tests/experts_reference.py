"""Definitions in 64 bits of the operators around experts (numpy, host), and
bounds of what 32-bit arithmetic may add."""
import numpy as np
import torch

U = 2.0 ** -24            # half a step of binary32, relative
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}


def host(x):
    return x.detach().cpu().double().numpy()


def step(dtype):
    """Half a step of a rounding to dtype, relative."""
    return float(torch.finfo(dtype).eps) / 2


def scores_of(x, kind):
    with np.errstate(all="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-x))
        top = x.max(-1, keepdims=True)
        e = np.where(np.isneginf(x), 0.0, np.exp(x - top))
        return e / e.sum(-1, keepdims=True)


def topk(x, k, scores="softmax", bias=None, groups=1, top_groups=1, group_score="best two", renormalize=True, scale=1.0,
         mask=None):
    """(weights, ids, r, s): r the weights before the scale, s the scores."""
    x = np.asarray(x, np.float64)
    t, e = x.shape
    s = scores_of(x, scores)
    by_logit = bias is None and (groups == 1 or group_score == "best")
    c = x if by_logit else s + (0 if bias is None else np.asarray(bias, np.float64))
    ids = np.full((t, k), -1, np.int64)
    r = np.zeros((t, k))
    for i in range(t):
        if mask is not None and not mask[i]:
            continue
        live = ~np.isneginf(x[i])
        key = np.where(np.isnan(c[i]), np.inf, c[i])   # tests hold no +inf beside a NaN
        size = e // groups
        if groups > 1:
            value = np.full(groups, -np.inf)
            for g in range(groups):
                part = np.sort(key[g * size:(g + 1) * size][live[g * size:(g + 1) * size]])[::-1]
                if len(part):
                    value[g] = part[:2 if group_score == "best two" else 1].sum()
            stays = np.argsort(-value, kind="stable")[:top_groups]
            live &= np.isin(np.arange(e) // size, stays)
        at = np.nonzero(live)[0]
        at = at[np.argsort(-key[at], kind="stable")][:k]
        ids[i, :len(at)] = at
        with np.errstate(all="ignore"):
            if not renormalize:
                r[i, :len(at)] = s[i, at]
            elif scores == "softmax":
                v = np.exp(x[i, at] - x[i, at].max()) if len(at) else np.zeros(0)
                r[i, :len(at)] = v / v.sum()
            else:   # logarithms of the scores: a common factor leaves
                v = -np.logaddexp(0.0, -x[i, at])
                v = np.exp(v - v.max()) if len(at) else np.zeros(0)
                r[i, :len(at)] = v / v.sum()
            if scores == "softmax" and (np.isnan(x[i]) | np.isposinf(x[i])).any():
                r[i, :len(at)] = np.nan
    return r * scale, ids, r, s


def topk_backward(x, ids, g, scores, renormalize, scale):
    """The formulas of the header, in 64 bits; and the magnitudes that its sums
    and differences pass through."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    s = scores_of(x, scores)
    has = ids >= 0
    at = np.where(has, ids, 0)
    g = np.where(has, g, 0)
    sc = np.where(has, np.take_along_axis(s, at, 1), 0)
    dx, size = np.zeros_like(x), np.zeros_like(x)
    # 1 - s as the logistic function of -x: the difference itself loses all its digits next to s = 1
    rest = scores_of(-np.take_along_axis(x, at, 1), "sigmoid") if scores == "sigmoid" else np.ones_like(sc)
    if renormalize:
        lx = np.where(has, np.take_along_axis(x, at, 1), -np.inf)
        if scores == "sigmoid":
            lx = np.where(has, -np.logaddexp(0.0, -lx), -np.inf)
        with np.errstate(all="ignore"):
            r = np.where(has, np.exp(lx - lx.max(-1, keepdims=True)), 0)
            r = np.where(has, r / r.sum(-1, keepdims=True), 0)
        d = scale * r * rest * (g - (g * r).sum(-1, keepdims=True))
        m = abs(scale) * r * rest * (abs(g) + (abs(g) * r).sum(-1, keepdims=True))
    elif scores == "sigmoid":
        d = scale * sc * rest * g
        m = abs(d)
    else:
        dense = np.zeros_like(x)
        for i, j in zip(*np.nonzero(has)):
            dense[i, ids[i, j]] = g[i, j]
        total, most = (g * sc).sum(-1, keepdims=True), (abs(g) * sc).sum(-1, keepdims=True)
        alive = has.any(-1, keepdims=True)
        return np.where(alive, scale * s * (dense - total), 0), np.where(alive, abs(scale) * s * (abs(dense) + most), 0)
    for i, j in zip(*np.nonzero(has)):
        dx[i, ids[i, j]] = d[i, j]
        size[i, ids[i, j]] = m[i, j]
    return dx, size


def weights_bound(x, ids):
    """Relative bound of a weight: an exponential's argument is off by half a
    step of itself (its own difference, at most the row's spread), the
    exponential by two steps, sums of up to 16 + 6 positive terms in a row by
    as many half steps on either side of the division, sums with 1 and three
    products or quotients by half a step each."""
    finite = np.where(np.isfinite(x), x, 0.0)
    spread = np.minimum(finite.max(-1, keepdims=True) - finite.min(-1, keepdims=True), 200.0)
    return (2 * spread + 2 * 4 + 2 * 22 + 6) * U


def order(ids, experts):
    flat = np.asarray(ids).reshape(-1)
    key = np.where((flat < 0) | (flat >= experts), experts, flat)
    by = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[by], np.arange(experts + 1)).astype(np.int32)
    n = offsets[-1]
    slots = np.where(np.arange(len(flat)) < n, by, -1).astype(np.int32)
    places = np.full(len(flat), -1, np.int32)
    places[by[:n]] = np.arange(n)
    return offsets, slots, places.reshape(np.asarray(ids).shape)


def int4_values(codes, scales, zeros, group):
    """Values in 64 bits of codes [..., K / 2] (numpy), and the codes."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).astype(np.float64)
    z = 8.0 if zeros is None else np.repeat(host(zeros), group, -1)
    return (c - z) * np.repeat(host(scales), group, -1), c


def int4_product(x, q):
    """(x q^T, the magnitude that its sums pass through) for x [M, K] and an
    Int4 [N, K]: codes are taken apart into code - 8 and zero - 8."""
    values, c = int4_values(q.codes.cpu().numpy(), q.scales, q.zeros, q.group)
    z = 0.0 if q.zeros is None else np.abs(np.repeat(host(q.zeros), q.group, -1) - 8)
    size = (np.abs(c - 8) + z) * np.abs(np.repeat(host(q.scales), q.group, -1))
    return x @ values.T, np.abs(x) @ size.T
