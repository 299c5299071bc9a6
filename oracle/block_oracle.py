"""Float64 NumPy oracle of the row operators (norm, dropout, expert routing).

Written from the definitions in include/muon_block.h; it shares no code with
the library, its binding or the benchmark cases.
"""
from __future__ import annotations

import numpy as np

FMAX = {"e4m3": 448.0, "e5m2": 57344.0}


# ---- dropout ----------------------------------------------------------------
def philox4x32(counter, key, rounds=10):
    """Philox4x32 (Salmon et al., 2011) on arrays of 32-bit words held in uint64."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(key[0]), int(key[1])]
    low, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> sh) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p: float) -> int:
    return int(np.floor(65536.0 * p + 0.5))


def keep_mask(rows, cols, p, seed, offset):
    r = np.arange(rows, dtype=np.uint64)[:, None]
    b = np.arange((cols + 7) // 8, dtype=np.uint64)[None, :]
    r, b = np.broadcast_arrays(r, b)
    w = philox4x32((b, r, np.full(r.shape, offset & 0xFFFFFFFF), np.full(r.shape, (offset >> 32) & 0xFFFFFFFF)),
                   (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    pieces = np.stack([x for v in w for x in (v & np.uint64(0xFFFF), v >> np.uint64(16))], axis=2)
    return pieces.reshape(rows, -1)[:, :cols] >= threshold(p)


def dropout(x, p, seed, offset):
    t = threshold(p)
    up = 65536.0 / (65536 - t) if t < 65536 else 0.0
    with np.errstate(invalid="ignore"):
        return np.where(keep_mask(x.shape[0], x.shape[1], p, seed, offset), x * up, 0.0)


# ---- norm -------------------------------------------------------------------
def norm_forward(x, residual=None, weight=None, eps=1e-6, drop=None):
    """(z, rstd, y); drop = (p, seed, offset)."""
    z = dropout(x, *drop) if drop else x
    z = z if residual is None else z + residual
    rstd = 1.0 / np.sqrt((z * z).mean(axis=1) + eps)
    y = z * rstd[:, None]
    return z, rstd, y if weight is None else y * weight


def scales_of(y, fmt, group):
    """One scale per row and group: max |y| / FMAX, 1 for zeros, NaN not counted."""
    g = group or y.shape[1]
    n = -(-y.shape[1] // g)
    a = np.zeros((y.shape[0], n * g))
    a[:, :y.shape[1]] = np.where(np.isnan(y), 0.0, np.abs(y))
    most = a.reshape(y.shape[0], n, g).max(axis=2)
    return np.where(most == 0, 1.0, np.maximum(most / FMAX[fmt], 2.0 ** -126))


def norm_backward(dy, h, rstd, weight=None, dh=None, drop=None):
    """(dz, dx, dweight)."""
    xh = h * rstd[:, None]
    g = dy if weight is None else dy * weight
    dz = rstd[:, None] * (g - xh * (g * xh).mean(axis=1, keepdims=True))
    if dh is not None:
        dz = dz + dh
    return dz, (dropout(dz, *drop) if drop else dz), (dy * xh).sum(axis=0)


# ---- routing ----------------------------------------------------------------
def log_scores(l, score):
    """log s of one row's logits; -inf for closed experts."""
    shut = np.isneginf(l)
    out = np.full(l.shape, -np.inf)
    v = l[~shut]
    if v.size == 0:
        return out
    if score == "sigmoid":
        out[~shut] = np.minimum(v, 0) - np.log1p(np.exp(-np.abs(v)))
    else:
        d = v - v.max()
        out[~shut] = d - np.log(np.exp(d).sum())
    return out


def route_row(l, top_k, score, bias=None, groups=1, top_groups=1, group_top=2, renormalise=True, scale=1.0):
    """(experts, weights, scores) of one row."""
    E = len(l)
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max)).astype(np.float64)
    ls = log_scores(l, score)
    s = np.exp(ls)
    open_ = ~np.isneginf(l)
    sel = s + bias if bias is not None else s
    rank = np.where(open_, sel if bias is not None else l, -np.inf)
    if groups > 1:
        n = E // groups
        value = []
        for g in range(groups):
            best = sorted((sel[e] for e in range(g * n, (g + 1) * n) if open_[e]), reverse=True)[:group_top]
            value.append(sum(best) if best else -np.inf)
        stay = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
        for e in range(E):
            if e // n not in stay:
                rank[e] = -np.inf
    order = sorted((e for e in range(E) if rank[e] > -np.inf), key=lambda e: (-rank[e], e))[:top_k]
    idx = np.full(top_k, -1, np.int64)
    w = np.zeros(top_k)
    idx[:len(order)] = order
    if order:
        c = ls[order]
        if renormalise:
            c = np.exp(c - c.max())
            w[:len(order)] = scale * c / c.sum()
        else:
            w[:len(order)] = scale * np.exp(c)
    return idx, w, s


def route_forward(logits, token_mask=None, **kw):
    rows = [route_row(l, **kw) for l in logits]
    idx, w, s = (np.array([r[i] for r in rows]) for i in range(3))
    if token_mask is not None:
        idx[token_mask == 0], w[token_mask == 0], s[token_mask == 0] = -1, 0, 0
    return idx, w, s


def route_backward(logits, experts, weights, dweights, score, renormalise, scale, dscores=None):
    """d/dl of sum(weights dweights) + sum(scores dscores) for the choice `experts`, by the chain rule."""
    out = np.zeros(logits.shape)
    for t in range(logits.shape[0]):
        on = experts[t] >= 0
        if not on.any():
            continue
        l = np.where(np.isnan(logits[t]), -np.inf, np.minimum(logits[t], np.finfo(np.float32).max))
        ls = log_scores(l, score)
        s, at = np.exp(ls), experts[t][on]
        w, dw = weights[t][on], dweights[t][on]
        a = w * dw
        if renormalise:
            a = a - w / scale * a.sum()
        da = np.zeros(len(l))          # d / d log s
        np.add.at(da, at, a)
        total = 0.0 if renormalise else a.sum()      # its sum; a sums to 0 where the weights are renormalised
        if dscores is not None:
            ds = np.where(np.isneginf(l), 0, dscores[t]) * s
            da, total = da + ds, total + ds.sum()
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                out[t] = np.where(np.isneginf(l), 0, da / (1 + np.exp(l)))
        else:
            out[t] = np.where(np.isneginf(l), 0, da - s * total)
    return out


# ---- order, balance -----------------------------------------------------------
def route_order(experts, num_experts):
    """(counts, offsets, order, position)."""
    flat = experts.reshape(-1)
    lists = [[] for _ in range(num_experts)]
    for p, e in enumerate(flat):
        if 0 <= e < num_experts:
            lists[e].append(p)
    counts = np.array([len(v) for v in lists])
    offsets = np.concatenate([[0], np.cumsum(counts)])
    order = np.full(len(flat), -1)
    position = np.full(len(flat), -1)
    i = 0
    for v in lists:
        for p in v:
            order[i], position[p] = p, i
            i += 1
    return counts, offsets, order, position.reshape(experts.shape)


def route_balance(counts, bias, rate):
    n, E = int(np.sum(counts)), len(counts)
    return np.array([b + rate * np.sign(n - int(c) * E) for b, c in zip(bias, counts)])
