"""Float64 NumPy oracle of the expert operators (gather, combine, gate, block
quantisation, products, weight gradients).

Written from the definitions in include/muon_experts.h; it shares no code with
the library, its binding or the benchmark cases.
"""
from __future__ import annotations

import numpy as np

FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
DIGITS = {"e4m3": (3, -6), "e5m2": (2, -14)}     # fraction bits, exponent of the smallest normal value


def runs(offsets, rows):
    """[lo, hi) of each expert, offsets taken into [0, rows], backward runs empty."""
    o = [min(max(int(v), 0), rows) for v in offsets]
    return [(lo, max(lo, hi)) for lo, hi in zip(o, o[1:])]


def gather(order, x, top_k):
    """{place: row} of the places that a pair owns."""
    n = x.shape[0] * top_k
    return {i: x[p // top_k] for i, p in enumerate(order) if 0 <= p < n}


def combine(position, y, weights=None, base=None):
    """(out, sum of the terms' magnitudes)."""
    rows, k = position.shape
    out = np.zeros((rows, y.shape[1])) if base is None else base.astype(np.float64).copy()
    size = np.abs(out)
    for t in range(rows):
        for j in range(k):
            i = position[t, j]
            if 0 <= i < y.shape[0]:
                term = y[i] * (1.0 if weights is None else weights[t, j])
                out[t] += term
                size[t] += np.abs(term)
    return out, size


def combine_backward(position, dout, y, weights=None):
    """({place: dy}, dweights, the dot products' sums of magnitudes)."""
    rows, k = position.shape
    dy, dw, size = {}, np.zeros((rows, k)), np.zeros((rows, k))
    for t in range(rows):
        for j in range(k):
            i = int(position[t, j])
            if 0 <= i < y.shape[0]:
                dy[i] = dout[t] * (1.0 if weights is None else weights[t, j])
                dw[t, j] = np.dot(dout[t], y[i])
                size[t, j] = np.dot(np.abs(dout[t]), np.abs(y[i]))
    return dy, dw, size


def sigmoid(g):
    t = np.exp(-np.abs(g))
    return np.where(g >= 0, 1 / (1 + t), t / (1 + t))


def gate(a):
    f = a.shape[1] // 2
    return a[:, :f] * sigmoid(a[:, :f]) * a[:, f:]


def gate_backward(a, dy):
    """(da, magnitude of the terms that its sums are made of)."""
    f = a.shape[1] // 2
    g, u = a[:, :f], a[:, f:]
    s, rest = sigmoid(g), sigmoid(-g)
    return (np.concatenate([dy * u * s * (1 + g * rest), dy * g * s], 1),
            np.concatenate([np.abs(dy * u * s) * (1 + np.abs(g) * rest), np.abs(dy * g * s)], 1))


def largest(v):
    """Largest magnitude, NaN left out."""
    m = np.abs(v[~np.isnan(v)])
    return m.max() if m.size else 0.0


def scale_of(v, fmt):
    m = largest(v)
    return 1.0 if m == 0 else max(float(np.float32(m) / np.float32(FMAX[fmt])), 2.0 ** -126)


def row_scales(v, fmt):
    """[rows, ceil(cols / 128)]"""
    return np.array([[scale_of(r[c:c + 128], fmt) for c in range(0, v.shape[1], 128)] for r in v]).reshape(v.shape[0],
                                                                                                      -(-v.shape[1] // 128))


def block_scales(v, fmt):
    """[ceil(rows / 128), ceil(cols / 128)]"""
    return np.array([[scale_of(v[r:r + 128, c:c + 128], fmt) for c in range(0, v.shape[1], 128)]
                     for r in range(0, v.shape[0], 128)])


def round8(v, fmt):
    """Nearest values of the 8-bit format, ties to even, the largest magnitude at most FMAX."""
    digits, low = DIGITS[fmt]
    with np.errstate(invalid="ignore"):
        step = np.exp2(np.maximum(np.frexp(np.where(np.isfinite(v), v, 1.0))[1] - 1, low) - digits)
        return np.clip(np.round(v / step) * step, -FMAX[fmt], FMAX[fmt])


def expand(scales, rows, cols, block_rows=1):
    """Scales for each element."""
    return np.repeat(np.repeat(scales, block_rows, 0)[:rows], 128, 1)[:, :cols]


def lifted(v, fmt):
    """Magnitudes, those of subnormal values the smallest normal one."""
    return np.where(v == 0, 0.0, np.maximum(np.abs(v), 2.0 ** DIGITS[fmt][1]))


def product(a, a_scales, w, w_scales, offsets, formats=("e4m3", "e4m3")):
    """(out, sums of magnitudes of the products with subnormal factors lifted); rows outside every run are NaN."""
    rows, k = a.shape
    out = np.full((rows, w.shape[1]), np.nan)
    size = np.zeros_like(out)
    sa = expand(a_scales, rows, k)
    for e, (lo, hi) in enumerate(runs(offsets, rows)):
        sw = expand(w_scales[e], w.shape[1], k, 128)
        out[lo:hi] = (a * sa)[lo:hi] @ (w[e] * sw).T
        size[lo:hi] = (lifted(a, formats[0]) * sa)[lo:hi] @ (lifted(w[e], formats[1]) * sw).T
    return out, size


def weight_grad(dy, x, offsets, experts):
    dw = np.zeros((experts, dy.shape[1], x.shape[1]))
    size = np.zeros_like(dw)
    for e, (lo, hi) in enumerate(runs(offsets, dy.shape[0])):
        dw[e] = dy[lo:hi].T @ x[lo:hi]
        size[e] = np.abs(dy[lo:hi]).T @ np.abs(x[lo:hi])
    return dw, size
