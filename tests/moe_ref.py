"""64-bit references of the MoE routing operators and of gradient clipping
(CPU, NumPy only), with the magnitudes their error bounds are scaled by."""

import numpy as np

U32 = 2.0 ** -24  # half a step of FP32, relative


def half_step(bf16):
    return 2.0 ** -8 if bf16 else U32


def scores(x, sigmoid):
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-x))
        top = x.max(1, keepdims=True)
        e = np.exp(x - np.where(np.isneginf(top), 0.0, top))
        s = e.sum(1, keepdims=True)
        return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def route(x, k, sigmoid, bias=None, renorm=True, scale=1.0):
    """(ids, weights) of logits x [T, E] in float64."""
    p = scores(x, sigmoid)
    key = x if bias is None else np.where(np.isneginf(x), -np.inf, p + bias)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    gone = np.isneginf(np.take_along_axis(key, ids, 1))
    return np.where(gone, -1, ids).astype(np.int32), weights_of(x, np.where(gone, -1, ids), sigmoid, renorm, scale)


def chosen_ratio(x, ids, sigmoid):
    """Chosen scores over their sum, formed from score / e^c with c the largest
    chosen logit (for sigmoids at most 0), so that small scores keep their ratio."""
    on = ids >= 0
    xj = np.where(on, np.take_along_axis(x, np.maximum(ids, 0), 1), -np.inf)
    c = xj.max(1, keepdims=True)
    c = np.where(np.isneginf(c), 0.0, np.minimum(c, 0.0) if sigmoid else c)
    with np.errstate(over="ignore"):
        w = np.where(xj < 0, np.exp(np.minimum(xj - c, 0.0)) / (1 + np.exp(np.minimum(xj, 0.0))),
                     1 / (1 + np.exp(-np.maximum(xj, 0.0)))) if sigmoid else np.exp(xj - c)
    s = w.sum(1, keepdims=True)
    return np.divide(w, s, out=np.zeros_like(w), where=s > 0)


def weights_of(x, ids, sigmoid, renorm, scale):
    """The weights of given choices (differentiable in x for fixed ids)."""
    if renorm:
        return chosen_ratio(x, ids, sigmoid) * scale
    return np.take_along_axis(scores(x, sigmoid), np.maximum(ids, 0), 1) * (ids >= 0) * scale


def route_bwd(dw, x, ids, sigmoid, renorm, scale):
    """(dlogits, sum of the magnitudes of the terms of each entry)."""
    p = scores(x, sigmoid)
    on = ids >= 0
    at = np.maximum(ids, 0)
    g = dw * scale * on
    pj = np.take_along_axis(p, at, 1) * on
    if renorm:
        w = chosen_ratio(x, ids, sigmoid)
        core, mag = w * (g - (g * w).sum(1, keepdims=True)), w * (abs(g) + (abs(g) * w).sum(1, keepdims=True))
        if sigmoid:
            xj = np.take_along_axis(x, at, 1)
            with np.errstate(over="ignore"):  # 1 - sigmoid
                rest = 1.0 / (1.0 + np.exp(xj))
            core, mag = core * rest, mag * rest
    elif sigmoid:
        core = g * pj * scores(-np.take_along_axis(x, at, 1), True)  # 1 - p without cancellation
        mag = abs(core)
    else:
        gd = np.zeros_like(p)
        np.put_along_axis(gd, at, 0.0, 1)
        for t, j in zip(*np.nonzero(on)):
            gd[t, at[t, j]] = g[t, j]
        return p * (gd - (pj * g).sum(1, keepdims=True)), p * (abs(gd) + (pj * abs(g)).sum(1, keepdims=True))
    d, m = np.zeros_like(p), np.zeros_like(p)
    for t, j in zip(*np.nonzero(on)):
        d[t, at[t, j]], m[t, at[t, j]] = core[t, j], mag[t, j]
    return d, m


def sort(ids, experts, cover=False):
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    src = np.argsort(key, kind="stable")
    row = np.empty_like(src)
    row[src] = np.arange(src.size)
    off = np.searchsorted(key[src], np.arange(experts + 1))
    if cover:
        off[experts] = flat.size
    return off.astype(np.int32), np.where(key < experts, row, -1 - row).astype(np.int32).reshape(ids.shape), \
        src.astype(np.int32)


def spread(v, dst):
    """v [T, k, H] or [T, 1, H] to its rows; zeros for dropped pairs."""
    t, k = dst.shape
    out = np.zeros((t * k, v.shape[2]), v.dtype)
    for j in range(k):
        on = dst[:, j] >= 0
        out[dst[on, j]] = v[on, j if v.shape[1] > 1 else 0]
    return out


def fetch(rows, dst):
    """rows[dst] in float64, zeros for dropped pairs: [T, k, H]."""
    return np.where((dst >= 0)[:, :, None], rows.astype(np.float64)[np.maximum(dst, 0)], 0.0)
