"""Plain float64 (numpy) forms of routing, its gradient, combine's gradient and
the INT8 product, written from the definitions in ``include/moe_ep.h``; shared
by the tests of those operators.  They share nothing with the CUDA code."""
import numpy as np

NEG = -np.inf


def scores(l, score):
    """Scores of float64 logits [T, E]; NaN counts as -inf, +inf as the largest
    float."""
    l = np.minimum(np.where(np.isnan(l), NEG, l), np.finfo(np.float32).max)
    if score == "sigmoid":
        e = np.exp(-np.abs(l))
        return np.where(l >= 0, 1 / (1 + e), e / (1 + e))
    top = l.max(axis=1, keepdims=True)
    e = np.exp(l - np.where(np.isfinite(top), top, 0.0))
    total = e.sum(axis=1, keepdims=True)
    return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def route_keys(l, bias, score, n_group, group_top):
    """(ranking key [T, E], group score [T, n_group], scores): -inf where
    nothing is available."""
    l = np.asarray(l, np.float64)
    s = scores(l, score)
    l = np.minimum(np.where(np.isnan(l), NEG, l), np.finfo(np.float32).max)
    c = s if bias is None else s + np.asarray(bias, np.float64)
    on = (l > NEG) & (c > NEG)                      # a NaN choice is not > -inf
    key = np.where(on, l if bias is None else c, NEG)
    per = np.where(on, c, NEG).reshape(l.shape[0], n_group, -1)
    best = -np.sort(-per, axis=2)[:, :, :group_top]
    total = np.where(best > NEG, best, 0.0).sum(axis=2)
    return key, np.where(best[:, :, 0] > NEG, total, NEG), s


def route(l, bias, score, k, n_group=1, topk_group=1, group_top=1, renormalise=True,
          scale=1.0):
    """ids int32 [T, k] and float64 weights [T, k]."""
    key, group, s = route_keys(l, bias, score, n_group, group_top)
    T, E = key.shape
    keep = np.argsort(-group, axis=1, kind="stable")[:, :topk_group]
    use = np.zeros((T, n_group), bool)
    np.put_along_axis(use, keep, True, axis=1)
    key = np.where(np.repeat(use, E // n_group, axis=1), key, NEG)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    there = np.take_along_axis(key, ids, 1) > NEG
    ids = np.where(there, ids, -1).astype(np.int32)
    return ids, weights_of(s, ids, renormalise, scale)


def weights_of(s, ids, renormalise, scale):
    w = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    if renormalise:
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return w * scale


def route_backward(l, ids, d_weights, score, renormalise=True, scale=1.0):
    """float64 d_logits [T, E] by the Jacobian of weights_of(scores(l))."""
    l = np.asarray(l, np.float64)
    s = scores(l, score)
    on = ids >= 0
    at = np.maximum(ids, 0)
    g = np.where(on, np.asarray(d_weights, np.float64) * scale, 0.0)
    p = np.where(on, np.take_along_axis(s, at, 1), 0.0)
    if renormalise:
        total = p.sum(axis=1, keepdims=True)
        ok = total > 0
        w = np.divide(p, total, out=np.zeros_like(p), where=ok)
        ds_s = w * (g - (w * g).sum(axis=1, keepdims=True))     # ds * s
    else:
        ds_s = g * p
    if score == "sigmoid":
        ds_s = ds_s * (1 - p)
    d = np.zeros_like(l)
    np.add.at(d, (np.arange(l.shape[0])[:, None], at), np.where(on, ds_s, 0.0))
    if score == "softmax" and not renormalise:
        d -= s * ds_s.sum(axis=1, keepdims=True)
    return d


def linear_i8(a, w, sizes, col=None, row=None, bias=None):
    """int64 accumulators, or the float32 value before the last rounding with
    one fp32 rounding per step: ((fp32(acc) * col) * row) + bias."""
    off = np.concatenate([[0], np.cumsum(sizes)])
    acc = np.zeros((int(off[-1]), w.shape[1]), np.int64)
    for g in range(len(sizes)):
        # products and sums of codes are exact in float64 (< 2^53)
        acc[off[g]:off[g + 1]] = np.rint(
            a[off[g]:off[g + 1]].astype(np.float64) @ w[g].T.astype(np.float64))
    if col is None:
        return acc
    of = np.repeat(np.arange(len(sizes)), sizes)
    v = acc.astype(np.float32) * col[of] * row[:off[-1], None]
    return v if bias is None else v + bias[of]
