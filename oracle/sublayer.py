"""The mixture-of-experts sublayer in float64 NumPy: layer norm, routing, the experts' products, combine, and
their gradients, straight from the formulas, one token or expert at a time."""

import numpy as np


def layer_norm(x, w=None, b=None, eps=1e-5):
    """(y, mean, rstd) over the last axis of x [rows, cols]."""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    return y * (1.0 if w is None else w) + (0.0 if b is None else b), mean, rstd


def layer_norm_backward(dy, x, w, mean, rstd):
    """(dx, dw, db), with the mean and rstd given."""
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * (1.0 if w is None else w)
    dx = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) - xh * (g * xh).mean(axis=1, keepdims=True))
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


def scores(logits, score):
    z = np.asarray(logits, np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-z))
        out = np.empty_like(z)
        for t, row in enumerate(z):
            if np.all(row == -np.inf):
                out[t] = 0.0
            else:
                e = np.exp(row - (np.nan if np.isnan(row).any() else row.max()))
                out[t] = e / e.sum()
        return out


def route(logits, top_k, bias=None, groups=1, top_groups=1, group_best=2, score="softmax", renormalize=True,
          scale=1.0):
    """(ids, weights, offsets, rows, slots)."""
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    s = scores(z, score)
    keys = z.copy() if bias is None else np.where(z == -np.inf, -np.inf, s + np.asarray(bias, np.float64))
    ranks = s if bias is None else keys
    keys = np.where(np.isnan(keys), -np.inf, keys)
    ids = np.zeros((T, top_k), np.int64)
    for t in range(T):
        allowed = np.arange(E)
        if groups > 1:
            n = E // groups
            r = np.where(np.isnan(ranks[t]), -np.inf, ranks[t]).reshape(groups, n)
            best = np.sort(r, axis=1)[:, ::-1][:, :group_best]
            none = best[:, 0] == -np.inf  # keys of -inf add nothing, and a group of nothing else comes last
            best = np.where(none, -np.inf, np.where(best == -np.inf, 0.0, best).sum(axis=1))
            kept = sorted(range(groups), key=lambda i: (-best[i], i))[:top_groups]
            allowed = np.array([e for e in range(E) if e // n in kept])
        ids[t] = sorted(allowed, key=lambda e: (-keys[t, e], e))[:top_k]
    w = np.take_along_axis(s, ids, 1)
    if renormalize:
        w = w / (w.sum(axis=1, keepdims=True) + 1e-20)
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    slots = np.empty_like(order)
    slots[order] = np.arange(T * top_k)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    return ids, w * scale, offsets, order // top_k, slots.reshape(T, top_k)


def route_backward(logits, ids, dweights, score="softmax", renormalize=True, scale=1.0):
    s = scores(logits, score)
    out = np.zeros_like(s)
    for t in range(s.shape[0]):
        sj = s[t, ids[t]]
        d = dweights[t] * scale
        if renormalize:
            total = sj.sum() + 1e-20
            d = (d - (d * sj).sum() / total) / total
        ds = np.zeros(s.shape[1])
        ds[ids[t]] = d
        if score == "sigmoid":
            out[t] = ds * s[t] * scores(-logits[t:t + 1], score)[0]  # (1 - s has no bits left of a large logit)
        else:
            out[t] = s[t] * (ds - (ds * s[t]).sum())
    return out


def experts_product(x, w, offsets, rows=None):
    x = x if rows is None else x[rows]
    y = np.zeros((x.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        y[a:b] = x[a:b] @ w[e].T
    return y


def experts_input_grad(dy, w, offsets):
    dx = np.zeros((dy.shape[0], w.shape[2]))
    for e in range(w.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        dx[a:b] = dy[a:b] @ w[e]
    return dx


def experts_weight_grad(dy, x, offsets, rows=None):
    x = x if rows is None else x[rows]
    dw = np.zeros((len(offsets) - 1, dy.shape[1], x.shape[1]))
    for e in range(dw.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        dw[e] = dy[a:b].T @ x[a:b]
    return dw


def combine(y, slots, weights=None):
    w = np.ones(slots.shape) if weights is None else weights
    out = np.zeros((slots.shape[0], y.shape[1]))
    for t in range(slots.shape[0]):
        for j in range(slots.shape[1]):
            if 0 <= slots[t, j] < y.shape[0]:
                out[t] += w[t, j] * y[slots[t, j]]
    return out


def combine_backward(dout, y, slots, weights=None):
    w = np.ones(slots.shape) if weights is None else weights
    dy, dw = np.zeros_like(y), np.zeros(slots.shape)
    for t in range(slots.shape[0]):
        for j in range(slots.shape[1]):
            if 0 <= slots[t, j] < y.shape[0]:
                dy[slots[t, j]] = w[t, j] * dout[t]
                dw[t, j] = (dout[t] * y[slots[t, j]]).sum()
    return dy, dw
