"""Router of a MoE layer in float64 (test infrastructure only): ids and
weights from the gate's logits, row by row, and the weights' gradient.

Parity: the selection is a sort of Python tuples (key, then id) per row; the
gradient is pinned against central differences of the weights at fixed ids in
``tests/test_oracle_operators.py``.
"""

from __future__ import annotations

import numpy as np


def scores(z: np.ndarray, score: str) -> np.ndarray:
    """softmax or sigmoid of one row; experts at -inf or NaN score 0."""
    there = z > -np.inf
    out = np.zeros(z.shape)
    if not there.any():
        return out
    with np.errstate(over="ignore"):
        if score == "softmax":
            out[there] = np.exp(z[there] - z[there].max())
            return out / out.sum()
        out[there] = 1.0 / (1.0 + np.exp(-z[there]))
    return out


def weights_of(z: np.ndarray, ids, score: str, renormalize: bool, scale: float) -> np.ndarray:
    """The weights of the chosen ids (-1: weight 0) of one row."""
    ids = np.asarray(ids)
    use = ids >= 0
    if renormalize:
        chosen = z[ids[use]]
        log_s = chosen if score == "softmax" else -np.logaddexp(0.0, -chosen)
        p = np.exp(log_s - log_s.max()) if use.any() else log_s
        val = p / p.sum() if use.any() else p
    else:
        val = scores(z, score)[ids[use]]
    w = np.zeros(len(ids))
    w[use] = val * scale
    return w


def route_row(z, k, *, score="softmax", bias=None, num_groups=1, topk_groups=1, group_top=1, renormalize=True,
              scale=1.0):
    z = np.minimum(np.asarray(z, np.float64), float(np.finfo(np.float32).max))
    E = z.size
    there = z > -np.inf
    s = scores(z, score)
    c = np.where(there, s + (0.0 if bias is None else np.asarray(bias, np.float64)), -np.inf)
    c = np.where(c > -np.inf, c, -np.inf)                     # a NaN bias
    key = c if bias is not None else np.where(there, z, -np.inf)
    if num_groups > 1:
        size = E // num_groups
        by = c if group_top == 2 else key
        rank = []
        for g in range(num_groups):
            best = sorted(by[g * size:(g + 1) * size], reverse=True)[:group_top]
            rank.append((-sum(best) if min(best) > -np.inf else np.inf, g))
        kept = {g for _, g in sorted(rank)[:topk_groups]}
        key = np.array([key[e] if e // size in kept else -np.inf for e in range(E)])
    order = sorted((-key[e], e) for e in range(E) if key[e] > -np.inf)[:k]
    ids = [e for _, e in order] + [-1] * (k - len(order))
    return ids, weights_of(z, ids, score, renormalize, scale)


def route(logits, k, **kw):
    rows = [route_row(z, k, **kw) for z in np.asarray(logits, np.float64)]
    T = len(rows)
    return (np.array([r[0] for r in rows], np.int64).reshape(T, k),
            np.array([r[1] for r in rows], np.float64).reshape(T, k))


def backward_row(z, ids, grad, *, score="softmax", renormalize=True, scale=1.0):
    """d(sum_j grad_j w_j) / dz at fixed ids: the Jacobian written out."""
    z = np.minimum(np.asarray(z, np.float64), float(np.finfo(np.float32).max))
    E, ids = z.size, np.asarray(ids)
    dz = np.zeros(E)
    use = [j for j, e in enumerate(ids) if 0 <= e < E and z[e] > -np.inf]
    if not use:
        return dz
    s = scores(z, score)
    idu = [e if j in use else -1 for j, e in enumerate(ids)]
    w = weights_of(z, idu, score, renormalize, 1.0)

    def dlog(e):                                              # d log s_e / dz
        d = np.zeros(E)
        if score == "softmax":
            d -= s
            d[e] += 1.0
        else:
            with np.errstate(over="ignore"):
                d[e] = 1.0 / (1.0 + np.exp(z[e]))
        return d

    for j in use:
        d = dlog(ids[j])
        if renormalize:
            d = d - sum(w[i] * dlog(ids[i]) for i in use)
        dz += scale * float(grad[j]) * w[j] * d
    return dz


def backward(logits, ids, grad, **kw):
    return np.stack([backward_row(z, i, g, **kw) for z, i, g in zip(np.asarray(logits, np.float64), ids, grad)])
