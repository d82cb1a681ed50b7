"""Gated feed-forward block of expert rows and the block-scaled product in
float64, with a bound on the rounding of each result (test infrastructure
only).

For one expert, rows x [n, H], W1 [2I, H] (gate rows, then up rows), W2 [H, I]:

    g = x Wg^T, u = x Wu^T, a = act(g) * u, y = a W2^T
    da = dy W2, dg = da u act'(g), du = da act(g)
    dx = [dg du] W1, dW1 = [dg du]^T x, dW2 = dy^T a

with act(z) = z / (1 + exp(-z)) or z Phi(z).  The backward pass takes g and u as
the checkpoint holds them.

Bounds (float64 arrays of the results' shapes): a float32 sum of n products of
bf16 values, which float32 holds exactly, in any order is off by at most
(n + 2) 2^-23 of the sum of the products' magnitudes (2^-23 also covers a sum
that truncates); a bf16 rounding by 2^-8 of the value (half a step relative
to the smallest value of a binade); act and act' evaluated in float32 by
2^-20 of the value and of 1 + |z| (a few roundings of quantities no larger
than that).  Errors of inputs go through products by the product rule, with
|act'| <= 1.13 and |act''| <= 1 (the largest |act'| is 1.0998 for silu and
1.1290 for gelu, the largest |act''| 0.5 and 0.798).

The block-scaled product is a plain float64 product of dequantised values.

Parity: no page describes these operators ("parity unpinned"); the formulas are
pinned by central differences and by brute-force sums in
``tests/test_oracle_ffn.py``.
"""

from __future__ import annotations

import numpy as np
from scipy.special import erf, expit

BF16_HALF = 2.0 ** -8
EVAL = 2.0 ** -20
SLOPE, BEND = 1.13, 1.0
TINY = 1e-37                     # below float32's normal range


def _sum(n):
    return (n + 2) * 2.0 ** -23


def act(kind, z):
    """The activation and its derivative."""
    if kind == "silu":
        p = expit(z)
        return z * p, p + z * p * (1.0 - p)
    p = 0.5 * (1.0 + erf(z / np.sqrt(2.0)))
    return z * p, p + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)


def _dot(a, b, ea=None):
    """a b^T and its bound, ea the bound of a."""
    v = a @ b.T
    e = _sum(a.shape[1]) * (np.abs(a) @ np.abs(b).T)
    if ea is not None:
        e = e + (1.0 + _sum(a.shape[1])) * (ea @ np.abs(b).T)
    return v, e


def _rounded(v, e):
    return v, e + BF16_HALF * (np.abs(v) + e) + TINY


def forward(x, w1, w2, kind):
    """dict of g, u (unrounded), out: (value, bound)."""
    inter = w2.shape[1]
    g, eg = _dot(x, w1[:inter])
    u, eu = _dot(x, w1[inter:])
    f, _ = act(kind, g)
    a = f * u
    ef = SLOPE * eg + EVAL * (1.0 + np.abs(g))
    ea = ef * (np.abs(u) + eu) + np.abs(f) * eu + EVAL * np.abs(a)
    a, ea = _rounded(a, ea)
    return dict(g=(g, eg), u=(u, eu), out=_rounded(*_dot(a, w2, ea)))


def backward(x, w1, w2, g, u, dy, kind):
    """dict of grad_x, grad_w1, grad_w2: (value, bound), from the
    checkpoint's g and u."""
    da, eda = _dot(dy, w2.T)
    f, df = act(kind, g)
    ef = EVAL * (1.0 + np.abs(g))                       # of f and of df
    dg, du, a = da * u * df, da * f, f * u
    edg = eda * np.abs(u) * (np.abs(df) + ef) + np.abs(da * u) * ef + EVAL * np.abs(dg)
    edu = eda * (np.abs(f) + ef) + np.abs(da) * ef + EVAL * np.abs(du)
    a, ea = _rounded(a, np.abs(u) * ef + EVAL * np.abs(a))
    d = np.concatenate((dg, du), axis=1)
    d, ed = _rounded(d, np.concatenate((edg, edu), axis=1))
    return dict(grad_x=_rounded(*_dot(d, w1.T, ed)), grad_w1=_rounded(*_dot(d.T, x.T, ed.T)),
                grad_w2=_rounded(*_t(_dot(a.T, dy.T, ea.T))))


def _t(pair):
    return pair[0].T, pair[1].T


def spread(scales, rows=1):
    """Scales of blocks of 128 (of 128 x 128 with rows = 128) spread over the
    values they cover."""
    return np.repeat(np.repeat(np.asarray(scales, np.float64), 128, axis=-1), rows, axis=-2)
