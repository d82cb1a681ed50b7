"""Expert layer and routed low-rank adapters in float64 (test infrastructure
only), with bounds on what rounding may do to them.

Parity: plain matrix products per (token, expert); the adapters' gradients are
pinned against central differences in ``tests/test_oracle_operators.py``.
"""

from __future__ import annotations

import numpy as np

from . import codecs
from .moe import mx_dequant, silu

F32 = 2.0 ** -24        # half a step of float32, relative
BF16 = 2.0 ** -8        # half a step of bf16, relative


def weight_values(w, scales, quant: str) -> np.ndarray:
    """float64 values of expert weights: bf16 patterns (uint16), MXFP8 codes
    or MXFP4 bytes."""
    if quant == "none":
        return codecs.bf16_bits_to_f32(w).astype(np.float64)
    if quant == "mxfp8":
        return mx_dequant(w, scales)
    v = codecs.e2m1_decode(codecs.unpack_e2m1_pairs(w))
    return v * np.repeat(codecs.e8m0_decode(scales), 32, axis=-1)


def expert_layer(x, ids, weights, w1, w2):
    """x [T, H] float64, ids [T, k], weights [T, k], w1 [E, 2I, H], w2
    [E, H, I] float64.  Returns (out, bound): float64 outputs and how far a
    bf16 output may be off that holds the sums in float32 and rounds the
    activations a and the result to bf16:

      g, u:  (K + 2) F32 sum |w x|         (K-term sums, any order)
      a:     1.1 dg |u| + |silu(g)| du (|silu'| < 1.1), 8 F32 |a| for silu
             and the product, BF16 |a| for the rounding
      y:     |W2| da + (K + 2) F32 |W2| |a|
      out:   sum |w| dy + (k + 1) F32 sum |w y| + BF16 |out|
    """
    T, H = x.shape
    E, inter = w2.shape[0], w2.shape[2]
    out, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < E:
                continue
            gu, mag = w1[e] @ x[t], np.abs(w1[e]) @ np.abs(x[t])
            d = (H + 2) * F32 * mag
            g, u, dg, du = gu[:inter], gu[inter:], d[:inter], d[inter:]
            a = silu(g) * u
            da = 1.1 * dg * (np.abs(u) + du) + np.abs(silu(g)) * du + (8 * F32 + BF16) * np.abs(a)
            da += BF16 * da
            y = w2[e] @ a
            dy = np.abs(w2[e]) @ (da + (inter + 2) * F32 * (np.abs(a) + da))
            wt = float(weights[t, j])
            out[t] += wt * y
            bound[t] += abs(wt) * dy + (len(ids[t]) + 1) * F32 * abs(wt) * (np.abs(y) + dy)
    return out, bound + BF16 * (np.abs(out) + bound) + 2.0 ** -133


def lora(x, ids, a, b, scale, base):
    """x [T, in], ids [T], a [N, r, in], b [N, out, r], scale [N], base
    [T, out], all float64.  Returns (out, out_bound, down, down_bound): v
    summed in float32, cut into two bf16 parts (2^-17 of it is lost at most:
    half a bf16 step of a remainder of half a bf16 step), summed in float32
    again and rounded to bf16 with base."""
    T = x.shape[0]
    r, fin = a.shape[1], a.shape[2]
    out, bound = base.copy(), np.zeros(base.shape)
    down, dv = np.zeros((T, r)), np.zeros((T, r))
    for t in range(T):
        e = ids[t]
        if not 0 <= e < len(a):
            continue
        down[t] = a[e] @ x[t]
        dv[t] = (fin + 2) * F32 * (np.abs(a[e]) @ np.abs(x[t]))
        out[t] += scale[e] * (b[e] @ down[t])
        dd = dv[t] + (2.0 ** -16 + (r + 4) * F32 * 3) * (np.abs(down[t]) + dv[t])
        bound[t] += abs(scale[e]) * (np.abs(b[e]) @ dd)
    bound += 2 * F32 * (np.abs(base) + bound)
    return out, bound + BF16 * (np.abs(out) + bound) + 2.0 ** -133, down, dv


def lora_backward(x, ids, a, b, scale, grad_out, grad_base, down, down_bound):
    """Returns {name: (value, bound)} of grad_x, grad_a and grad_b; ``down``
    is the exact v and ``down_bound`` how far the one used may be off."""
    N, r, fin = a.shape
    fout = b.shape[1]
    gx, bx = grad_base.copy(), np.zeros(grad_base.shape)
    ga, ba = np.zeros(a.shape), np.zeros(a.shape)
    gb, bb = np.zeros(b.shape), np.zeros(b.shape)
    count = np.bincount([i for i in ids if 0 <= i < N], minlength=N)
    for t in range(x.shape[0]):
        e = ids[t]
        if not 0 <= e < N:
            continue
        u = scale[e] * (b[e].T @ grad_out[t])
        du = abs(scale[e]) * (fout + 3) * F32 * (np.abs(b[e]).T @ np.abs(grad_out[t]))
        gx[t] += a[e].T @ u
        bx[t] += np.abs(a[e]).T @ (du + (2.0 ** -16 + (r + 4) * F32 * 3) * (np.abs(u) + du))
        # the float32 factor whole (three bf16 parts), the sum over the tokens in float32
        rel = 3 * (count[e] + 4) * F32
        ga[e] += np.outer(u, x[t])
        ba[e] += np.outer(du + rel * (np.abs(u) + du), np.abs(x[t]))
        gb[e] += scale[e] * np.outer(grad_out[t], down[t])
        bb[e] += abs(scale[e]) * np.outer(np.abs(grad_out[t]),
                                          down_bound[t] + rel * (np.abs(down[t]) + down_bound[t]))
    bx += 2 * F32 * (np.abs(grad_base) + bx)
    return {"grad_x": (gx, bx + BF16 * (np.abs(gx) + bx) + 2.0 ** -133), "grad_a": (ga, ba + 1e-37),
            "grad_b": (gb, bb + 1e-37)}
