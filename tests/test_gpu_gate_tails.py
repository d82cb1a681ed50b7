"""The gates' activations far below zero, where act(z) is many orders of
magnitude smaller than z: relative to the value itself, one element at a time.

The weights are unit rows, so that gate column i of a row is the row's element
i, up is 1 and a product has one term: every result is the activation or its
derivative at a known z, rounded to bf16.

Bounds: Phi(z) = e^(-z^2/2) P(z), the exponent's two products and its constant
each rounded to float32, is off by z^2 2^-23 of the value, P and the
instructions around it by 2^-18; z / (1 + e^-z) by |z| 2^-23 and 2^-18.  A
derivative is a sum of two such terms and is off by that share of each.  A
bf16 rounding: 2^-8 of the value."""

import numpy as np
import pytest
import torch
from scipy.special import expit, ndtr

from tests.hip_path import DEV
from tests.test_gpu_ffn import BF, Case, Rows, f64, within

pytestmark = pytest.mark.gpu

TINY = 1e-37                     # below float32's normal range
LOWEST = -12.5                   # Phi there: 4e-36


@pytest.fixture(scope="module")
def ep():
    from combine_topk_idx_amd import ep as _ep
    return _ep


def act(kind, z):
    """((value, bound), (derivative, bound)), float64."""
    if kind == "silu":
        p = expit(z)
        rel = np.abs(z) * 2.0 ** -23 + 2.0 ** -18
        return (z * p, rel * np.abs(z * p)), (p + z * p * (1 - p), rel * (p + np.abs(z) * p))
    p, d = ndtr(z), z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    rel = z * z * 2.0 ** -23 + 2.0 ** -18
    return (z * p, rel * np.abs(z * p)), (p + d, rel * (p + np.abs(d)))


def bf16(pair):
    v, err = pair
    return v, err + 2.0 ** -8 * (np.abs(v) + err) + TINY


@pytest.mark.parametrize("T", [8, 40, 400])
@pytest.mark.parametrize("quant", ["none", "fp8_b128"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_block_and_gradient(ep, kind, quant, T):
    inter = 64 if quant == "none" else 128
    H = inter + 64
    c = Case(ep, Rows(ep, 5, T=T, k=1, E=1), H, inter, kind, quant)
    z = torch.linspace(LOWEST, 4.0, T * inter, device=DEV).view(T, inter).to(BF)
    for t in (c.x, c.w1, c.w2, c.dy):
        t.zero_()
    c.x[:, :inter], c.x[:, inter] = z, 1.0
    at = torch.arange(inter, device=DEV)
    c.w1[0, at, at], c.w1[0, inter + at, inter], c.w2[0, at, at] = 1.0, 1.0, 1.0
    c.dy[:, :inter] = 1.0
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    zs = f64(z)
    value, _ = act(kind, zs)
    out = f64(c.out[:T])
    within(out[:, :inter], bf16(value), "out")               # bf16(a), exact from there on
    assert not out[:, inter:].any()
    # the gradients' gate and up are the checkpoint's
    ck, _ = c.checkpoint()
    g, u = ck[:, :inter], ck[:, inter:]
    assert np.all(np.abs(u - 1.0) <= 2.0 ** -20)
    if quant == "none":
        assert np.array_equal(g, zs)
    value, slope = act(kind, g)
    # u stands for 1 up to its scale's float32 roundings
    slope = (slope[0] * u, slope[1] + np.abs(slope[0]) * 2.0 ** -20)
    within(f64(c.gx[:T])[:, :inter], bf16(slope), "grad_x")
    # its element `inter`: the sum of du, each rounded to bf16
    total, err = value[0].sum(1), bf16(value)[1].sum(1) + (inter + 2) * 2.0 ** -23 * np.abs(value[0]).sum(1)
    within(f64(c.gx[:T])[:, inter], bf16((total, err)), "grad_x of up")


@pytest.mark.parametrize("T", [20, 500])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_block_scaled(ep, kind, T):
    r = Rows(ep, 6, T=T, k=1, E=1)
    K = I = 128
    z = torch.linspace(LOWEST, 4.0, T, device=DEV)           # one z a row, in every code that the scale allows
    scale = z.abs() / 448.0
    codes = torch.zeros(T, K, dtype=torch.float8_e4m3fn, device=DEV)
    codes[:, : K - 1] = (z.sign() * 448.0)[:, None].to(torch.float8_e4m3fn)
    codes[:, K - 1] = 448.0
    total, at = ep.ep_buffer_bytes(T, K, "fp8_b128")
    buf = torch.zeros(total, dtype=torch.uint8, device=DEV)
    buf[: T * K] = codes.view(torch.uint8).view(-1)
    buf[at:] = scale.view(torch.uint8)
    w = torch.zeros(1, 2 * I, K, dtype=torch.float8_e4m3fn, device=DEV)
    w.view(torch.uint8)[0, torch.arange(I - 1), torch.arange(I - 1)] = 0x38      # 1
    w.view(torch.uint8)[0, I:, K - 1] = 0x38
    out = torch.zeros(T, I, dtype=BF, device=DEV)
    ep.ep_moe_gmm_b128(r.h, buf, "fp8_b128", K, 2 * I, w, torch.ones(1, 2, 1, device=DEV), out, act=kind,
                       recv_count=r.count)
    s = f64(scale)
    g, u = f64(z.sign()) * 448.0 * s, 448.0 * s
    (v, err), (slope, _) = act(kind, g)
    # g and u: one float32 rounding of 448 times the scale
    near = err + np.abs(slope) * np.abs(g) * 2.0 ** -23 + np.abs(v) * 2.0 ** -23
    want = bf16((v * u, near * u + np.abs(v * u) * 2.0 ** -23))
    got = f64(out)
    within(got[:, : I - 1], tuple(np.repeat(x[:, None], I - 1, 1) for x in want), "out")
    assert not got[:, I - 1].any()
