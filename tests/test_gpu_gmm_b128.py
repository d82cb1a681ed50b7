"""GPU block-scaled product against float64, within the matrix-core model's
bound (``tests/moe_bounds.py``) and the roundings after it."""

import numpy as np
import pytest
import torch

from oracle import codecs, ffn as OF
from tests import moe_bounds as MB
from tests.hip_path import DEV
from tests.test_gpu_ffn import BF, CANARY, Counted, Rows, f64, few_rows, within

pytestmark = pytest.mark.gpu

MODES = ["fp8_b128", "fp8_b128_pow2", "fp8_b128_ue8m0"]


@pytest.fixture(scope="module")
def ep():
    from combine_topk_idx_amd import ep as _ep
    return _ep


class Case:
    def __init__(self, ep, rows, K, N, mode, transposed=False, act="none", out_quant="none", seed=0):
        g = np.random.default_rng(seed)
        E, R = rows.h.num_experts, rows.h.max_rows
        self.ep, self.rows, self.dims = ep, rows, (E, R, K, N)
        self.mode, self.transposed, self.act, self.out_quant = mode, transposed, act, out_quant
        # any code but NaN, scales over a wide range; rows that hold no pair are NaN
        finite = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
        codes = finite[g.integers(0, finite.size, size=(R, K))]
        exps = g.integers(-12, 4, size=(R, K // 128))
        scales = np.exp2(exps) * (1 if mode != "fp8_b128" else g.random(exps.shape) + 0.5)
        scales = scales.astype(np.float32)
        codes[~rows.held] = 0x7F
        self.x = codecs.e4m3_decode(codes).astype(np.float64) * OF.spread(scales)
        total, at = ep.ep_buffer_bytes(R, K, mode)
        buf = np.full(total, 0x7F, np.uint8)
        buf[: R * K] = codes.ravel()
        if mode == "fp8_b128_ue8m0":
            b = (exps + 127).astype(np.uint8)
            b[~rows.held] = 0xFF
            buf[at:] = b.ravel()
        else:
            scales[~rows.held] = np.nan
            buf[at:] = scales.ravel().view(np.uint8)
        self.buf = torch.from_numpy(buf).to(DEV)
        n, k = (K, N) if transposed else (N, K)
        w = finite[g.integers(0, finite.size, size=(E, n, k))]
        ws = ((g.random((E, n // 128, k // 128)) + 0.5) * 2.0 ** -8).astype(np.float32)
        self.w = codecs.e4m3_decode(w).astype(np.float64) * OF.spread(ws, 128)
        self.wd, self.wsd = torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV)
        self.width = N // 2 if act != "none" else N
        if out_quant == "none":
            self.out = torch.full((R + 1, self.width), CANARY, dtype=BF, device=DEV)
        else:
            self.total, self.at = ep.ep_buffer_bytes(R, self.width, out_quant)
            self.out = torch.full((self.total + 64,), 0x33, dtype=torch.uint8, device=DEV)

    def run(self, **kw):
        E, R, K, N = self.dims
        out = self.out[:R] if self.out_quant == "none" else self.out[:self.total]
        kw.setdefault("recv_count", self.rows.count)
        self.ep.ep_moe_gmm_b128(self.rows.h, self.buf, self.mode, K, N, self.wd, self.wsd, out, act=self.act,
                                transposed=self.transposed, out_quant=self.out_quant, **kw)

    def want(self, e, a, n):
        """(value, bound) of the rows' float32 results."""
        E, R, K, N = self.dims
        x, w = self.x[a:a + n], self.w[e].T if self.transposed else self.w[e]
        y = x @ w.T
        # the model's bound, and the scales' product, its use and the sum of the blocks in float32
        err = MB.dot_bound(x, w) + (K // 128 + 4) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
        if self.act == "none":
            return y, err
        g, u, eg, eu = y[:, :N // 2], y[:, N // 2:], err[:, :N // 2], err[:, N // 2:]
        f, _ = OF.act(self.act, g)
        ef = OF.SLOPE * eg + OF.EVAL * (1.0 + np.abs(g))
        return f * u, ef * (np.abs(u) + eu) + np.abs(f) * eu + OF.EVAL * np.abs(f * u)

    def check(self):
        E, R, K, N = self.dims
        if self.out_quant == "none":
            got = f64(self.out)
            for e, a, n in self.rows.spans:
                v, err = self.want(e, a, n)
                within(got[a:a + n], (v, err + 2.0 ** -8 * (np.abs(v) + err) + 1e-37), f"expert {e}")
            assert np.all(got[:-1][~self.rows.held] == CANARY) and np.all(got[-1] == CANARY)
            return
        raw = self.out.cpu().numpy()
        assert np.all(raw[self.total:] == 0x33)
        codes = raw[: R * self.width].reshape(R, self.width)
        assert np.all(codes[~self.rows.held] == 0x33)
        blocks = self.width // 128
        if self.out_quant == "fp8_b128_ue8m0":
            b = raw[self.at: self.at + R * blocks].reshape(R, blocks)
            scales = np.where(b > 0, np.exp2(b.astype(np.float64) - 127), 0.0)
        else:
            scales = raw[self.at: self.at + R * blocks * 4].view(np.float32).reshape(R, blocks).astype(np.float64)
        val = codecs.e4m3_decode(codes).astype(np.float64)
        for e, a, n in self.rows.spans:
            v, err = self.want(e, a, n)
            s = scales[a:a + n]
            top, top_err = np.abs(v).reshape(n, v.shape[1] // 128, 128).max(2), err.reshape(n, v.shape[1] // 128, 128).max(2)
            if self.out_quant == "fp8_b128":
                assert np.all(np.abs(s - top / 448) <= (top_err + top * 2.0 ** -22) / 448 + 1e-37)
                off = OF.spread(top_err) + np.abs(v) * 2.0 ** -20
            else:
                # a power of two, the smallest not below amax / 448 up to the amax's error
                assert np.all(np.exp2(np.round(np.log2(s))) == s)
                assert np.all(s * 448 >= (top - top_err) * (1 - 2.0 ** -22))
                assert np.all(s * 224 <= (top + top_err) * (1 + 2.0 ** -22))
                off = 0.0
            # a value within half a step of e4m3 (2^-4, or half the smallest step) and of its own error; where the
            # largest magnitude lies above 448 scales by its error, the code is clamped by as much
            half = np.maximum(2.0 ** -4 * (np.abs(v) + err), OF.spread(s) * 2.0 ** -10)
            within(val[a:a + n] * OF.spread(s), (v, 2 * err + half * (1 + 2.0 ** -20) + off + 1e-37), f"expert {e}")


CASES = [
    (dict(T=1, k=1, E=1), 128, 128),
    (dict(T=1, k=2, E=5), 384, 256),
    (dict(T=40, k=2, E=64, skew=1.0), 640, 384),
    (dict(T=100, k=2, E=4, neg=0.3), 1408, 256),
    (dict(T=150, k=2, E=3, skew=1.0), 256, 640),
    (dict(T=300, k=2, E=2), 768, 512),
    (dict(T=45, k=4, E=8, row_align=16), 512, 256),
    (dict(T=64, k=2, E=6, expert_capacity=24), 128, 512),
    (dict(T=20, k=2, E=512), 256, 128),
    (dict(T=20, k=3, E=7, tmax=300), 256, 256),
]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_product(ep, i, transposed, mode):
    lay, K, N = CASES[i]
    c = Case(ep, Rows(ep, 70 + i, **lay), K, N, mode, transposed=transposed, seed=i)
    c.run()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("out_quant", ["none", *MODES])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("i", [0, 2, 3, 4, 5, 6])
def test_gated(ep, i, act, out_quant):
    lay, K, N = CASES[i]
    c = Case(ep, Rows(ep, 70 + i, **lay), K, -(-N // 256) * 256, MODES[i % 3], act=act, out_quant=out_quant, seed=i)
    c.run()
    torch.cuda.synchronize()
    c.check()


def test_without_counts_and_repeated(ep):
    c = Case(ep, Rows(ep, 1, T=90, k=2, E=3), 512, 384, "fp8_b128")
    c.run()
    want = c.out.clone()
    for _ in range(3):
        c.out.fill_(CANARY)
        c.run(recv_count=None)
        assert torch.equal(c.out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("mode", MODES)
def test_the_rows_of_a_dispatch(ep, mode):
    """The receive rows as ep_dispatch writes them, through the gated product into the next one, and back."""
    T, k, E, H, I = 60, 2, 4, 256, 128
    r = Rows(ep, 8, T=T, k=k, E=E)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(T, H, generator=g, device=DEV).to(BF)
    R = r.h.max_rows
    new = lambda w, q: torch.zeros(ep.ep_buffer_bytes(R, w, q)[0], dtype=torch.uint8, device=DEV)   # noqa: E731
    recv, act, grad = new(H, mode), new(I, mode), new(H, mode)
    ep.ep_dispatch(r.h, x, H, mode, recv)
    w1 = torch.randn(E, 2 * I, H, generator=g, device=DEV).to(torch.float8_e4m3fn)
    w2 = torch.randn(E, H, I, generator=g, device=DEV).to(torch.float8_e4m3fn)
    s1 = torch.rand(E, 2 * I // 128, H // 128, generator=g, device=DEV) * 0.1 + 0.02
    s2 = torch.rand(E, H // 128, I // 128, generator=g, device=DEV) * 0.1 + 0.02
    y, gi = torch.zeros(R, H, dtype=BF, device=DEV), torch.zeros(R, I, dtype=BF, device=DEV)
    ep.ep_moe_gmm_b128(r.h, recv, mode, H, 2 * I, w1, s1, act, act="silu", out_quant=mode, recv_count=r.count)
    ep.ep_moe_gmm_b128(r.h, act, mode, I, H, w2, s2, y, recv_count=r.count)
    ep.ep_combine_backward(r.h, x, H, mode, grad)
    ep.ep_moe_gmm_b128(r.h, grad, mode, H, I, w2, s2, gi, transposed=True, recv_count=r.count)
    torch.cuda.synchronize()

    def values(buf, w):
        codes, scales = ep.split_recv(buf, R, w, mode)
        return f64(codes.float()) * OF.spread(f64(scales.float()))
    xr, ar, gr = values(recv, H), values(act, I), values(grad, H)
    for e, a, n in r.spans:
        s = slice(a, a + n)
        m1 = f64(w1[e].float()) * OF.spread(f64(s1[e]), 128)
        m2 = f64(w2[e].float()) * OF.spread(f64(s2[e]), 128)
        for got, rows, m in ((y, ar, m2), (gi, gr, m2.T)):
            err = MB.dot_bound(rows[s], m) + 8 * 2.0 ** -23 * (np.abs(rows[s]) @ np.abs(m).T)
            v = rows[s] @ m.T
            within(f64(got[s]), (v, err + 2.0 ** -8 * (np.abs(v) + err) + 1e-37), f"expert {e}")
        both = xr[s] @ m1.T
        eb = MB.dot_bound(xr[s], m1) + 8 * 2.0 ** -23 * (np.abs(xr[s]) @ np.abs(m1).T)
        v = OF.act("silu", both[:, :I])[0] * both[:, I:]
        err = OF.SLOPE * eb[:, :I] * (np.abs(both[:, I:]) + eb[:, I:]) + np.abs(both[:, :I]) * eb[:, I:] + 2.0 ** -18
        top = np.abs(v).max(1, keepdims=True)
        # e4m3: half a step, 2^-4 of the value or 2^-10 of the scale (at most twice amax / 448)
        assert np.all(np.abs(ar[s] - v) <= 2.0 ** -4 * (np.abs(v) + err) + 2 * err + (top + err.max()) / 224 * 2.0 ** -10
                      + err.max())


def test_side_stream_and_graph(ep):
    c = Case(ep, Rows(ep, 2, T=80, k=2, E=4), 512, 256, "fp8_b128", act="silu")
    c.run()
    want = c.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.run()
    for _ in range(4):
        c.out.fill_(CANARY)
        torch.randn(1000, device=DEV).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out.view(torch.int16), want.view(torch.int16))


HEIGHTS = [
    ([257, 321, 385, 449, 0, 256], 128, 128),
    ([255, 193, 254], 256, 384),
    ([700], 384, 512),
    ([200, 0, 330], 640, 256),
    ([100] + [1] * 14, 1152, 256),
    ([33, 0, 65, 31, 32, 1], 256, 128),
]


@pytest.mark.parametrize("form", ["plain", "transposed", "gated"])
@pytest.mark.parametrize("mode", ["fp8_b128", "fp8_b128_ue8m0"])
@pytest.mark.parametrize("i", range(len(HEIGHTS)))
def test_tile_heights(ep, i, mode, form):
    """Last tiles of every height, tiles cut into pieces, sums of one to nine blocks."""
    counts, K, N = HEIGHTS[i]
    c = Case(ep, Counted(ep, counts, i, row_align=1 if i % 2 else 16), K, N if form != "gated" else -(-N // 256) * 256, mode,
             transposed=form == "transposed", act="silu" if form == "gated" else "none", seed=i)
    c.run()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("mode", ["fp8_b128", "fp8_b128_ue8m0"])
@pytest.mark.parametrize("K", [128, 256, 384, 640, 1152])
def test_few_rows_many_units_a_workgroup(ep, K, mode, act):
    c = Case(ep, Counted(ep, few_rows(60, K)), K, 1024, mode, act=act, seed=K)
    c.run()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("T", [60, 500])
def test_nan_codes_and_scales_stay_in_their_rows(ep, T):
    c = Case(ep, Rows(ep, 6, T=T, k=1, E=2), 256, 256, "fp8_b128")
    c.run()
    want = c.out.clone()
    E, R, K, N = c.dims
    c.buf[3 * K + 5] = 0x7F                                    # a NaN code in row 3
    at = ep.ep_buffer_bytes(R, K, "fp8_b128")[1]
    c.buf[at + (R - 2) * 8: at + (R - 2) * 8 + 4].view(torch.float32).fill_(float("inf"))
    c.run()
    bad = torch.zeros(R + 1, dtype=torch.bool, device=DEV)
    bad[3] = bad[R - 2] = True
    assert torch.equal(c.out[~bad], want[~bad])
    assert c.out[3].isnan().all() and not torch.isfinite(c.out[R - 2]).any()
