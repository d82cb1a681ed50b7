"""GPU feed-forward block of expert rows against the float64 oracle, within
the rounding bounds that ``oracle/ffn.py`` derives per element."""

import numpy as np
import pytest
import torch

from oracle import ffn as OF
from tests.hip_path import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
CANARY = 77.0


@pytest.fixture(scope="module")
def ep():
    from combine_topk_idx_amd import ep as _ep
    return _ep


def f64(t):
    return t.double().cpu().numpy()


def routing(g, T, k, E, skew, neg):
    p = -skew * np.log(np.arange(1, E + 1)) + g.gumbel(size=(T, E))
    idx = np.argsort(-p, axis=1)[:, :k] if k <= E else g.integers(0, E, size=(T, k))
    idx = g.permutation(E)[idx]
    return np.where(g.random((T, k)) < neg, -1, idx)


class Rows:
    """A layout, and where each expert's rows lie."""

    def __init__(self, ep, seed, T, k, E, skew=0.0, neg=0.0, tmax=None, row_align=1, expert_capacity=0):
        g = np.random.default_rng(seed)
        self.idx = routing(g, T, k, E, skew, neg)
        self.tmax = tmax or T
        self.ws = torch.full((max(256, ep.ep_workspace_bytes_ex(self.tmax, k, E, row_align, expert_capacity)),), 0xA5,
                             dtype=torch.uint8, device=DEV)
        self.count = torch.full((E,), -1, dtype=torch.int64, device=DEV)
        self.h = ep.ep_layout_ex(torch.from_numpy(self.idx).to(DEV), E, self.tmax, row_align, expert_capacity, self.count,
                                 self.ws)
        n = np.bincount(self.idx[self.idx >= 0].ravel(), minlength=E)
        block = -(-n // row_align) * row_align
        if expert_capacity:
            n, block = np.minimum(n, expert_capacity), np.full(E, expert_capacity)
        start = np.cumsum(block) - block
        self.spans = [(e, int(start[e]), int(n[e])) for e in range(E)]
        self.held = np.zeros(self.h.max_rows, bool)
        for _, a, m in self.spans:
            self.held[a:a + m] = True


class Case:
    def __init__(self, ep, rows, H, I, act, quant, seed=1, x_scale=1.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        E, R = rows.h.num_experts, rows.h.max_rows
        rnd = lambda *s, by=1.0: (torch.randn(*s, generator=g, device=DEV) * by).to(BF)   # noqa: E731
        self.ep, self.rows, self.dims, self.act, self.quant = ep, rows, (E, R, H, I), act, quant
        # rows that hold no pair are never read: not a number
        gone = torch.from_numpy(~rows.held).to(DEV)[:, None]
        self.x, self.dy = rnd(R, H, by=x_scale).masked_fill_(gone, np.nan), rnd(R, H).masked_fill_(gone, np.nan)
        self.w1, self.w2 = rnd(E, 2 * I, H, by=H ** -0.5), rnd(E, H, I, by=I ** -0.5)
        new = lambda *s: torch.full(s, CANARY, dtype=BF, device=DEV)   # noqa: E731
        self.out, self.gx = new(R + 1, H), new(R + 1, H)
        self.gw1, self.gw2 = new(E, 2 * I, H), new(E, H, I)
        total, self.at = ep.ep_buffer_bytes(R, 2 * I, quant)
        self.ck = torch.full((total + 64,), 0x5A, dtype=torch.uint8, device=DEV)
        self.total = total
        self.ws = torch.full((ep.ep_ffn_workspace_bytes(R, H, I, E, True),), 0xFF, dtype=torch.uint8, device=DEV)

    def forward(self, count=True, ck=True, stream=None):
        E, R, H, I = self.dims
        self.ep.ep_ffn(self.rows.h, self.x, self.w1, self.w2, self.ws, self.out[:R], act=self.act,
                       recv_count=self.rows.count if count else None, checkpoint=self.ck[:self.total] if ck else None,
                       checkpoint_quant=self.quant, stream=stream)

    def backward(self, count=True, stream=None):
        E, R, H, I = self.dims
        self.ep.ep_ffn_backward(self.rows.h, self.dy, self.x, self.w1, self.w2, self.ck[:self.total], self.ws, self.gx[:R],
                                self.gw1, self.gw2, act=self.act, checkpoint_quant=self.quant,
                                recv_count=self.rows.count if count else None, stream=stream)

    def checkpoint(self):
        """(values, scales) of the checkpoint: float64 [R, 2I], float64 [R, 2I / 128]."""
        E, R, H, I = self.dims
        if self.quant == "none":
            return f64(self.ck[: R * 4 * I].view(BF).view(R, 2 * I)), None
        codes = f64(self.ck[: R * 2 * I].view(torch.float8_e4m3fn).view(R, 2 * I).float())
        scales = f64(self.ck[self.at: self.at + R * (2 * I // 128) * 4].view(torch.float32).view(R, 2 * I // 128))
        return codes * OF.spread(scales), scales

    def check_forward(self):
        E, R, H, I = self.dims
        x, w1, w2, out = f64(self.x), f64(self.w1), f64(self.w2), f64(self.out)
        ck, scales = self.checkpoint()
        for e, a, n in self.rows.spans:
            want = OF.forward(x[a:a + n], w1[e], w2[e], self.act)
            within(out[a:a + n], want["out"], f"out of expert {e}")
            both = tuple(np.concatenate((want["g"][i], want["u"][i]), axis=1) for i in (0, 1))
            if scales is None:
                within(ck[a:a + n], (both[0], both[1] + 2.0 ** -8 * (np.abs(both[0]) + both[1])), f"checkpoint {e}")
            else:
                # the scale is the block's largest magnitude / 448 (three float32 roundings); a value is off by its own
                # error, by a half step of e4m3 and by the scale's error
                v, err = both
                top = np.abs(v).reshape(n, v.shape[1] // 128, 128).max(2)
                top_err = err.reshape(n, v.shape[1] // 128, 128).max(2)
                assert np.all(np.abs(scales[a:a + n] - top / 448) <= (top_err + top * 2.0 ** -22) / 448 + 1e-37)
                half = np.maximum(2.0 ** -4 * (np.abs(v) + err), OF.spread((top + top_err) / 448) * 2.0 ** -10)
                within(ck[a:a + n], (v, err + half * (1 + 2.0 ** -20) + OF.spread(top_err) + np.abs(v) * 2.0 ** -20),
                       f"checkpoint {e}")
        self.untouched(out)

    def check_backward(self):
        E, R, H, I = self.dims
        x, w1, w2, dy = f64(self.x), f64(self.w1), f64(self.w2), f64(self.dy)
        gx, gw1, gw2 = f64(self.gx), f64(self.gw1), f64(self.gw2)
        ck, _ = self.checkpoint()
        for e, a, n in self.rows.spans:
            if n == 0:
                assert not gw1[e].any() and not gw2[e].any()
                continue
            s = slice(a, a + n)
            want = OF.backward(x[s], w1[e], w2[e], ck[s, :I], ck[s, I:], dy[s], self.act)
            within(gx[s], want["grad_x"], f"grad_x of expert {e}")
            within(gw1[e], want["grad_w1"], f"grad_w1 of expert {e}")
            within(gw2[e], want["grad_w2"], f"grad_w2 of expert {e}")
        self.untouched(gx)

    def untouched(self, rows):
        assert np.all(rows[:-1][~self.rows.held] == CANARY) and np.all(rows[-1] == CANARY)


def within(got, want, what):
    v, lim = want
    err = np.abs(got - v)
    assert np.all(err <= lim), f"{what}: worst error / bound {np.nanmax(err / lim):.3g}, NaN {np.isnan(err).sum()}"


# (layout, H, I): every tile height (mean rows an expert up to 32, 64, 192 and more), partial tiles of rows and columns,
# experts without rows, one row, long and short sums
CASES = [
    (dict(T=1, k=1, E=1), 64, 64),
    (dict(T=1, k=2, E=5), 128, 192),
    (dict(T=33, k=2, E=4), 192, 128),
    (dict(T=70, k=3, E=64, skew=1.0), 320, 64),
    (dict(T=129, k=2, E=5, neg=0.3), 448, 320),
    (dict(T=200, k=2, E=3, skew=1.5), 128, 448),
    (dict(T=257, k=1, E=1), 576, 128),
    (dict(T=600, k=2, E=3, skew=1.0), 256, 256),
    (dict(T=45, k=4, E=8, row_align=16, neg=0.2), 128, 128),
    (dict(T=90, k=2, E=4, row_align=128), 64, 384),
    (dict(T=64, k=2, E=6, expert_capacity=24), 192, 128),
    (dict(T=30, k=2, E=512), 64, 64),
    (dict(T=20, k=3, E=7, tmax=400), 128, 128),
]


@pytest.mark.parametrize("quant", ["none", "fp8_b128"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_oracle(ep, i, act, quant):
    lay, H, I = CASES[i]
    if quant != "none":
        I = -(-I // 128) * 128
    c = Case(ep, Rows(ep, 40 + i, **lay), H, I, act, quant, seed=i)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    c.check_forward()
    c.check_backward()
    assert torch.all(c.ck[c.total:] == 0x5A)


@pytest.mark.parametrize("i", [0, 4, 7, 8])
def test_without_checkpoint_the_output_is_the_same(ep, i):
    lay, H, I = CASES[i]
    c = Case(ep, Rows(ep, 40 + i, **lay), H, I, "silu", "none")
    c.forward()
    want = c.out.clone()
    c.out.fill_(CANARY)
    c.ck.fill_(0x11)
    c.forward(ck=False)
    assert torch.equal(c.out.view(torch.int16), want.view(torch.int16)) and torch.all(c.ck == 0x11)
    if lay.get("row_align", 1) == 1:
        c.forward(count=False, ck=False)
        assert torch.equal(c.out.view(torch.int16), want.view(torch.int16))


def test_runs_repeat_bit_for_bit(ep):
    c = Case(ep, Rows(ep, 3, T=300, k=3, E=5, skew=1.0), 320, 192, "silu", "none")
    first = None
    for _ in range(3):
        c.ws.fill_(0xFF)
        c.forward()
        c.backward()
        got = [t.clone().view(torch.int16) for t in (c.out, c.gx, c.gw1, c.gw2)]
        if first:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        first = got


@pytest.mark.parametrize("quant", ["none", "fp8_b128"])
def test_no_tokens_gives_zero_weight_gradients(ep, quant):
    ws = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    idx = torch.zeros(0, 2, dtype=torch.int64, device=DEV)
    r = Rows.__new__(Rows)
    r.ws, r.count = ws, torch.full((3,), -1, dtype=torch.int64, device=DEV)
    r.h = ep.ep_layout(idx, 3, 8, r.count, ws)
    r.held, r.spans = np.zeros(r.h.max_rows, bool), [(e, 0, 0) for e in range(3)]
    c = Case(ep, r, 128, 128, "silu", quant)
    c.forward()
    c.backward()
    assert not c.gw1.any() and not c.gw2.any()
    assert torch.all(c.out == CANARY) and torch.all(c.gx == CANARY)


def test_all_ids_masked(ep):
    c = Case(ep, Rows(ep, 3, T=17, k=2, E=4, neg=1.1), 128, 64, "gelu", "none")
    c.forward()
    c.backward()
    c.check_forward()
    assert not c.gw1.any() and not c.gw2.any()


def test_infinities_stay_in_their_rows(ep):
    """A row with an infinity or NaN changes no other row of the outputs."""
    c = Case(ep, Rows(ep, 9, T=40, k=2, E=3), 128, 128, "silu", "fp8_b128")
    c.forward()
    want, ck = c.out.clone(), c.ck.clone()
    (_, a, n) = c.rows.spans[1]
    c.x[a, 3], c.x[a + n - 1, 100] = np.inf, np.nan
    c.forward()
    bad = torch.zeros(c.out.shape[0], dtype=torch.bool, device=DEV)
    bad[a] = bad[a + n - 1] = True
    assert torch.equal(c.out[~bad], want[~bad])
    assert not torch.isfinite(c.out[bad]).any()
    codes = lambda t: t[: c.dims[1] * 256].view(-1, 256)[~bad[:-1]]   # noqa: E731
    assert torch.equal(codes(c.ck), codes(ck))
    v, scales = c.checkpoint()
    assert not np.isfinite(v[a]).any() and not np.isfinite(v[a + n - 1]).any()


def test_large_and_small_values(ep):
    """Sums far outside the activation's bend: silu(g) u by formula, no overflow inside."""
    for scale in (1e-6, 300.0):
        for act in ("silu", "gelu"):
            c = Case(ep, Rows(ep, 11, T=50, k=2, E=3), 128, 128, act, "fp8_b128", x_scale=scale)
            c.forward()
            c.backward()
            c.check_forward()
            c.check_backward()


def test_busy_side_stream(ep):
    c = Case(ep, Rows(ep, 5, T=200, k=2, E=4), 256, 128, "silu", "fp8_b128")
    c.forward()
    c.backward()
    want = [t.clone() for t in (c.out, c.gx, c.gw1, c.gw2)]
    for t in (c.out, c.gx, c.gw1, c.gw2):
        t.fill_(CANARY)
    side = torch.cuda.Stream()
    x = c.x.clone()
    c.x.fill_(0)
    big = torch.randn(4096, 4096, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(10):
            big = big @ big * 1e-3
        c.x.copy_(x)
        c.forward()
        c.backward()
    side.synchronize()
    for a, b in zip(want, (c.out, c.gx, c.gw1, c.gw2)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("quant", ["none", "fp8_b128"])
def test_whole_step_eager_and_as_a_graph(ep, quant):
    """layout, dispatch, block, combine, its gradient, the block's: replayed over new inputs, eager work between."""
    T, k, E, H, I = 48, 3, 6, 256, 128
    g = torch.Generator(device=DEV).manual_seed(4)
    rnd = lambda *s, by=1.0: (torch.randn(*s, generator=g, device=DEV) * by).to(BF)   # noqa: E731
    new = lambda *s, d=BF: torch.zeros(*s, dtype=d, device=DEV)   # noqa: E731
    R = T * k
    x, gout, w1, w2 = rnd(T, H), rnd(T, H), rnd(E, 2 * I, H, by=H ** -0.5), rnd(E, H, I, by=I ** -0.5)
    idx = torch.randint(-1, E, (T, k), generator=g, device=DEV)
    wts = torch.rand(T, k, generator=g, device=DEV)
    lws, count = new(ep.ep_workspace_bytes(T, k, E), d=torch.uint8), new(E, d=torch.int64)
    recv, dy = new(R, H), new(R, H)
    y, gx, gw1, gw2, out = new(R, H), new(R, H), new(E, 2 * I, H), new(E, H, I), new(T, H)
    ck = new(ep.ep_buffer_bytes(R, 2 * I, quant)[0], d=torch.uint8)
    ws = new(ep.ep_ffn_workspace_bytes(R, H, I, E, True), d=torch.uint8)
    raw = lambda t: t.view(-1).view(torch.uint8)   # noqa: E731

    def step():
        h = ep.ep_layout(idx, E, T, count, lws)
        ep.ep_dispatch(h, x, H, "none", raw(recv))
        ep.ep_ffn(h, recv, w1, w2, ws, y, recv_count=count, checkpoint=ck, checkpoint_quant=quant)
        ep.ep_combine(h, raw(y), "none", H, idx, wts, out)
        ep.ep_combine_backward(h, gout, H, "none", raw(dy), wts)
        ep.ep_ffn_backward(h, dy, recv, w1, w2, ck, ws, gx, gw1, gw2, checkpoint_quant=quant, recv_count=count)

    def results():
        # rows past the last pair keep what was there: compare those that hold one
        n = int(count.sum())
        return [t.clone() for t in (out, y[:n], gx[:n], gw1, gw2)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for i in range(4):
        x.copy_(rnd(T, H))
        gout.copy_(rnd(T, H))
        idx.copy_(torch.randint(-1, E, (T, k), generator=g, device=DEV))
        step()
        want = results()
        for t in (out, y, gx, gw1, gw2, ck, ws):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, results())), i
    # the same step against the formulas, through autograd in float64
    xr = x.double().cpu().requires_grad_()
    p1, p2 = w1.double().cpu().requires_grad_(), w2.double().cpu().requires_grad_()
    total = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            if e >= 0:
                both = p1[e] @ xr[t]
                total[t] = total[t] + float(wts[t, j]) * (p2[e] @ (torch.nn.functional.silu(both[:I]) * both[I:]))
    total.backward(gout.double().cpu())
    near = lambda a, b: (a.double().cpu() - b).norm() / b.norm()   # noqa: E731
    # a few bf16 roundings (2^-9 of the norm each); the 8-bit checkpoint's values are off by up to 2^-4
    assert near(out, total.detach()) < 2.0 ** -6
    lim = 2.0 ** -6 if quant == "none" else 2.0 ** -3
    assert near(gw1, p1.grad) < lim and near(gw2, p2.grad) < lim


@pytest.mark.slow
def test_rows_past_32_bits(ep):
    """Rows whose byte offsets pass 2^32: the last expert's rows against the oracle, the others' by a copy of them."""
    H, I, E, n = 8192, 64, 3, 96
    rows = 4 * (1 << 30) // (2 * H) + 256                 # over 4 GiB of rows, most of them the second expert's
    idx = torch.ones(rows, 1, dtype=torch.int64, device=DEV)
    idx[:40], idx[40:40 + n] = 0, 2
    ws = torch.empty(ep.ep_workspace_bytes(rows, 1, E), dtype=torch.uint8, device=DEV)
    count = torch.empty(E, dtype=torch.int64, device=DEV)
    h = ep.ep_layout(idx, E, rows, count, ws)
    g = torch.Generator(device=DEV).manual_seed(2)
    rnd = lambda *s, by=1.0: (torch.randn(*s, generator=g, device=DEV) * by).to(BF)   # noqa: E731
    x, dy = rnd(rows, H), rnd(rows, H)
    w1, w2 = rnd(E, 2 * I, H, by=H ** -0.5), rnd(E, H, I, by=I ** -0.5)
    out, gx, gw1, gw2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w1), torch.empty_like(w2)
    wsp = torch.empty(ep.ep_ffn_workspace_bytes(rows, H, I, E, True), dtype=torch.uint8, device=DEV)
    ck = torch.empty(ep.ep_buffer_bytes(rows, 2 * I, "none")[0], dtype=torch.uint8, device=DEV)
    ep.ep_ffn(h, x, w1, w2, wsp, out, recv_count=count, checkpoint=ck)
    ep.ep_ffn_backward(h, dy, x, w1, w2, ck, wsp, gx, gw1, gw2, recv_count=count)
    torch.cuda.synchronize()
    ckv = ck.view(BF).view(rows, 2 * I)
    for e, sel, at in ((2, slice(rows - n, rows), 0), (1, slice(rows - n - 64, rows - n), None), (0, slice(0, 40), 0)):
        xs, dys, ws1, ws2 = f64(x[sel]), f64(dy[sel]), f64(w1[e]), f64(w2[e])
        within(f64(out[sel]), OF.forward(xs, ws1, ws2, "silu")["out"], f"out {e}")
        c = f64(ckv[sel])
        want = OF.backward(xs, ws1, ws2, c[:, :I], c[:, I:], dys, "silu")
        within(f64(gx[sel]), want["grad_x"], f"grad_x {e}")
        if at is not None:
            within(f64(gw1[e]), want["grad_w1"], f"grad_w1 {e}")
            within(f64(gw2[e]), want["grad_w2"], f"grad_w2 {e}")


class Counted(Rows):
    """A layout whose experts have the given numbers of rows, tokens in a random order."""

    def __init__(self, ep, counts, seed=0, **layout):
        g = np.random.default_rng(seed)
        ids = g.permutation(np.repeat(np.arange(len(counts)), counts))
        E, T = len(counts), int(sum(counts))
        row_align = layout.get("row_align", 1)
        self.idx, self.tmax = ids.reshape(-1, 1), T
        self.ws = torch.full((ep.ep_workspace_bytes_ex(T, 1, E, row_align, 0),), 0xA5, dtype=torch.uint8, device=DEV)
        self.count = torch.full((E,), -1, dtype=torch.int64, device=DEV)
        self.h = ep.ep_layout_ex(torch.from_numpy(self.idx).to(DEV), E, T, row_align, 0, self.count, self.ws)
        block = -(-np.array(counts) // row_align) * row_align
        start = np.cumsum(block) - block
        self.spans = [(e, int(start[e]), int(n)) for e, n in enumerate(counts)]
        self.held = np.zeros(self.h.max_rows, bool)
        for _, a, n in self.spans:
            self.held[a:a + n] = True


# rows by expert: last tiles of every height of a 256-row tile (and none), whole tiles only, tiles cut into pieces, sums
# of one, two, three and more stages
HEIGHTS = [
    ([257, 321, 385, 449, 0, 512, 256, 300], 64, 64),
    ([257, 321, 385, 449, 0, 512, 256, 300], 192, 128),
    ([255, 256, 193, 254], 320, 192),
    ([1030], 64, 128),
    ([4099], 128, 64),
    ([700, 0, 0, 1], 128, 320),
    # more units than workgroups, the last round half empty or less: its tiles in 2 pieces
    ([9001, 8300], 64, 640),
    # over 32 rows in some experts of a launch of few
    ([100] + [1] * 14, 192, 128),
    ([33, 0, 65, 31, 32, 1], 1024, 64),
]


@pytest.mark.parametrize("quant", ["none", "fp8_b128"])
@pytest.mark.parametrize("i", range(len(HEIGHTS)))
def test_tile_heights(ep, i, quant):
    counts, H, I = HEIGHTS[i]
    if quant != "none":
        I = -(-I // 128) * 128
    c = Case(ep, Counted(ep, counts, i, row_align=1 if i % 2 else 16), H, I, "silu", quant, seed=i)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    c.check_forward()
    c.check_backward()


def few_rows(E, seed):
    """Rows by expert: none to three, 20 and 45 in some."""
    n = np.random.default_rng(seed).integers(0, 4, size=E)
    n[:: 9], n[4:: 31] = 20, 45
    return n


# H and I: from one stage of 64 to eleven, so that waves have none, one and more of them
@pytest.mark.parametrize("ck", [False, True])
@pytest.mark.parametrize("H, I", [(64, 640), (128, 704), (192, 576), (320, 512), (1344, 64), (1088, 128), (1024, 192),
                                  (576, 320)])
def test_few_rows_many_units_a_workgroup(ep, H, I, ck):
    c = Case(ep, Counted(ep, few_rows(150, H)), H, I, "gelu", "none", seed=I)
    assert (c.rows.held.sum() + 149) // 150 <= 32
    c.forward()                                              # fills the checkpoint that check_forward reads
    if not ck:
        first = c.out.clone()
        c.out.fill_(CANARY)
        c.forward(ck=False)
        assert torch.equal(first, c.out)
    torch.cuda.synchronize()
    c.check_forward()


def test_two_graphs_in_turn(ep):
    """Two captured steps of different sizes with a workspace each, replayed in turn and together on two streams."""
    cases = [Case(ep, Rows(ep, 3, T=300, k=2, E=3), 128, 128, "silu", "none"),
             Case(ep, Rows(ep, 4, T=20, k=2, E=5), 192, 64, "gelu", "none")]
    outs = lambda c: (c.out, c.gx, c.gw1, c.gw2)   # noqa: E731
    want, graphs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for c, s in zip(cases, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            c.forward()
            c.backward()
            s.synchronize()
            want.append([t.clone() for t in outs(c)])
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                c.forward()
                c.backward()
            graphs.append(g)
    torch.cuda.synchronize()
    for turn in range(4):
        for c in cases:
            for t in outs(c):
                t.fill_(CANARY)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s if turn % 2 else streams[0]):
                g.replay()
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(outs(c), w))


def test_many_experts_and_the_same_expert_twice(ep):
    """512 experts, most without rows; a token routed to one expert twice has two rows."""
    idx = np.full((40, 2), 7)
    idx[10:, 1] = np.arange(30) * 17 % 512
    r = Rows.__new__(Rows)
    r.ws = torch.zeros(ep.ep_workspace_bytes(40, 2, 512), dtype=torch.uint8, device=DEV)
    r.count = torch.zeros(512, dtype=torch.int64, device=DEV)
    r.idx = idx
    r.h = ep.ep_layout(torch.from_numpy(idx).to(DEV), 512, 40, r.count, r.ws)
    n = np.bincount(idx.ravel(), minlength=512)
    start = np.cumsum(n) - n
    r.spans, r.held = [(e, int(start[e]), int(n[e])) for e in range(512)], np.ones(80, bool)
    c = Case(ep, r, 64, 64, "silu", "none")
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    c.check_forward()
    c.check_backward()
