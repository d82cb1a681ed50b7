"""GPU routed low-rank adapters against the float64 oracle, within the
rounding bounds that ``oracle/layer.py`` derives per element."""

import numpy as np
import pytest
import torch

from combine_topk_idx_amd import workloads as W
from oracle import codecs, layer as OY
from tests.hip_path import DEV, to_dev

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def ep():
    from combine_topk_idx_amd import ep as _ep
    return _ep


def _f64(bits):
    return codecs.bf16_bits_to_f32(bits).astype(np.float64)


class Lora:
    def __init__(self, ep, seed, T, fin, fout, r, N, none=0.2, skew=False, tmax=None, **layout):
        g = np.random.default_rng(seed)
        self.ep, self.shape = ep, (T, fin, fout, r, N)
        rows = lambda *s: W.bf16_from_f32(g.normal(size=s).astype(np.float32))   # noqa: E731
        self.x, self.base, self.dy, self.gb = rows(T, fin), rows(T, fout), rows(T, fout), rows(T, fin)
        self.a = W.bf16_from_f32((g.normal(size=(N, r, fin)) / np.sqrt(fin)).astype(np.float32))
        self.b = W.bf16_from_f32((g.normal(size=(N, fout, r)) / np.sqrt(r)).astype(np.float32))
        self.scale = (g.random(N) + 0.5).astype(np.float32)
        self.ids = g.integers(0, max(1, N // 4) if skew else N, size=T)
        self.ids[g.random(T) < none] = -1
        self.layout, self.tmax = layout, tmax or T

    def handle(self):
        T, N = self.shape[0], self.shape[4]
        ep, align, cap = self.ep, self.layout.get("row_align", 1), self.layout.get("expert_capacity", 0)
        self.lws = torch.full((ep.ep_workspace_bytes_ex(self.tmax, 1, N, align, cap),), 0xA5, dtype=torch.uint8, device=DEV)
        self.rc = torch.empty(N, dtype=torch.int64, device=DEV)
        self.idt = torch.from_numpy(self.ids.reshape(T, 1)).to(DEV)
        return ep.ep_layout_ex(self.idt, N, self.tmax, align, cap, self.rc, self.lws)

    def buffers(self):
        T, fin, fout, r, N = self.shape
        rows = max(T, self.ep.ep_layout_rows(self.tmax, 1, N, self.layout.get("row_align", 1),
                                             self.layout.get("expert_capacity", 0)))
        nan = float("nan")
        d = dict(out=torch.full((T, fout), nan, dtype=BF, device=DEV), down=torch.full((T, r), nan, device=DEV),
                 grad_x=torch.full((T, fin), nan, dtype=BF, device=DEV),
                 grad_a=torch.full((N, r, fin), nan, device=DEV), grad_b=torch.full((N, fout, r), nan, device=DEV),
                 ws=torch.full((self.ep.ep_lora_workspace_bytes(rows, fin, fout, r, N, True),), 0xFF, dtype=torch.uint8,
                               device=DEV))
        d.update({n: to_dev(getattr(self, n)) for n in ("x", "base", "dy", "gb", "a", "b", "scale")})
        return d

    def run(self, d, h, base="base", gb="gb"):
        base, gb = (d[n] if isinstance(n, str) else n for n in (base, gb))
        self.ep.ep_lora(h, d["x"], d["a"], d["b"], d["out"], d["down"], d["ws"], scale=d["scale"], base=base)
        self.ep.ep_lora_backward(h, d["dy"], d["x"], d["a"], d["b"], d["down"], d["grad_x"], d["grad_a"], d["grad_b"],
                                 d["ws"], scale=d["scale"], grad_base=gb)

    def check(self, d, base=True, scale=True):
        T, fin, fout, r, N = self.shape
        x, a, b = _f64(self.x), _f64(self.a), _f64(self.b)
        s = self.scale.astype(np.float64) if scale else np.ones(N)
        bs = _f64(self.base) if base else np.zeros((T, fout))
        gb = _f64(self.gb) if base else np.zeros((T, fin))
        out, bound, down, dv = OY.lora(x, self.ids, a, b, s, bs)
        want = OY.lora_backward(x, self.ids, a, b, s, _f64(self.dy), gb, down, dv)
        want["out"] = (out, bound)
        for n, (v, lim) in want.items():
            err = np.abs(d[n].double().cpu().numpy() - v)
            assert np.all(err <= lim), f"{n}: worst error / bound {np.nanmax(err / lim):.3g}"
        got = d["down"].double().cpu().numpy()
        on = (self.ids >= 0) & (self.ids < N)
        assert np.all(np.abs(got - down)[on] <= dv[on] + 1e-37)
        assert np.all(np.isnan(got[~on]))                    # rows without an adapter are left as they were


CASES = [
    # T, in, out, rank, N
    (1, 32, 32, 8, 1), (1, 2080, 96, 16, 5), (3, 64, 544, 24, 2), (37, 96, 64, 40, 3), (200, 160, 96, 64, 4),
    (65, 64, 64, 128, 2), (129, 1056, 32, 8, 64), (70, 32, 1056, 104, 512), (500, 64, 96, 32, 3),
    # every number of 16-rank steps
    (40, 64, 160, 72, 2), (40, 96, 64, 96, 3), (33, 64, 64, 112, 2), (64, 64, 64, 48, 1),
    # adapters of several pieces (256 tokens at rank 8), beside some of one and of none
    (1100, 64, 32, 8, 2), (900, 32, 96, 8, 9), (700, 160, 64, 16, 65), (2300, 32, 32, 40, 3),
    # more tokens than the reduction axis is split for
    (17000, 128, 64, 8, 3),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_lora(ep, i):
    print(f"\n[case] lora {CASES[i]}", flush=True)
    l = Lora(ep, 40 + i, *CASES[i], none=0.0 if i == 0 else 0.2, skew=i % 2 == 0)
    d = l.buffers()
    l.run(d, l.handle())
    l.check(d)


@pytest.mark.parametrize("T,fin,fout,r,n", [
    # long axes and few rows an adapter: the down products in several shares, at every number of rank steps
    (2, 2112, 2080, 24, 3), (5, 2080, 1056, 40, 7), (3, 3104, 2112, 64, 4), (2, 2080, 2080, 88, 5), (2, 3104, 4160, 128, 70),
    # adapters without tokens beside some with: their gradients are zeros, whole or in part of a column block
    (3, 160, 96, 32, 60), (40, 608, 32, 72, 33), (9, 32, 1184, 16, 500),
])
def test_lora_long_axes_and_idle_adapters(ep, T, fin, fout, r, n):
    print(f"\n[case] lora {(T, fin, fout, r, n)}", flush=True)
    l = Lora(ep, 90 + r, T, fin, fout, r, n, none=0.0, skew=False)
    d = l.buffers()
    l.run(d, l.handle())
    l.check(d)


@pytest.mark.parametrize("layout", [dict(row_align=48), dict(row_align=1024), dict(expert_capacity=70)])
def test_lora_padded_layouts(ep, layout):
    l = Lora(ep, 60, 66, 96, 64, 16, 4, tmax=90, **layout)
    d = l.buffers()
    l.run(d, l.handle())
    l.check(d)


def test_lora_small_capacity(ep):
    """Fewer rows than tokens, and blocks of several pieces that are mostly padding."""
    for seed, T, cap in ((67, 90, 3), (68, 300, 600)):
        l = Lora(ep, seed, T, 64, 96, 8, 4, none=0.0, expert_capacity=cap)
        d = l.buffers()
        l.run(d, l.handle())
        seen = [0] * 4
        for t, e in enumerate(l.ids):
            seen[e] += 1
            if seen[e] > cap:
                l.ids[t] = -1
        l.check(d)


def test_lora_capacity_drops(ep):
    """Tokens past an adapter's capacity have no row: they get the base alone."""
    l = Lora(ep, 61, 40, 64, 64, 8, 2, none=0.0, expert_capacity=12)
    d = l.buffers()
    l.run(d, l.handle())
    seen = {}
    for t, e in enumerate(l.ids):
        seen[e] = seen.get(e, 0) + 1
        if seen[e] > 12:
            l.ids[t] = -1
    l.check(d)


def test_lora_in_place_and_without_base(ep):
    l = Lora(ep, 62, 45, 64, 96, 16, 3)
    d, h = l.buffers(), l.handle()
    d["out"].copy_(d["base"])
    d["grad_x"].copy_(d["gb"])
    l.run(d, h, base=d["out"], gb=d["grad_x"])
    l.check(d)
    d = l.buffers()
    d["scale"] = None
    l.run(d, h, base=None, gb=None)
    l.check(d, base=False, scale=False)


def test_lora_masked_rows_hold_nan(ep):
    l = Lora(ep, 63, 50, 96, 64, 24, 3, none=0.3)
    l.ids[7] = 3                                             # out of range: dropped like -1
    off = (l.ids < 0) | (l.ids > 2)
    l.x[off], l.dy[off] = 0x7FC0, 0x7F80
    d = l.buffers()
    l.run(d, l.handle())
    l.x[off], l.dy[off] = 0, 0
    l.check(d)


def test_lora_nobody_has_an_adapter(ep):
    l = Lora(ep, 64, 20, 64, 64, 8, 2, none=1.1)
    d = l.buffers()
    l.run(d, l.handle())
    assert torch.equal(d["out"], d["base"]) and torch.equal(d["grad_x"], d["gb"])
    assert not d["grad_a"].any() and not d["grad_b"].any()


def test_lora_no_tokens(ep):
    l = Lora(ep, 65, 0, 64, 64, 8, 2, tmax=4)
    d = l.buffers()
    l.run(d, l.handle())
    assert not d["grad_a"].any() and not d["grad_b"].any()


def test_lora_same_bits_every_time(ep):
    l = Lora(ep, 66, 300, 256, 128, 16, 3)
    d, h = l.buffers(), l.handle()
    names = ("out", "grad_x", "grad_a", "grad_b")
    l.run(d, h)
    ref = {n: d[n].clone() for n in names}
    for rep in range(3):
        d["ws"].fill_(0x40 + rep)
        for n in names:
            d[n].fill_(float("nan"))
        l.run(d, h)
        for n in names:
            assert torch.equal(d[n], ref[n]), n


@pytest.mark.parametrize("layout", [dict(expert_capacity=70), dict(expert_capacity=600), dict(row_align=48),
                                    dict(row_align=1024)])
@pytest.mark.parametrize("r", [8, 128])
def test_lora_no_tokens_in_padded_layouts(ep, layout, r):
    """No tokens and blocks of padding all the same (also several pieces of them): the gradients are zeros, and no
    row is read (x, grad_out and down are empty, their pointers NULL)."""
    print(f"\n[case] lora without tokens {layout} rank {r}", flush=True)
    l = Lora(ep, 69, 0, 96, 64, r, 4, tmax=9, **layout)
    d = l.buffers()
    l.run(d, l.handle())
    assert not d["grad_a"].any() and not d["grad_b"].any()


def _check_nonfinite(l, d, under=0.0):
    """As Lora.check, but infinities and NaN have to stand where the definition (float64) has them; finite values
    are within their bounds (``under``: what float32's smallest number adds to grad_x)."""
    T, fin, fout, r, N = l.shape
    x, a, b = _f64(l.x), _f64(l.a), _f64(l.b)
    with np.errstate(all="ignore"):
        out, bound, down, dv = OY.lora(x, l.ids, a, b, l.scale.astype(np.float64), _f64(l.base))
        want = OY.lora_backward(x, l.ids, a, b, l.scale.astype(np.float64), _f64(l.dy), _f64(l.gb), down, dv)
        want["out"] = (out, bound)
        want["grad_x"] = (want["grad_x"][0], want["grad_x"][1] + under)
        for n, (v, lim) in want.items():
            got = d[n].double().cpu().numpy()
            fin = np.isfinite(v)
            assert np.array_equal(np.isnan(got), np.isnan(v)), f"{n}: NaN in the wrong places"
            assert np.array_equal(got[np.isinf(v)], v[np.isinf(v)]), f"{n}: infinities"
            assert np.all(np.abs(got - v)[fin] <= lim[fin]), n


INF_BF16 = 0x7F80


@pytest.mark.parametrize("where", ["a", "b", "x", "grad_out"])
@pytest.mark.parametrize("T,fin,fout,r,N", [
    (40, 64, 96, 8, 2), (33, 64, 160, 24, 2), (37, 96, 64, 40, 3), (90, 96, 64, 72, 2),
    # the down product in several shares
    (5, 2080, 1056, 40, 3), (4, 2080, 2080, 8, 2),
    # an adapter's gradient in several pieces
    (1100, 64, 32, 8, 2),
])
def test_lora_infinities(ep, where, T, fin, fout, r, N):
    """One infinity in A, B, x or grad_out: out and the gradients are infinite or NaN where the products of the
    definition are, and nowhere else (the last rank is the one that stands in for ranks that are filled up)."""
    print(f"\n[case] lora infinity in {where} {(T, fin, fout, r, N)}", flush=True)
    l = Lora(ep, 300 + r, T, fin, fout, r, N, none=0.0)
    l.ids[0] = 0
    l.a[l.a == 0], l.b[l.b == 0], l.x[l.x == 0], l.dy[l.dy == 0] = 0x3C00, 0x3C00, 0x3C00, 0x3C00   # inf * 0 by none
    if where == "a":
        l.a[0, r - 1, 3] = INF_BF16
    elif where == "b":
        l.b[0, fout - 5, r - 1] = INF_BF16 | 0x8000
    elif where == "x":
        l.x[0, fin - 2] = INF_BF16
    else:
        l.dy[0, 7] = INF_BF16
    d = l.buffers()
    l.run(d, l.handle())
    _check_nonfinite(l, d)


def test_lora_largest_floats(ep):
    """down values between the largest bf16 and the largest float32 are cut into parts like any other."""
    T, fin, fout, r, N = 40, 64, 96, 8, 2
    l = Lora(ep, 310, T, fin, fout, r, N, none=0.0)
    l.ids[:] = np.arange(T) % N
    l.scale[:] = 1.0
    l.a[:], l.b[:], l.x[:], l.dy[:], l.base[:], l.gb[:] = 0, 0, 0, 0, 0, 0
    # the largest bf16, 2^128 - 2^120, and three quarters of its step (bf16 rounds 2^128 - 2^118 to infinity)
    l.a[:, 2, 0], l.a[:, 2, 1], l.a[:, 2, 2] = 0x7F7F, 0x7B00, 0x7A80
    l.x[:, :3] = 0x3F80
    l.b[:, :, 2], l.b[:, 1::2, 2] = 0x0080, 0x8080           # +- 2^-126
    l.dy[:, 5] = 0x0080
    d = l.buffers()
    l.run(d, l.handle())
    assert float(d["down"].max()) > 3.397e38 and bool(torch.isfinite(d["down"]).all())
    # u = b dy is one product 2^-126 2^-126 a token, 0 in float32: grad_x = a u lacks up to 3 2^128 2^-252 < 2^-122
    _check_nonfinite(l, d, 2.0 ** -122)


@pytest.mark.parametrize("T,fin,fout,r,N", [(9000, 64, 96, 128, 2), (5000, 96, 64, 72, 2), (7001, 32, 160, 104, 5),
                                            (5200, 64, 64, 96, 3)])
def test_lora_several_pieces_at_high_ranks(ep, T, fin, fout, r, N):
    """Above 64 ranks an adapter's gradient is built from pieces of 32 r tokens: one adapter of several, others idle."""
    print(f"\n[case] lora pieces {(T, fin, fout, r, N)}", flush=True)
    l = Lora(ep, 330 + r, T, fin, fout, r, N, none=0.1, skew=True)
    d = l.buffers()
    l.run(d, l.handle())
    l.check(d)
