"""Router, few-token expert layer and adapters as one step uses them: eagerly
and as a captured graph, against each other and against the chain of layout,
dispatch, expert GEMMs and combine."""

import numpy as np
import pytest
import torch

from combine_topk_idx_amd import workloads as W
from tests.hip_path import DEV, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    from combine_topk_idx_amd import ep as _ep
    return _ep


class Step:
    """logits -> ids and weights -> expert layer -> adapters on top, and the backward of router and adapters."""

    def __init__(self, ep, T=24, H=512, I=256, E=32, k=4, r=16, N=5):
        self.ep, self.dims = ep, (T, H, I, E, k, r, N)
        g = torch.Generator(device=DEV).manual_seed(9)
        rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)   # noqa: E731
        new = lambda *s, d=torch.float32: torch.full(s, 7, dtype=d, device=DEV)   # noqa: E731
        bf = torch.bfloat16
        self.x, self.logits, self.bias = rnd(T, H).to(bf), rnd(T, E), rnd(E) * 0.1
        w1, s1 = W.make_mx_weights(3, E, 2 * I, H)
        w2, s2 = W.make_mx_weights(4, E, H, I)
        self.p1 = ep.pack_moe_weights(to_dev(w1), to_dev(s1), True)
        self.p2 = ep.pack_moe_weights(to_dev(w2), to_dev(s2), False)
        self.a, self.b = (rnd(N, r, H) * H ** -0.5).to(bf), (rnd(N, H, r) * 0.2).to(bf)
        self.ids = torch.randint(-1, N, (T, 1), generator=g, device=DEV)
        self.idx, self.w = new(T, k, d=torch.int64), new(T, k)
        self.out, self.down = new(T, H, d=bf), new(T, r)
        self.dy, self.gw = rnd(T, H).to(bf), rnd(T, k)
        self.grads = [new(T, H, d=bf), new(N, r, H), new(N, H, r), new(T, E)]
        self.lws = new(ep.ep_workspace_bytes(T, 1, N), d=torch.uint8)
        self.rc = new(N, d=torch.int64)
        self.ws = new(ep.ep_moe_layer_workspace_bytes(T, k, E, H, I), d=torch.uint8)
        self.ows = new(ep.ep_lora_workspace_bytes(T, H, H, r, N, True), d=torch.uint8)

    def __call__(self):
        ep, (T, H, I, E, k, r, N) = self.ep, self.dims
        kw = dict(score="sigmoid", renormalize=True, scale=2.0)
        ep.ep_router(self.logits, self.idx, self.w, bias=self.bias, num_groups=4, topk_groups=2, group_top=2, **kw)
        ep.ep_moe_layer(self.x, self.idx, self.w, E, I, "mxfp8", *self.p1, *self.p2, self.ws, self.out)
        h = ep.ep_layout(self.ids, N, T, self.rc, self.lws)
        ep.ep_lora(h, self.x, self.a, self.b, self.out, self.down, self.ows, base=self.out)
        ep.ep_lora_backward(h, self.dy, self.x, self.a, self.b, self.down, *self.grads[:3], self.ows)
        ep.ep_router_backward(self.logits, self.idx, self.gw, self.grads[3], **kw)

    def results(self):
        return [self.idx, self.w, self.out, *self.grads]


def test_graph_replays_match_eager(ep):
    s, other = Step(ep), Step(ep, T=7, H=256, I=128, E=16, k=2, r=8, N=3)
    s()
    torch.cuda.synchronize()
    ref = [t.clone() for t in s.results()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s()
    torch.cuda.synchronize()
    for rep in range(4):
        for t in s.results():
            t.fill_(3)
        for w in (s.ws, s.ows, s.lws):
            w.fill_(0x5A + rep)
        other()                                              # unrelated eager work in between
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (t, r) in enumerate(zip(s.results(), ref)):
            assert torch.equal(t, r), f"replay {rep}, result {i}"
    # new inputs in the captured buffers
    s.logits.copy_(torch.randn_like(s.logits))
    s.x.copy_(torch.randn_like(s.x))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in s.results()]
    s()
    torch.cuda.synchronize()
    for i, (t, r) in enumerate(zip(got, s.results())):
        assert torch.equal(t, r), i


def test_layer_against_the_separate_calls(ep):
    """The layer and the chain dispatch (MXFP8) -> GMM1 -> GMM2 -> combine on the same packed weights differ by
    the chain's quantisation of x and of the activations: under 2^-3 of the row in norm (e4m3 is off by at most
    2^-4 of a value, and two quantisations and the rest stay below twice that)."""
    s = Step(ep)
    T, H, I, E, k, r, N = s.dims
    ep.ep_router(s.logits, s.idx, s.w)
    ep.ep_moe_layer(s.x, s.idx, s.w, E, I, "mxfp8", *s.p1, *s.p2, s.ws, s.out)
    u8 = lambda n: torch.empty(n, dtype=torch.uint8, device=DEV)   # noqa: E731
    rc = torch.empty(E, dtype=torch.int64, device=DEV)
    lws = u8(ep.ep_workspace_bytes(T, k, E))
    xb, ab = u8(ep.ep_buffer_bytes(T * k, H, "mxfp8")[0]), u8(ep.ep_buffer_bytes(T * k, I, "mxfp8")[0])
    h = ep.ep_layout_dispatch(s.idx, E, T, rc, lws, s.x, H, "mxfp8", xb)
    ep.ep_moe_gmm1(h, xb, H, I, *s.p1, "mxfp8", ab, recv_count=rc)
    yb, out = u8(T * k * H * 2), torch.empty_like(s.out)
    ep.ep_moe_gmm2(h, ab, I, H, *s.p2, yb, recv_count=rc)
    ep.ep_combine(h, yb, "none", H, s.idx, s.w, out)
    rel = (out.float() - s.out.float()).norm(dim=1) / s.out.float().norm(dim=1)
    assert float(rel.max()) < 0.125


def test_small_calls_in_graphs(ep):
    """The forms for a few tokens captured: the layer whose second launch sums the pairs, the adapters' down product
    in several shares; two graphs over workspaces of their own, replayed in turn with eager work between."""
    steps = [Step(ep, T=3, H=2048, I=128, E=24, k=4, r=8, N=3), Step(ep, T=8, H=1152, I=192, E=12, k=2, r=40, N=2)]
    other = Step(ep, T=40, H=512, I=256, E=8, k=2)
    refs, graphs = [], []
    for s in steps:
        s()
        torch.cuda.synchronize()
        refs.append([t.clone() for t in s.results()])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s()
        graphs.append(g)
    for rep in range(4):
        for s in steps:
            for t in s.results():
                t.fill_(3)
            for w in (s.ws, s.ows, s.lws):
                w.fill_(0xA5 - rep)
        for g in graphs:
            g.replay()
            other()
        torch.cuda.synchronize()
        for s, ref in zip(steps, refs):
            for i, (t, r) in enumerate(zip(s.results(), ref)):
                assert torch.equal(t, r), f"replay {rep}, {s.dims}, result {i}"


def test_one_workspace_for_calls_of_every_size(ep):
    """Layer calls of few and of more tokens, and of other shapes, one after the other over one workspace that
    nobody clears: each call's rows are its own."""
    g = torch.Generator(device=DEV).manual_seed(3)
    H, I, E, k = 1024, 256, 16, 4
    w1, s1 = W.make_mx_weights(5, E, 2 * I, H)
    w2, s2 = W.make_mx_weights(6, E, H, I)
    p = ep.pack_moe_weights(to_dev(w1), to_dev(s1), True) + ep.pack_moe_weights(to_dev(w2), to_dev(s2), False)
    u8 = lambda T: torch.zeros(ep.ep_moe_layer_workspace_bytes(T, k, E, H, I), dtype=torch.uint8, device=DEV)   # noqa: E731
    shared = u8(64)
    for rep in range(3):
        for T in (6, 40, 1, 64, 8, 9, 3):
            x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
            idx = torch.randint(-1, E, (T, k), generator=g, device=DEV)
            w = torch.rand(T, k, generator=g, device=DEV)
            outs = [torch.full((T, H), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
            for ws, out in zip((shared, u8(T)), outs):
                ep.ep_moe_layer(x, idx, w, E, I, "mxfp8", *p, ws, out)
            assert torch.equal(*outs), (rep, T)
            assert bool(outs[0].float().abs().sum() > 0)
