"""GPU few-token expert layer against the float64 oracle, within the rounding
bound that ``oracle/layer.py`` derives per element."""

import numpy as np
import pytest
import torch

from combine_topk_idx_amd import workloads as W
from oracle import codecs, layer as OY
from tests.hip_path import DEV, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    from combine_topk_idx_amd import ep as _ep
    return _ep


def _weights(g, quant, E, N, K):
    if quant == "none":
        return W.bf16_from_f32((g.normal(size=(E, N, K)) / np.sqrt(K)).astype(np.float32)), None
    base = 127 - int(round(np.log2(K) / 2))
    scales = g.integers(base - 2, base + 2, size=(E, N, K // 32)).astype(np.uint8)
    if quant == "mxfp4":
        return g.integers(0, 256, size=(E, N, K // 2)).astype(np.uint8), scales
    codes = g.integers(0, 256, size=(E, N, K)).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x30                      # no NaN
    codes[(codes & 0x78) > 0x40] &= 0xC7                      # magnitudes up to 3.75, subnormals among them
    return codes, scales


class Layer:
    def __init__(self, ep, seed, T, H, I, E, k, quant, idt=np.int64):
        g = np.random.default_rng(seed)
        self.ep, self.shape, self.quant = ep, (T, H, I, E, k), quant
        self.x = W.bf16_from_f32(g.normal(size=(T, H)).astype(np.float32))
        self.ids = g.integers(0, E, size=(T, k)).astype(idt)
        self.w = g.random((T, k)).astype(np.float32)
        self.w1, self.w2 = _weights(g, quant, E, 2 * I, H), _weights(g, quant, E, H, I)
        dev = lambda p: (to_dev(p[0]), None if p[1] is None else to_dev(p[1]))   # noqa: E731
        self.p1 = ep.pack_moe_weights(*dev(self.w1), True, quant=quant)
        self.p2 = ep.pack_moe_weights(*dev(self.w2), False, quant=quant)

    def workspace(self):
        T, H, I, E, k = self.shape
        ws = torch.empty(self.ep.ep_moe_layer_workspace_bytes(T, k, E, H, I), dtype=torch.uint8, device=DEV)
        return ws.fill_(0xA5)

    def run(self, ws=None, out=None, stream=None):
        T, H, I, E, k = self.shape
        ws = self.workspace() if ws is None else ws
        out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV) if out is None else out
        self.ep.ep_moe_layer(to_dev(self.x), to_dev(self.ids), to_dev(self.w), E, I, self.quant, *self.p1, *self.p2, ws,
                             out, stream=stream)
        return out

    def check(self, got):
        val = lambda p: OY.weight_values(p[0], p[1], self.quant)   # noqa: E731
        x = codecs.bf16_bits_to_f32(self.x).astype(np.float64)
        out, bound = OY.expert_layer(x, self.ids, self.w, val(self.w1), val(self.w2))
        err = np.abs(got.double().cpu().numpy() - out)
        assert np.all(err <= bound), f"worst error / bound {np.max(err / bound):.3g}"


CASES = [
    # T, H, I, E, k
    (1, 64, 64, 1, 1),
    (1, 512, 128, 8, 2),
    (3, 448, 192, 5, 3),            # odd step counts, a partial last block of groups
    (17, 128, 320, 16, 4),
    (40, 256, 64, 2, 2),            # more than 32 rows of an expert
    (128, 128, 64, 3, 16),          # 2048 pairs, repeated ids
    (2, 1088, 64, 512, 8),
    (13, 64, 1088, 40, 6),
    (64, 2048, 768, 16, 4),
]


@pytest.mark.parametrize("quant", ["none", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_layer(ep, i, quant):
    print(f"\n[case] layer {CASES[i]} {quant}", flush=True)
    l = Layer(ep, 10 * i, *CASES[i], quant, idt=np.int32 if i % 2 else np.int64)
    l.check(l.run())


@pytest.mark.parametrize("quant", ["none", "mxfp8", "mxfp4"])
def test_layer_masks(ep, quant):
    """Ids of -1 and out of range, a token and a whole call without an expert; x holds NaN where no id is valid."""
    l = Layer(ep, 5, 9, 192, 128, 6, 3, quant)
    l.ids[0] = [-1, 2, -1]
    l.ids[1] = -1
    l.ids[2] = [6, -9, 1 << 40]
    l.ids[3] = [4, 4, 4]
    l.x[1:3] = 0x7FC0
    got = l.run()
    assert not got[1:3].float().any()
    l.x[1:3] = 0
    l.check(got)
    l.ids[:] = -1
    assert not l.run().float().any()


@pytest.mark.parametrize("T,H,I,E,k", [(7, 192, 128, 6, 3), (8, 320, 64, 9, 11), (9, 320, 64, 9, 11), (10, 64, 128, 3, 2)])
def test_layer_masks_around_the_third_launch(ep, T, H, I, E, k):
    """Calls of up to 8 tokens sum their pairs in the second launch, larger ones in a third."""
    l = Layer(ep, 70 + T, T, H, I, E, k, "mxfp8")
    l.ids[0, 1:] = -1
    l.ids[1] = -1
    l.ids[2, 0] = E
    l.x[1] = 0x7FC0
    got = l.run()
    assert not got[1].float().any()
    l.x[1] = 0
    l.check(got)
    l.ids[:] = -1
    assert not l.run().float().any()


def test_layer_weight_codes(ep):
    """Every MXFP8 and MXFP4 code under every scale byte that keeps the product in bf16's normal range, one at a
    time through the down product: the output is the code's value exactly."""
    H = I = 64
    for quant, ncode in (("mxfp8", 256), ("mxfp4", 16)):
        E = 4                                                 # 4 experts x 64 rows of codes
        codes = np.zeros((E, H, I), np.uint8)
        flat = np.arange(E * H) % ncode
        flat[(flat & 0x7F) == 0x7F] = 0
        codes[:, :, 5] = flat.reshape(E, H)
        for sb in (20, 100, 126, 127, 128, 180):
            sc = np.full((E, H, I // 32), sb, np.uint8)
            w2 = codes if quant == "mxfp8" else (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
            # activation 5 is silu(g) u with g = 64 (silu = 64 to within 2^-60 of it), u = 1/64: 1; the others 0
            w1 = np.zeros((E, 2 * I, H), np.float32)
            w1[:, 5, 0], w1[:, I + 5, 1] = 64.0, 1.0 / 64
            from oracle import quant as OQ
            if quant == "mxfp8":
                w1c = np.zeros((E, 2 * I, H), np.uint8)
                w1s = np.full((E, 2 * I, H // 32), 127, np.uint8)
                w1c[:, 5, 0] = w1c[:, I + 5, 1] = 0x38        # 1.0
            else:
                w1c = np.zeros((E, 2 * I, H // 2), np.uint8)
                w1s = np.full((E, 2 * I, H // 32), 127, np.uint8)
                w1c[:, 5, 0], w1c[:, I + 5, 0] = 0x02, 0x20   # 1.0 at element 0, at element 1
            w1s[:, 5], w1s[:, I + 5] = 127 + 6, 127 - 6
            x = np.zeros((E, H), np.float32)
            x[:, :2] = 1.0
            p1 = ep.pack_moe_weights(to_dev(w1c), to_dev(w1s), True, quant=quant)
            p2 = ep.pack_moe_weights(to_dev(w2), to_dev(sc), False, quant=quant)
            out = torch.full((E, H), float("nan"), dtype=torch.bfloat16, device=DEV)
            ws = torch.empty(ep.ep_moe_layer_workspace_bytes(E, 1, E, H, I), dtype=torch.uint8, device=DEV)
            ep.ep_moe_layer(torch.from_numpy(x).bfloat16().to(DEV), torch.arange(E, device=DEV).view(E, 1),
                            torch.ones(E, 1, device=DEV), E, I, quant, *p1, *p2, ws, out)
            want = OY.weight_values(w2, sc, quant)[:, :, 5]
            assert np.array_equal(out.double().cpu().numpy(), want), (quant, sb)


def test_pack_ex_is_the_mxfp8_packing(ep):
    g = np.random.default_rng(1)
    codes, scales = _weights(g, "mxfp8", 3, 128, 320)
    for gate_up in (True, False):
        c, s = ep.pack_moe_weights(to_dev(codes), to_dev(scales), gate_up)
        c2, s2 = torch.empty_like(c), torch.empty_like(s)
        ep.ep_moe_pack_weights_ex(to_dev(codes), to_dev(scales), 3, 128, 320, "mxfp8", gate_up, c2, s2)
        assert torch.equal(c, c2) and torch.equal(s, s2)


def test_layer_repeats_and_streams(ep):
    """The same bits from every call, from calls on two streams at once, and over a workspace of garbage."""
    a, b = Layer(ep, 21, 16, 512, 256, 24, 4, "mxfp8"), Layer(ep, 22, 5, 256, 512, 12, 3, "none")
    ra, rb = a.run().clone(), b.run().clone()
    torch.cuda.synchronize()
    wa, wb = a.workspace(), b.workspace()
    oa, ob = torch.empty_like(ra), torch.empty_like(rb)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (sa, sb):
        s.wait_stream(torch.cuda.current_stream())
    keep = []
    for rep in range(4):
        for l, ws, out, s in ((a, wa, oa, sa), (b, wb, ob, sb)):
            with torch.cuda.stream(s):
                keep.append(l.run(ws, out))
        torch.cuda.synchronize()
        assert torch.equal(oa.view(torch.int16), ra.view(torch.int16))
        assert torch.equal(ob.view(torch.int16), rb.view(torch.int16))
        wa.fill_(0x5A + rep)
        oa.fill_(float("nan"))
        torch.cuda.synchronize()


def test_layer_no_tokens(ep):
    l = Layer(ep, 3, 1, 64, 64, 2, 1, "none")
    l.shape = (0, 64, 64, 2, 1)
    l.x, l.ids, l.w = l.x[:0], l.ids[:0], l.w[:0]
    assert l.run().shape == (0, 64)


@pytest.mark.parametrize("quant,ncode,bytes_", [("mxfp8", 256, range(10, 247)), ("mxfp4", 16, range(2, 252))])
def test_layer_every_scale_byte(ep, quant, ncode, bytes_):
    """Every code under every scale byte whose products all stay in bf16's normal range (smallest e4m3 2^-9, e2m1
    2^-1; largest 448 and 6), through the down product, where the other activations are zero: its value exactly."""
    H, I = 256, 64
    bytes_ = list(bytes_)
    E = len(bytes_)
    flat = np.arange(H) % ncode
    if quant == "mxfp8":
        flat[(flat & 0x7F) == 0x7F] = 0
    codes = np.zeros((E, H, I), np.uint8)
    codes[:, :, 37] = flat
    sc = np.broadcast_to(np.array(bytes_, np.uint8)[:, None, None], (E, H, I // 32)).copy()
    w2 = codes if quant == "mxfp8" else (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
    # activation 37 is silu(64) / 64 = 1 (to 2^-60 of it): gate 1.0 and up 1.0 under the scales 2^6 and 2^-6
    one = 0x38 if quant == "mxfp8" else 0x02
    w1 = np.zeros((E, 2 * I, H if quant == "mxfp8" else H // 2), np.uint8)
    w1[:, 37, 0] = w1[:, I + 37, 0] = one
    s1 = np.full((E, 2 * I, H // 32), 127, np.uint8)
    s1[:, 37], s1[:, I + 37] = 127 + 6, 127 - 6
    x = torch.zeros(E, H)
    x[:, 0] = 1.0
    p1 = ep.pack_moe_weights(to_dev(w1), to_dev(s1), True, quant=quant)
    p2 = ep.pack_moe_weights(to_dev(w2), to_dev(sc), False, quant=quant)
    out = torch.full((E, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(ep.ep_moe_layer_workspace_bytes(E, 1, E, H, I), dtype=torch.uint8, device=DEV)
    ep.ep_moe_layer(x.bfloat16().to(DEV), torch.arange(E, device=DEV).view(E, 1), torch.ones(E, 1, device=DEV), E, I,
                    quant, *p1, *p2, ws, out)
    want = OY.weight_values(w2, sc, quant)[:, :, 37]
    assert np.array_equal(out.double().cpu().numpy(), want)


@pytest.mark.parametrize("quant", ["none", "mxfp8", "mxfp4"])
def test_layer_wide(ep, quant):
    """The widest reduction axes of the measured sizes on few experts, and the odd group counts 64-wide blocks allow."""
    print(f"\n[case] layer wide {quant}", flush=True)
    for i, case in enumerate([(3, 7168, 192, 3, 2), (9, 320, 2112, 4, 2), (34, 1024, 4160, 2, 1)]):
        l = Layer(ep, 300 + i, *case, quant)
        l.check(l.run())


@pytest.mark.parametrize("quant", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("part", ["up", "down"])
def test_layer_nan_weights(ep, quant, part):
    """An e4m3 NaN code and an e8m0 NaN scale (0xFF) make NaN of the rows they stand in and of no other."""
    l = Layer(ep, 320, 3, 128, 128, 4, 2, quant)
    l.ids[:] = [[0, 1], [1, 2], [2, 3]]
    w, s = l.w2 if part == "down" else l.w1
    s[0, 3, 1] = 0xFF                                         # expert 0, row 3 (a gate row in the up product)
    if quant == "mxfp8":
        w[2, 40, 70] = 0xFF                                   # expert 2, row 40
    dev = lambda p: (to_dev(p[0]), to_dev(p[1]))              # noqa: E731
    l.p1, l.p2 = (ep.pack_moe_weights(*dev(p), up, quant=quant) for p, up in ((l.w1, True), (l.w2, False)))
    got = np.isnan(l.run().float().cpu().numpy())
    want = np.zeros(got.shape, bool)
    if part == "down":
        want[0, 3] = True
        want[1:, 40] = quant == "mxfp8"
    else:                                                     # a NaN activation reaches every output of its tokens
        want[0] = True
        want[1:] = quant == "mxfp8"
    assert np.array_equal(got, want)
