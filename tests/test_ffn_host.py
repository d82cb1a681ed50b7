"""Host-side refusals of the feed-forward block and the block-scaled product
(no GPU needed): every rule returns its code before anything is launched."""

import ctypes

import pytest
import torch

FAKE = 1 << 40          # 256-byte aligned, never dereferenced on the host
GAP = 1 << 32


@pytest.fixture(scope="module")
def ep():
    from combine_topk_idx_amd import ep as _ep
    return _ep


def _handle(ep, T=4, tmax=4, k=2, E=3, align=1, cap=0, **kw):
    h = ep.ep_handle_t()
    h.num_tokens, h.num_max_tokens, h.num_topk, h.num_experts = T, tmax, k, E
    h.row_align, h.expert_capacity = align, cap
    h.max_rows = ep.ep_layout_rows(tmax, k, E, align, cap)
    h.offsets = h.slot = h.row_src = h.status = FAKE
    for n, v in kw.items():
        setattr(h, n, v)
    return h


def _ffn(ep, backward, hargs=None, **kw):
    H, I = kw.get("H", 128), kw.get("I", 128)
    a = dict(count=FAKE, x=FAKE, xb=1 << 30, H=H, I=I, act=0, w1=FAKE + GAP, w2=FAKE + 2 * GAP, q=0, ck=FAKE + 3 * GAP,
             ckb=1 << 30, ws=FAKE + 4 * GAP, wsb=1 << 30, out=FAKE + 5 * GAP, ob=1 << 30, dy=FAKE + 6 * GAP, dyb=1 << 30,
             gw1=FAKE + 7 * GAP, gw2=FAKE + 8 * GAP)
    a.update(kw)
    h = _handle(ep, **(hargs or {}))
    hp = ctypes.byref(h) if a.get("handle", True) else None
    if backward:
        return ep._lib.ep_ffn_backward(hp, a["count"], a["dy"], a["dyb"], a["x"], a["xb"], a["H"], a["I"], a["act"], a["w1"],
                                       a["w2"], a["q"], a["ck"], a["ckb"], a["ws"], a["wsb"], a["out"], a["ob"], a["gw1"],
                                       a["gw2"], None)
    return ep._lib.ep_ffn(hp, a["count"], a["x"], a["xb"], a["H"], a["I"], a["act"], a["w1"], a["w2"], a["q"], a["ck"],
                          a["ckb"], a["ws"], a["wsb"], a["out"], a["ob"], None)


ROWS = 8 * 128 * 2       # bytes of the 8 rows of the default handle
BOTH_BAD = [
    (dict(handle=False), 1), (dict(H=0), 1), (dict(H=96), 1), (dict(H=-64), 1), (dict(I=0), 1), (dict(I=32), 1),
    (dict(H=65536 + 64), 2), (dict(I=65536 + 64), 2), (dict(act=-1), 1), (dict(act=2), 1), (dict(q=1), 1), (dict(q=3), 1),
    (dict(q=5), 1), (dict(q=6), 1), (dict(q=0x102), 1), (dict(q=2, I=64), 1), (dict(count=FAKE + 4), 1), (dict(w1=None), 1),
    (dict(w1=FAKE + GAP + 8), 1), (dict(w2=None), 1), (dict(w2=FAKE + 2), 1), (dict(ws=None), 1),
    (dict(ws=FAKE + 16), 1), (dict(wsb=100), 3), (dict(ck=FAKE + 3 * GAP + 4), 1), (dict(ckb=4095), 3),
    (dict(q=2, ckb=2048), 3), (dict(x=None), 1), (dict(x=FAKE + 8), 1), (dict(xb=ROWS - 1), 3), (dict(out=None), 1),
    (dict(out=FAKE + 5 * GAP + 2), 1), (dict(ob=ROWS - 1), 3), (dict(out=FAKE), 1), (dict(out=FAKE + ROWS - 16), 1),
    (dict(hargs=dict(E=513)), 1), (dict(hargs=dict(k=17)), 1), (dict(hargs=dict(max_rows=9)), 1),
    (dict(hargs=dict(align=16), count=None), 1), (dict(hargs=dict(cap=8), count=None), 1),
    (dict(hargs=dict(offsets=None)), 1), (dict(hargs=dict(T=1 << 30, tmax=1 << 30, k=1), H=65536), 2),
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("i", range(len(BOTH_BAD)))
def test_ffn_rejects(ep, i, backward):
    kw, code = BOTH_BAD[i]
    assert _ffn(ep, backward, **kw) == code
    assert ep.ep_last_error().startswith("ep_ffn_backward:" if backward else "ep_ffn:")


def test_ffn_checkpoint_overlap(ep):
    for ck in (FAKE, FAKE + 5 * GAP):
        assert _ffn(ep, False, ck=ck) == 1
        assert "checkpoint overlaps" in ep.ep_last_error()


@pytest.mark.parametrize("kw", [dict(ck=None), dict(dy=None), dict(dy=FAKE + 2), dict(dyb=ROWS - 1), dict(gw1=None),
                                dict(gw1=FAKE + 8), dict(gw2=None), dict(gw2=FAKE + 2), dict(out=FAKE + 6 * GAP),
                                dict(wsb=8 * 128 * 2)])
def test_ffn_backward_rejects(ep, kw):
    assert _ffn(ep, True, **kw) in (1, 3)
    assert ep.ep_last_error().startswith("ep_ffn_backward:")


def test_ffn_of_no_rows_is_fine(ep):
    """An empty capacity: nothing is launched, the row buffers may be NULL."""
    assert _ffn(ep, False, hargs=dict(T=0, tmax=0), x=None, out=None, ck=None) == 0


def test_ffn_workspace_bytes(ep):
    f = ep.ep_ffn_workspace_bytes
    assert f(8, 128, 128, 3) == 2048 and f(8, 128, 128, 3, True) == 2048 + 4096
    assert f(9, 64, 64, 3) == 1280                      # 9 * 128 = 1152, rounded up to 256
    assert f(0, 64, 64, 1) > 0
    for bad in ((-1, 64, 64, 1), (1 << 31, 64, 64, 1), (8, 96, 64, 1), (8, 64, 96, 1), (8, 0, 64, 1), (8, 64, 0, 1),
                (8, 65600, 64, 1), (8, 64, 65600, 1), (8, 64, 64, 0), (8, 64, 64, 513)):
        assert f(*bad) == 0


def _gmm(ep, hargs=None, **kw):
    a = dict(count=FAKE, a=FAKE, ab=1 << 30, aq=2, k=256, n=256, w=FAKE + GAP, ws=FAKE + 2 * GAP, tr=0, act=-1, oq=0,
             out=FAKE + 3 * GAP, ob=1 << 30)
    a.update(kw)
    h = _handle(ep, **(hargs or {}))
    return ep._lib.ep_moe_gmm_b128(ctypes.byref(h) if a.get("handle", True) else None, a["count"], a["a"], a["ab"],
                                   a["aq"], a["k"], a["n"], a["w"], a["ws"], a["tr"], a["act"], a["oq"], a["out"], a["ob"],
                                   None)


GMM_BAD = [
    (dict(handle=False), 1), (dict(aq=0), 1), (dict(aq=3), 1), (dict(aq=0x102), 1), (dict(aq=7), 1), (dict(k=0), 1),
    (dict(k=64), 1), (dict(n=0), 1), (dict(n=192), 1), (dict(n=128, act=0), 1), (dict(k=65536 + 128), 2),
    (dict(n=65536 + 128), 2), (dict(tr=2), 1), (dict(tr=1, act=0), 1), (dict(act=2), 1), (dict(act=-2), 1),
    (dict(oq=2), 1), (dict(oq=1, act=0), 1), (dict(oq=3, act=0), 1), (dict(oq=0x102, act=0), 1), (dict(w=None), 1),
    (dict(w=FAKE + 8), 1), (dict(ws=None), 1), (dict(ws=FAKE + 2), 1), (dict(a=None), 1), (dict(a=FAKE + 8), 1),
    (dict(out=None), 1), (dict(out=FAKE + 3 * GAP + 8), 1), (dict(ab=8 * 256 + 63), 3), (dict(ob=8 * 512 - 1), 3),
    (dict(ob=8 * 256 - 1, act=0), 3), (dict(ob=8 * 128 + 31, act=1, oq=2), 3), (dict(out=FAKE), 1),
    (dict(out=FAKE + 1024), 1), (dict(count=FAKE + 4), 1), (dict(hargs=dict(align=16), count=None), 1),
    (dict(hargs=dict(cap=4), count=None), 1), (dict(hargs=dict(E=0)), 1),
    (dict(hargs=dict(T=1 << 30, tmax=1 << 30, k=1), n=65536), 2),
]


@pytest.mark.parametrize("i", range(len(GMM_BAD)))
def test_gmm_rejects(ep, i):
    kw, code = GMM_BAD[i]
    assert _gmm(ep, **kw) == code
    assert ep.ep_last_error().startswith("ep_moe_gmm_b128:")


def test_gmm_of_no_rows_is_fine(ep):
    assert _gmm(ep, hargs=dict(T=0, tmax=0), a=None, out=None) == 0


# ---------------------------------------------------------------------------
# the binding's own checks (CPU tensors: valid ones end at "must be a GPU tensor")
# ---------------------------------------------------------------------------

E, H, I, R = 3, 128, 128, 8
BF = torch.bfloat16


def _tensors():
    z = torch.zeros
    return dict(x=z(R, H, dtype=BF), w1=z(E, 2 * I, H, dtype=BF), w2=z(E, H, I, dtype=BF), ws=z(1 << 16, dtype=torch.uint8),
                out=z(R, H, dtype=BF), ck=z(1 << 13, dtype=torch.uint8), dy=z(R, H, dtype=BF), gx=z(R, H, dtype=BF),
                gw1=z(E, 2 * I, H, dtype=BF), gw2=z(E, H, I, dtype=BF), count=z(E, dtype=torch.int64))


BINDING_BAD = [("x", dict(x=torch.zeros(R, H))), ("x", dict(x=torch.zeros(R - 1, H, dtype=BF))),
               ("w1", dict(w1=torch.zeros(E, I, H, dtype=BF))), ("w1", dict(w1=torch.zeros(E, 2 * I, H))),
               ("w2", dict(w2=torch.zeros(E + 1, H, I, dtype=BF))), ("w1 and w2", dict(w2=torch.zeros(H, I, dtype=BF))),
               ("recv_count", dict(count=torch.zeros(E, dtype=torch.int32))),
               ("recv_count", dict(count=torch.zeros(E - 1, dtype=torch.int64))),
               ("contiguous", dict(w1=torch.zeros(E, H, 2 * I, dtype=BF).transpose(1, 2)))]


@pytest.mark.parametrize("i", range(len(BINDING_BAD)))
@pytest.mark.parametrize("backward", [False, True])
def test_binding_rejects(ep, i, backward):
    word, kw = BINDING_BAD[i]
    t = _tensors()
    t.update(kw)
    with pytest.raises(ep.EpError, match=word):
        if backward:
            ep.ep_ffn_backward(_handle(ep), t["dy"], t["x"], t["w1"], t["w2"], t["ck"], t["ws"], t["gx"], t["gw1"],
                               t["gw2"], recv_count=t["count"])
        else:
            ep.ep_ffn(_handle(ep), t["x"], t["w1"], t["w2"], t["ws"], t["out"], recv_count=t["count"], checkpoint=t["ck"])


def test_binding_wants_the_gpu_and_known_names(ep):
    t = _tensors()
    with pytest.raises(ep.EpError, match="GPU tensor"):
        ep.ep_ffn(_handle(ep), t["x"], t["w1"], t["w2"], t["ws"], t["out"])
    with pytest.raises(ep.EpError, match="unknown act"):
        ep.ep_moe_gmm_b128(_handle(ep), t["ck"], "fp8_b128", 128, 256, t["ck"], t["ck"], t["out"], act="relu")
    u8 = torch.uint8
    w, s = torch.zeros(E, 256, 128, dtype=u8), torch.zeros(E, 2, 1)
    for name, kw in (("w must", dict(w=torch.zeros(E, 256, 128))), ("w must have", dict(w=torch.zeros(E, 128, 256, dtype=u8))),
                     ("w_scales", dict(s=torch.zeros(E, 1, 2))), ("w_scales", dict(s=s.double())),
                     ("out", dict(out=torch.zeros(R, 255, dtype=BF))), ("out", dict(out=torch.zeros(R, 256)))):
        a = dict(w=w, s=s, out=torch.zeros(R, 256, dtype=BF))
        a.update(kw)
        with pytest.raises(ep.EpError, match=name):
            ep.ep_moe_gmm_b128(_handle(ep), t["ck"], "fp8_b128", 128, 256, a["w"], a["s"], a["out"])
