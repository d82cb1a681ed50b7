"""Host-side refusals of the router, the few-token expert layer and the
low-rank adapters (no GPU needed): every rule returns its code before
anything is launched."""

import ctypes

import pytest
import torch

FAKE = 1 << 40          # 256-byte aligned, never dereferenced on the host


@pytest.fixture(scope="module")
def ep():
    from combine_topk_idx_amd import ep as _ep
    return _ep


def _router(ep, z=FAKE, dtype=0, T=4, E=16, k=2, score=0, bias=None, groups=4, keep=2, top=2, renorm=1, idx=FAKE,
            idx_dtype=1, w=FAKE):
    return ep._lib.ep_router(z, dtype, T, E, k, score, bias, groups, keep, top, renorm, 1.0, idx, idx_dtype, w, None)


ROUTER_BAD = [dict(z=None), dict(z=FAKE + 2), dict(dtype=1, z=FAKE + 1), dict(dtype=3), dict(dtype=-1), dict(T=-1),
              dict(T=1 << 31), dict(E=0), dict(E=513), dict(k=0), dict(k=17), dict(E=4, k=5, groups=1, keep=1),
              dict(score=2), dict(bias=FAKE + 2), dict(groups=3), dict(groups=0), dict(E=512, groups=128),
              dict(keep=0), dict(keep=5), dict(top=0), dict(top=3), dict(groups=16, keep=1, top=2), dict(renorm=2),
              dict(idx=None), dict(idx=FAKE + 4), dict(idx_dtype=2), dict(w=None), dict(w=FAKE + 2)]


@pytest.mark.parametrize("kw", ROUTER_BAD)
def test_router_rejects(ep, kw):
    assert _router(ep, **kw) == ep.EP_ERR_INVALID_ARG
    assert ep.ep_last_error().startswith("ep_router:")


def test_router_of_no_tokens_is_fine(ep):
    assert _router(ep, T=0, z=None, idx=None, w=None) == 0


@pytest.mark.parametrize("kw", [dict(z=None), dict(dtype=5), dict(k=17), dict(score=-1), dict(renorm=-1),
                                dict(idx=FAKE + 4), dict(grad=None), dict(grad=FAKE + 1), dict(dz=None),
                                dict(dz=FAKE + 2), dict(dz=FAKE + 64), dict(dz=FAKE - 64)])
def test_router_backward_rejects(ep, kw):
    a = dict(z=FAKE, dtype=0, T=4, E=16, k=2, score=0, renorm=1, idx=FAKE, grad=FAKE, dz=FAKE)
    a.update(kw)
    rc = ep._lib.ep_router_backward(a["z"], a["dtype"], a["T"], a["E"], a["k"], a["score"], a["renorm"], 1.0, a["idx"],
                                    1, a["grad"], a["dz"], None)
    assert rc == ep.EP_ERR_INVALID_ARG
    assert ep.ep_last_error().startswith("ep_router_backward:")


LAYER_BAD = [(dict(k=0), 1), (dict(k=17), 1), (dict(E=0), 1), (dict(E=513), 1), (dict(T=-1), 1), (dict(T=1025), 2),
             (dict(T=129, k=16), 2), (dict(H=0), 1), (dict(H=96), 1), (dict(I=32), 1), (dict(H=65536 + 64), 2),
             (dict(idx_dtype=2), 1), (dict(q=1), 1), (dict(q=2), 1), (dict(q=0x103), 1), (dict(idx=None), 1),
             (dict(idx=FAKE + 4), 1), (dict(w=None), 1), (dict(x=None), 1), (dict(x=FAKE + 8), 1), (dict(out=None), 1),
             (dict(out=FAKE + 1024), 1), (dict(w1=None), 1), (dict(w2=FAKE + 4), 1), (dict(s1=None), 1),
             (dict(s2=FAKE + 4), 1), (dict(ws=None), 1), (dict(ws=FAKE + 16), 1), (dict(wsb=100), 3)]


@pytest.mark.parametrize("kw,code", LAYER_BAD)
def test_layer_rejects(ep, kw, code):
    a = dict(x=FAKE, T=4, H=256, idx=FAKE, idx_dtype=1, w=FAKE, k=2, E=8, I=128, q=3, w1=FAKE, s1=FAKE, w2=FAKE,
             s2=FAKE, ws=FAKE, wsb=1 << 30, out=FAKE * 2)
    a.update(kw)
    rc = ep._lib.ep_moe_layer(a["x"], a["T"], a["H"], a["idx"], a["idx_dtype"], a["w"], a["k"], a["E"], a["I"], a["q"],
                              a["w1"], a["s1"], a["w2"], a["s2"], a["ws"], a["wsb"], a["out"], None)
    assert rc == code, ep.ep_last_error()
    assert ep.ep_last_error().startswith("ep_moe_layer:")


def test_layer_sizes(ep):
    assert ep.ep_moe_layer_workspace_bytes(0, 8, 256, 7168, 2048) > 0
    one, many = (ep.ep_moe_layer_workspace_bytes(T, 8, 256, 7168, 2048) for T in (1, 256))
    assert many >= 256 * 8 * (2048 * 2 + 7168 * 4) and one < many
    for bad in ((257, 8, 256, 7168, 2048), (1, 0, 1, 64, 64), (1, 1, 513, 64, 64), (1, 1, 1, 96, 64), (-1, 1, 1, 64, 64)):
        assert ep.ep_moe_layer_workspace_bytes(*bad) == 0
    n = 6 * 512 * 256
    scales = ep.ep_moe_packed_bytes(6, 512, 256)[1]
    assert ep.ep_moe_packed_bytes_ex(6, 512, 256, "mxfp8") == ep.ep_moe_packed_bytes(6, 512, 256) == (n, scales)
    assert ep.ep_moe_packed_bytes_ex(6, 512, 256, "none") == (2 * n, 0)
    assert ep.ep_moe_packed_bytes_ex(6, 512, 256, "mxfp4") == (n // 2, scales)
    for bad in ((0, 32, 64, 3), (1, 48, 64, 3), (1, 32, 96, 3), (1, 32, 64, 1), (1, 32, 64, 7)):
        with pytest.raises(ep.EpError):
            ep.ep_moe_packed_bytes_ex(*bad)


@pytest.mark.parametrize("kw,code", [(dict(E=0), 1), (dict(N=48), 1), (dict(K=96), 1), (dict(q=1), 1), (dict(gu=2), 1),
                                     (dict(N=32, gu=1), 1), (dict(w=None), 1), (dict(pw=FAKE + 8), 1),
                                     (dict(s=None), 1), (dict(ps=None), 1)])
def test_pack_ex_rejects(ep, kw, code):
    a = dict(w=FAKE, s=FAKE, E=2, N=64, K=128, q=4, gu=0, pw=FAKE, ps=FAKE)
    a.update(kw)
    rc = ep._lib.ep_moe_pack_weights_ex(a["w"], a["s"], a["E"], a["N"], a["K"], a["q"], a["gu"], a["pw"], a["ps"], None)
    assert rc == code
    assert ep.ep_last_error().startswith("ep_moe_pack_weights_ex:")


def _handle(ep, T=4, k=1, N=8):
    h = ep.ep_handle_t()
    h.num_tokens, h.num_max_tokens, h.max_rows = T, 8, 8 * k
    h.num_topk, h.num_experts, h.row_align = k, N, 1
    h.offsets = h.slot = h.row_src = h.status = FAKE
    return h


LORA_BAD = [(dict(h=None), 1), (dict(k=2), 1), (dict(fin=48), 1), (dict(fout=0), 1), (dict(fin=65536 + 32), 2),
            (dict(r=4), 1), (dict(r=12), 1), (dict(r=136), 1), (dict(a=None), 1), (dict(b=FAKE + 2), 1),
            (dict(scale=FAKE + 2), 1), (dict(x=None), 1), (dict(x=FAKE + 8), 1), (dict(out=None), 1),
            (dict(base=FAKE + 2), 1), (dict(down=None), 1), (dict(down=FAKE + 4), 1), (dict(out=FAKE + 64), 1),
            (dict(base=2 * FAKE + 64), 1), (dict(ws=None), 1), (dict(ws=FAKE + 64), 1), (dict(wsb=64), 3)]


def _lora_args(ep, kw):
    a = dict(k=1, x=FAKE, fin=64, fout=96, r=16, a=FAKE, b=FAKE, scale=None, base=None, out=2 * FAKE, down=FAKE, ws=FAKE,
             wsb=1 << 30)
    a.update(kw)
    h = None if "h" in kw else ctypes.byref(_handle(ep, k=a["k"]))
    return h, a


@pytest.mark.parametrize("kw,code", LORA_BAD)
def test_lora_rejects(ep, kw, code):
    h, a = _lora_args(ep, kw)
    rc = ep._lib.ep_lora(h, a["x"], a["fin"], a["fout"], a["r"], a["a"], a["b"], a["scale"], a["base"], a["out"],
                         a["down"], a["ws"], a["wsb"], None)
    assert rc == code, ep.ep_last_error()
    assert ep.ep_last_error().startswith("ep_lora:")


@pytest.mark.parametrize("kw,code", [*LORA_BAD[:11], (dict(x=None), 1), (dict(dy=None), 1), (dict(down=None), 1),
                                     (dict(dx=None), 1), (dict(dx=FAKE), 1), (dict(base=2 * FAKE + 64), 1),
                                     (dict(da=None), 1), (dict(db=FAKE + 4), 1), (dict(ws=None), 1), (dict(wsb=64), 3)])
def test_lora_backward_rejects(ep, kw, code):
    h, a = _lora_args(ep, kw)
    dy, dx = kw.get("dy", FAKE), kw.get("dx", 2 * FAKE)
    rc = ep._lib.ep_lora_backward(h, dy, a["x"], a["fin"], a["fout"], a["r"], a["a"], a["b"], a["scale"], a["down"],
                                  a["base"], dx, kw.get("da", FAKE), kw.get("db", FAKE), a["ws"], a["wsb"], None)
    assert rc == code, ep.ep_last_error()
    assert ep.ep_last_error().startswith("ep_lora_backward:")


def test_lora_workspace_bytes(ep):
    fwd, bwd = (ep.ep_lora_workspace_bytes(128, 7168, 2048, 16, 8, b) for b in (False, True))
    assert 128 * 16 * 4 <= fwd < bwd
    for bad in ((-1, 64, 64, 8, 1), (1, 48, 64, 8, 1), (1, 64, 0, 8, 1), (1, 64, 64, 12, 1), (1, 64, 64, 136, 1),
                (1, 64, 64, 8, 513)):
        assert ep.ep_lora_workspace_bytes(*bad) == 0


# the binding: dtypes, shapes, density and device are checked before the library sees a pointer


def test_binding_rejects(ep):
    def bad(match, fn, *a, **kw):
        with pytest.raises(ep.EpError, match=match):
            fn(*a, **kw)

    z, idx, w = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)
    bad("must be a GPU tensor", ep.ep_router, z, idx, w)
    bad("logits must be", ep.ep_router, z.double(), idx, w)
    bad("logits must be contiguous", ep.ep_router, torch.zeros(16, 4).t(), idx, w)
    bad("topk_idx must have 4 rows", ep.ep_router, z, idx[:3], w)
    bad("topk_weights must have shape", ep.ep_router, z, idx, w[:, :1].contiguous())
    bad("bias must have shape", ep.ep_router, z, idx, w, bias=torch.zeros(8))
    bad("grad_logits must be", ep.ep_router_backward, z, idx, w, z.bfloat16())
    bad("unknown quant|KeyError|must be", ep.ep_moe_layer, torch.zeros(4, 96), idx, w, 8, 64, "mxfp8", None, None, None,
        None, torch.zeros(1), z)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)          # noqa: E731
    (b1, s1), (b2, s2) = (ep.ep_moe_packed_bytes_ex(8, n, 64, "mxfp8") for n in (128, 64))
    ok = [x, idx, w, 8, 64, "mxfp8", u8(b1), u8(s1), u8(b2), u8(s2), u8(1 << 20), torch.zeros_like(x)]
    bad("must be a GPU tensor", ep.ep_moe_layer, *ok)
    for i, t, match in [(0, x.float(), "x must be"), (6, u8(b1 - 1), "w1 must have shape"),
                        (9, u8(s2 + 1), "w2_scales must have shape"), (11, torch.zeros(4, 64), "out must be"),
                        (2, w.double(), "topk_weights must be")]:
        bad(match, ep.ep_moe_layer, *ok[:i], t, *ok[i + 1:])
    h = _handle(ep)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)     # noqa: E731
    ok = [h, bf(4, 64), bf(8, 16, 64), bf(8, 96, 16), bf(4, 96), torch.zeros(4, 16), u8(1 << 16)]
    bad("must be a GPU tensor", ep.ep_lora, *ok)
    for i, t, match in [(1, bf(3, 64), "x must have shape"), (2, bf(7, 16, 64), "holds 7 adapters"),
                        (3, bf(8, 96, 8), "b must have shape"), (5, bf(4, 16), "down must be")]:
        bad(match, ep.ep_lora, *ok[:i], t, *ok[i + 1:])
    bad("scale must have shape", ep.ep_lora, *ok, scale=torch.zeros(3))
    bad("base must be", ep.ep_lora, *ok, base=torch.zeros(4, 96))


@pytest.mark.parametrize("N,cap,fin,fout,r", [
    (512, 4194303, 65536, 65536, 128),                       # units past 2^32: the count used to be cut to 32 bits
    (512, 4194303, 64, 65536, 8),
    (1, (1 << 31) - 1, 64, 96, 16),                           # a block whose rows and a tile pass 2^31
    (512, 4000000, 4096, 4096, 128),                          # units times threads past 2^32
])
def test_lora_refuses_layouts_past_a_launch(ep, N, cap, fin, fout, r):
    """Capacity layouts whose work items do not fit one launch (or 32-bit rows) are refused before anything runs."""
    h = ep.ep_handle_t()
    h.num_tokens, h.num_max_tokens, h.max_rows = 4, 8, N * cap
    h.num_topk, h.num_experts, h.row_align, h.expert_capacity = 1, N, 1, cap
    h.offsets = h.slot = h.row_src = h.status = FAKE
    far = [FAKE * (i + 1) for i in range(12)]                # apart by more than any buffer's bytes
    rc = ep._lib.ep_lora(ctypes.byref(h), far[0], fin, fout, r, far[1], far[2], None, None, far[3], far[4], far[5],
                         1 << 50, None)
    assert rc == ep.EP_ERR_UNSUPPORTED, ep.ep_last_error()
    assert ep.ep_last_error().startswith("ep_lora:")
    rc = ep._lib.ep_lora_backward(ctypes.byref(h), far[6], far[0], fin, fout, r, far[1], far[2], None, far[4], None,
                                  far[7], far[8], far[9], far[5], 1 << 50, None)
    assert rc == ep.EP_ERR_UNSUPPORTED, ep.ep_last_error()
    assert ep.ep_last_error().startswith("ep_lora_backward:")


def test_lora_takes_layouts_within_a_launch(ep):
    """Large blocks whose work items do fit get past that check (to the workspace's)."""
    h = ep.ep_handle_t()
    h.num_tokens, h.num_max_tokens, h.max_rows = 4, 8, 512 * 65536
    h.num_topk, h.num_experts, h.row_align, h.expert_capacity = 1, 512, 1, 65536
    h.offsets = h.slot = h.row_src = h.status = FAKE
    rc = ep._lib.ep_lora(ctypes.byref(h), FAKE, 512, 512, 16, FAKE, FAKE, None, None, 2 * FAKE, FAKE, FAKE, 64, None)
    assert rc == ep.EP_ERR_BUFFER_TOO_SMALL, ep.ep_last_error()


@pytest.mark.parametrize("q,other", [(0, False), (3, True), (4, False)])
def test_layer_refusal_names_a_way_out(ep, q, other):
    """Past 2048 pairs: split the tokens; dispatch, GEMMs and combine only where they take such weights."""
    rc = ep._lib.ep_moe_layer(FAKE, 1025, 256, FAKE, 1, FAKE, 2, 8, 128, q, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40,
                              FAKE * 2, None)
    assert rc == ep.EP_ERR_UNSUPPORTED
    assert "split the tokens" in ep.ep_last_error()
    assert ("dispatch" in ep.ep_last_error()) == other
