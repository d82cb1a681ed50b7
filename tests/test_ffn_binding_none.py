"""Buffers left out of the binding's feed-forward and block-scaled calls: the
library's own answer, as for its C callers (an empty capacity needs no row
buffers; what is missing is named)."""

import pytest
import torch

from tests.test_ffn_host import FAKE, GAP, _handle, ep  # noqa: F401


def test_block_scaled_without_buffers(ep):  # noqa: F811
    def call(h, a, out):
        ep.ep_moe_gmm_b128(h, a, "fp8_b128", 128, 128, FAKE, FAKE + GAP, out, recv_count=FAKE, stream=0)
    call(_handle(ep, T=0, tmax=0), None, None)
    for a, out in ((None, FAKE), (FAKE, None)):
        with pytest.raises(ep.EpError, match="a_buf / out_buf NULL"):
            call(_handle(ep), a, out)


@pytest.mark.gpu
def test_block_without_buffers(ep):  # noqa: F811
    E, H, I = 3, 64, 64
    new = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    w1, w2, g1, g2, rows = new(E, 2 * I, H), new(E, H, I), new(E, 2 * I, H) + 1, new(E, H, I) + 1, new(8, H)
    ws, ck = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda"), torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    lws, count = torch.zeros(4096, dtype=torch.uint8, device="cuda"), torch.zeros(E, dtype=torch.int64, device="cuda")
    h = ep.ep_layout(torch.zeros(0, 2, dtype=torch.int64, device="cuda"), E, 0, count, lws)
    assert h.max_rows == 0
    ep.ep_ffn(h, None, w1, w2, ws, None, recv_count=count)
    ep.ep_ffn_backward(h, None, None, w1, w2, None, ws, None, g1, g2, recv_count=count)
    assert not g1.any() and not g2.any()
    full = ep.ep_layout(torch.zeros(4, 2, dtype=torch.int64, device="cuda"), E, 4, count, lws)
    for name, a in (("x_buf", dict(x=None)), ("workspace", dict(ws=None)), ("out_buf", dict(out=None))):
        b = dict(x=rows, ws=ws, out=rows.clone())
        b.update(a)
        with pytest.raises(ep.EpError, match=name):
            ep.ep_ffn(full, b["x"], w1, w2, b["ws"], b["out"], recv_count=count)
    for name, a in (("x_buf", dict(x=None)), ("checkpoint", dict(ck=None)), ("grad_out / grad_x", dict(dy=None)),
                    ("grad_out / grad_x", dict(gx=None)), ("grad_w1", dict(g1=None)), ("workspace", dict(ws=None))):
        b = dict(x=rows, dy=rows, ck=ck, ws=ws, gx=rows.clone(), g1=g1)
        b.update(a)
        with pytest.raises(ep.EpError, match=name):
            ep.ep_ffn_backward(full, b["dy"], b["x"], w1, w2, b["ck"], b["ws"], b["gx"], b["g1"], g2, recv_count=count)
