"""Checkpoints of wide blocks (no GPU needed): every inner size that ep_ffn
takes has a checkpoint whose size ep_buffer_bytes gives."""

import pytest

from oracle import dispatch as OD
from tests.test_ffn_host import FAKE, GAP, _ffn, ep  # noqa: F401


@pytest.mark.parametrize("inter,quant", [(32768, "none"), (32832, "none"), (32896, "fp8_b128"), (65536, "none"),
                                         (65536, "fp8_b128")])
def test_checkpoint_of_every_inner_size_has_a_size(ep, inter, quant):  # noqa: F811
    rows = 8                                                  # of the default handle
    total, at = ep.ep_buffer_bytes(rows, 2 * inter, quant)
    assert (total, at) == OD.buffer_bytes(rows, 2 * inter, quant)
    for backward in (False, True):
        # a checkpoint of that size passes (the rows, checked later, are missing); one byte less does not
        kw = dict(I=inter, q=0 if quant == "none" else 2, x=None)
        assert _ffn(ep, backward, ckb=total - 1, **kw) == 3 and f"checkpoint needs {total} bytes" in ep.ep_last_error()
        assert _ffn(ep, backward, ckb=total, **kw) == 1 and "x_buf" in ep.ep_last_error()


def test_widths_end_there(ep):  # noqa: F811
    for width, quant in ((131072 + 32, "none"), (131072 + 128, "fp8_b128"), (1 << 30, "mxfp8")):
        with pytest.raises(ep.EpError) as e:
            ep.ep_buffer_bytes(8, width, quant)
        assert e.value.code == 2


def test_rows_of_tokens_stay_at_65536(ep):  # noqa: F811
    import ctypes
    from tests.test_ffn_host import _handle
    h = _handle(ep)
    rc = ep._lib.ep_dispatch(ctypes.byref(h), FAKE, 65536 + 128, None, 0, FAKE + GAP, 1 << 30, None, None)
    assert rc == 2 and "65536" in ep.ep_last_error()
