"""Every row-tile height of the feed-forward block's and of the block-scaled
product's launches against 64 bits, with more units than the card has
workgroups: stages that go on from unit to unit, stores still in flight over
the border, row scales and largest magnitudes whose LDS the next unit takes.
Which height a case runs on is computed (tests/gemm_tiles.py)."""

import numpy as np
import pytest
import torch

from oracle import ffn as OF
from tests import gemm_tiles as T
from tests.hip_path import DEV
from tests.moe_bounds import MFMA_FRAC_BITS
from tests.test_gpu_ffn import CANARY, Case as FfnCase, Counted
from tests.test_gpu_gmm_b128 import Case as GmmCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    from combine_topk_idx_amd import ep as _ep
    return _ep


@pytest.fixture(scope="module", autouse=True)
def _the_card_has_the_cus_of_the_cases():
    assert torch.cuda.get_device_properties(0).multi_processor_count <= T.CUS


def _name(counts, *rest):
    kind = [k for k in ("LOW", "MIDDLE", "UPPER", "MANY") if getattr(T, k) is counts][0]
    return "-".join(map(str, (kind, *rest)))


@pytest.mark.parametrize("i", range(len(T.FFN)), ids=[_name(*c) for c in T.FFN])
def test_feed_forward(ep, i):
    counts, H, inter, quant = T.FFN[i]
    c = FfnCase(ep, Counted(ep, counts, i, row_align=1 if i % 3 else 16), H, inter, ("silu", "gelu")[i % 2], quant, seed=i)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    c.check_forward()
    c.check_backward()
    assert torch.all(c.ck[c.total:] == 0x5A)


class OnDevice(GmmCase):
    """The same case, its float64 products and the matrix cores' bound formed on the device (elementwise and by 2-D
    products)."""

    def want(self, e, a, n):
        E, R, K, N = self.dims
        x = torch.from_numpy(self.x[a:a + n]).to(DEV)
        w = torch.from_numpy(np.ascontiguousarray(self.w[e].T if self.transposed else self.w[e])).to(DEV)
        wt, wa = w.t().contiguous(), w.abs().t().contiguous()
        y, mag = x @ wt, x.abs() @ wa
        # 2^-11 of each step's largest |product|, float32 accumulation (tests/moe_bounds.py) ...
        top = torch.zeros_like(y)
        for s in range(0, K, 64):
            xs, ws = x[:, s:s + 64].abs(), w[:, s:s + 64].abs()
            for r in range(0, n, 64):
                top[r:r + 64] += (xs[r:r + 64, None, :] * ws[None]).amax(dim=-1)
        err = 2.0 ** -MFMA_FRAC_BITS * top + (K // 64) * 2.0 ** -24 * mag
        # ... and the scales' product, its use and the sum of the blocks
        err = (err + (K // 128 + 4) * 2.0 ** -23 * mag).cpu().numpy()
        y = y.cpu().numpy()
        if self.act == "none":
            return y, err
        g, u, eg, eu = y[:, :N // 2], y[:, N // 2:], err[:, :N // 2], err[:, N // 2:]
        f, _ = OF.act(self.act, g)
        ef = OF.SLOPE * eg + OF.EVAL * (1.0 + np.abs(g))
        return f * u, ef * (np.abs(u) + eu) + np.abs(f) * eu + OF.EVAL * np.abs(f * u)


# the output's form goes through all four with the reduction's length
OUT = ["none", "fp8_b128", "fp8_b128_pow2", "fp8_b128_ue8m0"]


@pytest.mark.parametrize("K", T.GMM_K)
@pytest.mark.parametrize("form", ["plain", "transposed", "gated", "gated e4m3"])
@pytest.mark.parametrize("i", range(len(T.GMM)), ids=[_name(*c) for c in T.GMM])
def test_block_scaled(ep, i, form, K):
    counts, N = T.GMM[i]
    mode = ("fp8_b128", "fp8_b128_ue8m0")[(T.GMM_K.index(K) + (form == "transposed")) % 2]
    out = OUT[1 + (T.GMM_K.index(K) + i) % 3] if form == "gated e4m3" else "none"
    c = OnDevice(ep, Counted(ep, counts, i + 1, row_align=16 if i % 2 else 1), K, N, mode, transposed=form == "transposed",
                 act="none" if form in ("plain", "transposed") else ("silu", "gelu")[i % 2], out_quant=out, seed=K + i)
    c.run()
    torch.cuda.synchronize()
    c.check()


def test_units_repeat_bit_for_bit(ep):
    """A second run over what the first left, on other stages' leftovers in LDS, gives the same bits."""
    for counts, H, inter, quant in (T.FFN[8 + 4], T.FFN[16 + 3], T.FFN[24 + 5]):
        c = FfnCase(ep, Counted(ep, counts, 3), H, inter, "silu", quant, seed=3)
        first = None
        for _ in range(4):
            for t in (c.out, c.gx, c.gw1, c.gw2):
                t.fill_(CANARY)
            c.forward()
            c.backward()
            got = [t.clone().view(torch.int16) for t in (c.out, c.gx, c.gw1, c.gw2)]
            assert first is None or all(torch.equal(a, b) for a, b in zip(first, got))
            first = got
