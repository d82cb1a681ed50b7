"""The feed-forward block at its widest inner sizes, whose checkpoints are
wider than any row of tokens, against the float64 oracle."""

import pytest
import torch

from tests.test_gpu_ffn import Case, Rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    from combine_topk_idx_amd import ep as _ep
    return _ep


@pytest.mark.parametrize("T", [6, 45, 300])
@pytest.mark.parametrize("inter,quant", [(32832, "none"), (32896, "fp8_b128"), (65536, "none"), (65536, "fp8_b128")])
def test_matches_oracle(ep, inter, quant, T):
    c = Case(ep, Rows(ep, T, T=T, k=1, E=1), 64, inter, "silu", quant, seed=T)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    c.check_forward()
    c.check_backward()
    assert torch.all(c.ck[c.total:] == 0x5A)
