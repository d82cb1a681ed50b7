"""The cases of tests/gemm_tiles.py reach every tile height of every product
with more units than workgroups (no GPU needed)."""

from tests import gemm_tiles as T

HEIGHTS = {32, 64, 128, 256}


def test_feed_forward_cases_reach_every_kernel():
    seen = {}
    for counts, H, inter, quant in T.FFN:
        for mode, (h, units, stages) in T.ffn_launches(counts, H, inter, quant).items():
            if units > T.CUS:
                seen.setdefault((mode, h), set()).add(stages)
    for h in HEIGHTS:
        assert {1, 2, 3, 5} <= seen["up", h], (h, seen["up", h])
        assert {1, 2, 3, 5} <= seen["act", h], (h, seen["act", h])
        assert {2, 4, 6, 10} <= seen["grad_x", h], (h, seen["grad_x", h])
        # (few rows an expert have the other form there)
        assert {1, 2, 3, 5} <= seen["down", h if h > 32 else 0], h
    assert max(seen["weights", 256]) >= 5


def test_block_scaled_cases_reach_every_kernel():
    seen = set()
    for counts, N in T.GMM:
        for form in ("plain", "transposed", "gated"):
            for out_quant in ("none", "fp8_b128"):
                if out_quant == "none" or form == "gated":
                    h, units, _ = T.gmm_launch(counts, 128, N, form, out_quant)
                    assert units > T.CUS, (form, N, h, units)
                    seen.add((form, out_quant != "none", h))
    assert {h for f, q, h in seen if f == "plain"} == {0, 64, 128, 256}
    assert {h for f, q, h in seen if f == "transposed"} == HEIGHTS
    assert {h for f, q, h in seen if f == "gated" and q} == HEIGHTS
    assert {h for f, q, h in seen if f == "gated" and not q} == {0, 64, 128, 256}
