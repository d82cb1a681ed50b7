"""Which tile the grouped products of the feed-forward block and of the
block-scaled product run on, and the cases that reach each of them with more
units than workgroups.

The rule restates the library's: from the mean rows of an expert, and from the
units that a launch of a height has at least.  Heights: 0 is the form of few
rows (64 columns, the reduction split over the waves)."""

import numpy as np

CUS = 256


def height(rows, experts, column_tiles, few):
    used = min(experts, rows)
    mean = rows // used
    if mean <= 32 and few:
        return 0

    def units(bm):
        return (rows // bm + (used + 1) // 2) * column_tiles
    if mean > 192:
        return 256
    if mean > 32 and units(128) >= 640:
        return 128
    if mean > 32 and units(64) >= 128:
        return 64
    return 32


def up(n, by):
    return -(-n // by)


def units(counts, bm, column_tiles):
    return sum(up(n, bm) for n in counts) * column_tiles


def launch(counts, cols, tile_cols, few):
    """(height, units) of a launch; few: the columns of that form's tile, or 0."""
    h = height(sum(counts), len(counts), up(cols, tile_cols), few > 0)
    return h, units(counts, h or 32, up(cols, few if h == 0 else tile_cols))


def ffn_launches(counts, H, inter, quant):
    """{mode: (height, units, stages of the reduction)} of a forward and backward pass."""
    made = dict(up=(*launch(counts, inter, 128, 32 if quant == "none" else 0), H // 64),
                down=(*launch(counts, H, 256, 64), inter // 64),
                act=(*launch(counts, inter, 256, 0), H // 64),
                grad_x=(*launch(counts, H, 256, 0), 2 * inter // 64))
    tiles = up(2 * inter, 256) * up(H, 256) + up(H, 256) * up(inter, 256)
    made["weights"] = (256, tiles * len(counts), up(max(counts), 64))
    return made


def gmm_launch(counts, K, N, form, out_quant="none"):
    """(height, units, stages)."""
    gated = form == "gated"
    few = 0 if form == "transposed" or out_quant != "none" else 32 if gated else 64
    return (*launch(counts, N // 2 if gated else N, 128 if gated else 256, few), K // 128)


def uneven(E, lo, hi, seed, mean):
    """Rows by expert between lo and hi, one expert without and one with a single one, `mean` in all but the remainder."""
    g = np.random.default_rng(seed)
    n = g.integers(lo, hi + 1, size=E)
    n[E // 3], n[E // 2] = 0, 1
    while n.sum() != mean * E:                                # spread what is left over, one row at a time
        e = g.integers(0, E)
        if n[e] > 1 and lo <= n[e] + np.sign(mean * E - n.sum()) <= hi:
            n[e] += np.sign(mean * E - n.sum())
    return [int(v) for v in n]


LOW = uneven(150, 1, 33, 1, 17)                               # up to 32 rows an expert on average
MIDDLE = uneven(64, 20, 140, 2, 84)
UPPER = uneven(64, 65, 190, 3, 129)
MANY = uneven(40, 65, 400, 4, 232)

# (rows by expert, H, I, checkpoint): one wide side at a time, reductions of one, two, three and five stages on the other.
# (Few rows an expert with a bf16 checkpoint have the form of few rows.)
FFN = []
for counts, wide in ((LOW, 640), (MIDDLE, 640), (UPPER, 1600), (MANY, 1344)):
    for i, short in enumerate((64, 128, 192, 320)):
        quant = "none" if i % 2 and counts is not LOW else "fp8_b128"
        FFN.append((counts, short, wide if quant == "none" else up(wide, 128) * 128, quant))
        FFN.append((counts, wide, short, "fp8_b128" if short == 128 else "none"))
FFN += [(MIDDLE, 576, 640, "none"), (LOW, 576, 640, "fp8_b128")]

# (rows by expert, N): N of a gated product too
GMM = [(LOW, 1024), (MIDDLE, 768), (UPPER, 1792), (MANY, 1536)]
GMM_K = [128, 256, 384, 640]
