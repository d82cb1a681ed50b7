"""GPU router against the float64 oracle: ids exactly, weights and gradients
within bounds derived from the roundings.

Weights: the logits' float32 logs carry an error of at most (|z| + 2) 2^-24
each, expf, the sums and the quotient a few dozen half steps more; a relative
error of (40 + 4 max|z|) 2^-24 covers all of them.  Gradients: products of
such values; (120 + 12 max|z|) 2^-24 of scale * sum |p q| per element, plus
half a step of the output type.
"""

import numpy as np
import pytest
import torch

from oracle import router as OR
from tests.hip_path import DEV

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -24


@pytest.fixture(scope="module")
def ep():
    from combine_topk_idx_amd import ep as _ep
    return _ep


def _logits(seed, T, E, dtype, masked=0.0):
    g = np.random.default_rng(seed)
    z = torch.from_numpy(g.normal(size=(T, E)) * 2.0).to(dtype)
    if masked:
        z[torch.from_numpy(g.random((T, E)) < masked)] = -float("inf")
    return z


def _run(ep, z, k, idt, **kw):
    T = z.shape[0]
    idx = torch.full((T, k), 77, dtype=idt, device=DEV)
    w = torch.full((T, k), float("nan"), device=DEV)
    bias = kw.pop("bias", None)
    ep.ep_router(z.to(DEV), idx, w, bias=None if bias is None else bias.to(DEV), **kw)
    return idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def _check(ep, z, k, idt=torch.int64, **kw):
    idx, w = _run(ep, z, k, idt, **dict(kw))
    if kw.get("bias") is not None:
        kw["bias"] = kw["bias"].double().numpy()
    want_idx, want_w = OR.route(z.double().numpy(), k, **kw)
    assert np.array_equal(idx, want_idx)
    zmax = float(z[torch.isfinite(z)].abs().max()) if torch.isfinite(z).any() else 0.0
    assert np.all(np.abs(w - want_w) <= (40 + 4 * zmax) * HALF * np.abs(want_w) + 2.0 ** -126)
    return want_idx, zmax


CASES = [
    (1, 1, 1, torch.float32, 0.0, dict()),
    (1, 256, 8, torch.float32, 0.0, dict(score="sigmoid", bias=True, num_groups=8, topk_groups=4, group_top=2, scale=2.5)),
    (5, 60, 4, torch.bfloat16, 0.1, dict(renormalize=False)),
    (67, 512, 16, torch.float16, 0.05, dict(score="sigmoid", renormalize=False)),
    (130, 96, 6, torch.float32, 0.3, dict(bias=True, num_groups=3, topk_groups=2, group_top=1)),
    (64, 64, 16, torch.bfloat16, 0.9, dict(score="sigmoid", num_groups=16, topk_groups=16, group_top=2)),
    (33, 65, 3, torch.float32, 0.0, dict(score="softmax", num_groups=5, topk_groups=1, group_top=2, renormalize=False)),
    (40, 160, 6, torch.float32, 0.0, dict(num_groups=8, topk_groups=3, group_top=1, renormalize=False, scale=16.0)),
    (300, 128, 8, torch.bfloat16, 0.0, dict(bias=True)),
    (9, 512, 8, torch.float32, 0.0, dict(num_groups=64, topk_groups=5, group_top=2, bias=True)),
]


@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
def test_router(ep, i, idt):
    T, E, k, dtype, masked, kw = CASES[i]
    kw = dict(kw)
    z = _logits(i, T, E, dtype, masked)
    if kw.pop("bias", False):
        kw["bias"] = torch.from_numpy(np.random.default_rng(100 + i).normal(size=E) * 0.2).float()
    ids, zmax = _check(ep, z, k, idt, **kw)
    # the gradient at these ids
    grad = np.random.default_rng(200 + i).normal(size=(T, k)).astype(np.float32)
    dz = torch.full((T, E), float("nan"), dtype=dtype, device=DEV)
    gkw = {n: kw[n] for n in ("score", "renormalize", "scale") if n in kw}
    ep.ep_router_backward(z.to(DEV), torch.from_numpy(ids).to(idt).to(DEV), torch.from_numpy(grad).to(DEV), dz, **gkw)
    want = OR.backward(z.double().numpy(), ids, grad, **gkw)
    _, p = OR.route(z.double().numpy(), k, **{**gkw, **{n: v for n, v in kw.items() if n not in gkw and n != "bias"},
                                              **({"bias": kw["bias"].double().numpy()} if "bias" in kw else {})})
    mag = np.abs(p).max(axis=1, keepdims=True) * (np.abs(grad) * (ids >= 0)).sum(axis=1, keepdims=True) * 2
    tol = (120 + 12 * zmax) * HALF * mag + torch.finfo(dtype).eps / 2 * np.abs(want) + torch.finfo(dtype).tiny
    got = dz.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))


def test_masks(ep):
    lowest = torch.finfo(torch.float32).min
    z = torch.full((6, 8), -float("inf"))
    z[1, 6] = 0.25                                            # one expert left
    z[2] = float("nan")
    z[3] = torch.tensor([lowest] * 4 + [1.0, lowest, lowest, -2.0])   # the type's lowest is finite: still there
    z[4] = lowest
    z[5] = torch.tensor([float("inf"), 1, 2, 3, -float("inf"), float("nan"), 0, 0])
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            for bias in (None, torch.zeros(8)):
                idx, w = _run(ep, z, 3, torch.int64, score=score, renormalize=renorm, bias=bias)
                assert idx[0].tolist() == [-1, -1, -1] and not w[0].any()
                assert idx[1].tolist() == [6, -1, -1] and not w[1, 1:].any()
                assert idx[2].tolist() == [-1, -1, -1] and not w[2].any()
                assert idx[3].tolist() == [4, 7, 0]
                assert idx[4].tolist() == [0, 1, 2]
                if score == "softmax":                        # sigmoids tie in float64 above 37
                    assert idx[5].tolist()[0] == 0
                assert np.all(np.isfinite(w))
    dz = torch.full((6, 8), float("nan"), device=DEV)
    idx, _ = _run(ep, z, 3, torch.int64)
    ep.ep_router_backward(z.to(DEV), torch.from_numpy(idx).to(DEV), torch.ones(6, 3, device=DEV), dz, renormalize=False)
    dz = dz.cpu()
    assert torch.isfinite(dz).all() and not dz[0].any() and not dz[2].any()


def test_ties_and_near_ties(ep):
    z = torch.zeros(3, 70)
    z[1, 40:] = 1.0
    assert _run(ep, z, 4, torch.int64)[0].tolist() == [[0, 1, 2, 3], [40, 41, 42, 43], [0, 1, 2, 3]]
    assert _run(ep, z, 4, torch.int64, bias=torch.zeros(70), score="sigmoid")[0].tolist()[1] == [40, 41, 42, 43]
    # keys s + bias that float32 cannot tell apart: the order is float64's
    g = np.random.default_rng(11)
    z = torch.from_numpy(g.normal(size=(50, 64))).float()
    s = 1.0 / (1.0 + np.exp(-z[0].double().numpy()))
    bias = torch.from_numpy((0.9 - s)).float()               # every key of row 0 is 0.9 to within 2^-25
    _check(ep, z, 8, score="sigmoid", bias=bias)
    _check(ep, z, 8, score="sigmoid", bias=bias, num_groups=8, topk_groups=4, group_top=2)
    s = np.exp(z[0].double().numpy())
    _check(ep, z, 8, score="softmax", bias=torch.from_numpy(0.5 - s / s.sum()).float())
    # saturated scores: without a bias the logits decide
    z = torch.tensor([[50.0, 60.0, 40.0, 70.0], [-200.0, -150.0, -100.0, -180.0]])
    for score in ("softmax", "sigmoid"):
        assert _run(ep, z, 4, torch.int64, score=score)[0].tolist() == [[3, 1, 0, 2], [2, 1, 3, 0]]
    _check(ep, z, 4, score="sigmoid")


def test_backward_ids(ep):
    """Ids of the caller's own: repeated, out of range and -1; the logits' memory for the gradient."""
    g = np.random.default_rng(17)
    z = torch.from_numpy(g.normal(size=(4, 12))).float()
    ids = np.array([[3, 3, 5], [-1, 12, 7], [-5, 1 << 20, -1], [0, 11, 0]])
    grad = g.normal(size=(4, 3)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            dz = z.to(DEV).clone()
            ep.ep_router_backward(dz, torch.from_numpy(ids).to(DEV), torch.from_numpy(grad).to(DEV), dz, score=score,
                                  renormalize=renorm, scale=2.0)
            want = OR.backward(z.double().numpy(), np.where(ids > 11, -1, ids), grad, score=score, renormalize=renorm,
                               scale=2.0)
            assert np.all(np.abs(dz.cpu().double().numpy() - want) <= 200 * HALF * 2 * np.abs(grad).sum())


def test_no_tokens(ep):
    z = torch.zeros(0, 8, device=DEV)
    idx, w = torch.zeros(0, 2, dtype=torch.int64, device=DEV), torch.zeros(0, 2, device=DEV)
    ep.ep_router(z, idx, w)
    ep.ep_router_backward(z, idx, w, torch.zeros_like(z))


@pytest.mark.parametrize("E,groups", [(256, 8), (256, 2), (64, 4), (128, 16), (60, 5), (512, 64)])
@pytest.mark.parametrize("top", [1, 2])
def test_equal_groups(ep, E, groups, top):
    """Groups of equal rank: the lower ones stay; a better one anywhere comes first."""
    keep = max(1, groups // 2)
    for bias in (None, torch.zeros(E)):
        for score in ("softmax", "sigmoid"):
            z = torch.zeros(groups + 1, E)
            for g in range(groups):
                z[g, g * (E // groups):(g + 1) * (E // groups)] = 1.0
            _check(ep, z, min(16, E // groups * keep), score=score, bias=bias, num_groups=groups, topk_groups=keep,
                   group_top=top)


@pytest.mark.parametrize("T", [1, 15, 16, 17, 1000])
def test_many_tokens_grouped(ep, T):
    g = np.random.default_rng(T)
    z = torch.from_numpy(g.normal(size=(T, 256)) * 1.5).float()
    bias = torch.from_numpy(g.normal(size=256) * 0.1).float()
    _check(ep, z, 8, torch.int32, score="sigmoid", bias=bias, num_groups=8, topk_groups=4, group_top=2, scale=2.5)
    _check(ep, z.bfloat16(), 9, torch.int64, score="softmax", bias=bias, renormalize=False)
    # strided storage is refused, an unaligned start is not
    big = torch.zeros(T * 256 + 1)
    big[1:] = z.reshape(-1)
    zu = big.to(DEV)[1:].view(T, 256)
    idx, w = torch.empty(T, 8, dtype=torch.int64, device=DEV), torch.empty(T, 8, device=DEV)
    ep.ep_router(zu, idx, w)
    assert np.array_equal(idx.cpu().numpy(), OR.route(z.double().numpy(), 8)[0])
    with pytest.raises(ep.EpError):
        ep.ep_router(torch.zeros(256, max(T, 2), device=DEV).t(), idx, w)


@pytest.mark.parametrize("E,groups", [(64, 4), (60, 5)])
def test_infinite_biases(ep, E, groups):
    """+inf chooses first, -inf and NaN never; a group with one key left ranks last by sums, even if it is +inf."""
    size = E // groups
    z = _logits(3, 12, E, torch.float32)
    z[5, 1:size] = -float("inf")                              # group 0 of row 5 has one expert
    bias = torch.zeros(E)
    bias[0], bias[size], bias[size + 1], bias[2 * size] = float("inf"), float("nan"), -float("inf"), float("inf")
    for top in (1, 2):
        ids, _ = _check(ep, z, 6, score="sigmoid", bias=bias, num_groups=groups, topk_groups=2, group_top=top)
        assert (ids[:, 0] == 0).sum() >= 11 and not np.isin(ids, [size, size + 1]).any()
        _check(ep, z, 6, score="softmax", bias=bias, num_groups=groups, topk_groups=groups - 1, group_top=top)


@pytest.mark.parametrize("E,groups", [(64, 4), (256, 8), (32, 16), (60, 5), (238, 2)])
def test_several_infinite_biases_in_a_group(ep, E, groups):
    """A group's sum is infinite with one +inf key and with two: among such groups the lower ones stay, whichever
    path the group shape takes."""
    size = E // groups
    last = groups - 1
    z = _logits(4, 20, E, torch.float32)
    one_two, two_one = torch.zeros(E), torch.zeros(E)
    one_two[[0, last * size, last * size + 1]] = float("inf")
    two_one[[0, 1, last * size]] = float("inf")
    for score in ("softmax", "sigmoid"):
        for bias in (one_two, two_one):
            for keep in (1, max(1, groups - 1)):
                ids, _ = _check(ep, z, min(3, size), score=score, bias=bias, num_groups=groups, topk_groups=keep,
                                group_top=2)
                assert (ids[:, 0] == 0).all()
    # every group infinite, in one place or two: the order of the groups decides
    bias = torch.zeros(E)
    bias[::size] = float("inf")
    bias[1 + size * (groups // 2)::2 * size] = float("inf")
    _check(ep, z, min(4, size), score="sigmoid", bias=bias, num_groups=groups, topk_groups=max(1, groups // 2),
           group_top=2)


@pytest.mark.parametrize("T,E,groups", [((1 << 28) + 37, 2, 1), ((1 << 26) + 21, 6, 3)])
def test_more_tokens_than_a_launch_holds(ep, T, E, groups):
    """One thread short of 2^32 is the most a launch takes: 16 threads a token on the row path, 64 on the wave path."""
    print(f"\n[case] router of {T} tokens", flush=True)
    z = torch.randint(-8, 9, (T, E), dtype=torch.int8, device=DEV).to(torch.bfloat16)
    idx = torch.full((T, 1), 77, dtype=torch.int32, device=DEV)
    w = torch.full((T, 1), float("nan"), device=DEV)
    ep.ep_router(z, idx, w, renormalize=True, num_groups=groups, topk_groups=1, scale=2.0)
    best = z[:, 0].clone()
    want = torch.zeros(T, dtype=torch.int32, device=DEV)
    for e in range(1, E):                                     # the first of the largest
        more = z[:, e] > best
        want[more] = e
        best = torch.maximum(best, z[:, e])
    assert torch.equal(idx[:, 0], want)
    assert bool((w == 2.0).all())
    if groups > 1:
        return
    dz = torch.full((T, E), float("nan"), dtype=torch.bfloat16, device=DEV)
    ep.ep_router_backward(z, idx, w, dz, renormalize=True, scale=2.0)
    assert not dz.any()                                       # one choice, renormalised: its weight is constant


@pytest.mark.parametrize("T,E,groups,keep,top,score,biased", [
    (4099, 238, 2, 1, 2, "softmax", True), (4096, 60, 5, 2, 1, "sigmoid", False), (2051, 500, 4, 3, 2, "softmax", False),
    (3001, 120, 24, 11, 2, "sigmoid", True), (1030, 511, 7, 5, 2, "sigmoid", True),
])
def test_prefill_off_whole_lanes(ep, T, E, groups, keep, top, score, biased):
    """Group shapes that do not fall on whole lanes, at the sizes of a prompt, some experts masked out."""
    z = _logits(T, T, E, torch.float32, 0.05)
    kw = dict(score=score, num_groups=groups, topk_groups=keep, group_top=top)
    if biased:
        kw["bias"] = torch.from_numpy(np.random.default_rng(E).normal(size=E) * 0.1).float()
    _check(ep, z, 8, torch.int32, **kw)
