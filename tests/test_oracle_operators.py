"""CPU pins of the oracle's router, expert layer and low-rank adapters."""

import numpy as np
import pytest

from oracle import layer as OY, router as OR
from oracle.moe import silu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_router_gradient_against_differences(score, renormalize):
    g = np.random.default_rng(3)
    z, grad = g.normal(size=(5, 11)), g.normal(size=(5, 4))
    z[1, 3] = -np.inf
    ids, _ = OR.route(z, 4, score=score, renormalize=renormalize, scale=1.7)
    ids[2, 1] = -1
    ids[3, 2] = ids[3, 0]                                    # the same expert twice
    kw = dict(score=score, renormalize=renormalize, scale=1.7)
    dz = OR.backward(z, ids, grad, **kw)
    h = 1e-6
    for t in range(5):
        for e in range(11):
            if not np.isfinite(z[t, e]):
                assert dz[t, e] == 0
                continue
            up, dn = z[t].copy(), z[t].copy()
            up[e] += h
            dn[e] -= h
            d = grad[t] @ (OR.weights_of(up, ids[t], score, renormalize, 1.7) -
                           OR.weights_of(dn, ids[t], score, renormalize, 1.7)) / (2 * h)
            assert abs(d - dz[t, e]) < 1e-8


def test_router_rules():
    z = np.array([0.5, 2.0, 2.0, -np.inf, np.nan, 1.0, 0.0, 0.0])
    assert OR.route_row(z, 3)[0] == [1, 2, 5]                # a tie goes to the lower id
    ids, w = OR.route_row(np.where(np.arange(8) == 6, z, -np.inf), 3)
    assert ids == [6, -1, -1] and w.tolist() == [1.0, 0.0, 0.0]
    ids, w = OR.route_row(np.full(8, -np.inf), 2, score="sigmoid")
    assert ids == [-1, -1] and not w.any()
    ids, w = OR.route_row(z, 8, renormalize=False)
    assert ids == [1, 2, 5, 0, 6, 7, -1, -1] and abs(w.sum() - 1.0) < 1e-12


def test_expert_layer_against_loops():
    g = np.random.default_rng(5)
    T, H, I, E, k = 3, 8, 6, 4, 2
    x, w1, w2 = g.normal(size=(T, H)), g.normal(size=(E, 2 * I, H)), g.normal(size=(E, H, I))
    ids, w = np.array([[0, 3], [-1, 2], [1, 1]]), g.random((T, k))
    out, bound = OY.expert_layer(x, ids, w, w1, w2)
    for t in range(T):
        want = np.zeros(H)
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            a = [silu(sum(w1[e, i, h] * x[t, h] for h in range(H))) * sum(w1[e, I + i, h] * x[t, h] for h in range(H))
                 for i in range(I)]
            want += w[t, j] * np.array([sum(w2[e, h, i] * a[i] for i in range(I)) for h in range(H)])
        assert np.allclose(out[t], want, rtol=1e-12)
    assert np.all(bound > 0)


def test_lora_gradients_against_differences():
    g = np.random.default_rng(7)
    T, fin, fout, r, N = 6, 5, 4, 3, 3
    x, a, b = g.normal(size=(T, fin)), g.normal(size=(N, r, fin)), g.normal(size=(N, fout, r))
    s, base, dy, gb = g.random(N), g.normal(size=(T, fout)), g.normal(size=(T, fout)), g.normal(size=(T, fin))
    ids = np.array([0, 2, -1, 0, 2, 2])
    out, _, down, dv = OY.lora(x, ids, a, b, s, base)
    res = OY.lora_backward(x, ids, a, b, s, dy, gb, down, dv)

    def loss(x, a, b):
        return float((OY.lora(x, ids, a, b, s, base)[0] * dy).sum())

    h = 1e-6
    for name, arr in (("grad_x", x), ("grad_a", a), ("grad_b", b)):
        for at in np.ndindex(arr.shape):
            p, m = arr.copy(), arr.copy()
            p[at] += h
            m[at] -= h
            args = {"grad_x": [(p, a, b), (m, a, b)], "grad_a": [(x, p, b), (x, m, b)],
                    "grad_b": [(x, a, p), (x, a, m)]}[name]
            d = (loss(*args[0]) - loss(*args[1])) / (2 * h)
            want = res[name][0][at] - (gb[at] if name == "grad_x" else 0.0)
            assert abs(d - want) < 1e-7
    assert not res["grad_a"][0][1].any() and not res["grad_b"][0][1].any()
    assert np.array_equal(out[2], base[2])


def test_router_groups():
    z = np.array([3.0, -3.0, 1.0, 1.0, 2.0, 0.9, -1.0, -1.0])
    # sums of the two best softmax scores: group 0 (one large) > 2 > 1 > 3
    kw = dict(num_groups=4, topk_groups=2)
    assert OR.route_row(z, 8, group_top=2, **kw)[0] == [0, 4, 5, 1, -1, -1, -1, -1]
    # by sigmoid the sums are 1.0, 1.46, 1.59, 0.54: groups 2 and 1
    assert OR.route_row(z, 4, group_top=2, score="sigmoid", **kw)[0] == [4, 2, 3, 5]
    assert OR.route_row(z, 4, group_top=1, score="sigmoid", **kw)[0] == [0, 4, 5, 1]
    # a bias moves the choice, not the weights
    ids, w = OR.route_row(z, 1, bias=np.array([0, 0, 0, 0, 0, 0, 5.0, 0]), renormalize=False)
    assert ids == [6] and abs(w[0] - OR.scores(z, "softmax")[6]) < 1e-15
