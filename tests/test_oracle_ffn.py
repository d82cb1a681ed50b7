"""Pins of the feed-forward oracle: central differences, brute force, the
activations' constants."""

import numpy as np
import pytest

from oracle import ffn as OF


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gradients_match_differences(kind):
    g = np.random.default_rng(5)
    n, H, inter = 3, 6, 4
    x, w1, w2, dy = (g.normal(size=s) for s in ((n, H), (2 * inter, H), (H, inter), (n, H)))

    def loss(x, w1, w2):
        return float((OF.forward(x, w1, w2, kind)["out"][0] * dy).sum())

    both = x @ w1.T
    got = OF.backward(x, w1, w2, both[:, :inter], both[:, inter:], dy, kind)
    h = 1e-5
    for name, i in (("grad_x", 0), ("grad_w1", 1), ("grad_w2", 2)):
        args = [x, w1, w2]
        want = np.empty_like(args[i])
        for at in np.ndindex(args[i].shape):
            d = np.zeros_like(args[i])
            d[at] = h
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + d, args[i] - d
            want[at] = (loss(*up) - loss(*down)) / (2 * h)
        # the differences' own error is of order h^2 and 1e-16 / h
        assert np.allclose(got[name][0], want, rtol=1e-6, atol=1e-8), name


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activation_constants(kind):
    z = np.linspace(-12, 12, 200001)
    f, df = OF.act(kind, z)
    assert np.abs(df).max() <= OF.SLOPE
    assert np.abs(np.diff(df) / np.diff(z)).max() <= OF.BEND
    assert np.allclose(np.diff(f) / np.diff(z), (df[1:] + df[:-1]) / 2, atol=1e-6)


def test_forward_matches_loops():
    g = np.random.default_rng(6)
    n, H, inter = 2, 5, 3
    x, w1, w2 = g.normal(size=(n, H)), g.normal(size=(2 * inter, H)), g.normal(size=(H, inter))
    out = OF.forward(x, w1, w2, "silu")["out"][0]
    for r in range(n):
        a = []
        for i in range(inter):
            gate = sum(x[r, h] * w1[i, h] for h in range(H))
            up = sum(x[r, h] * w1[inter + i, h] for h in range(H))
            a.append(gate / (1 + np.exp(-gate)) * up)
        for h in range(H):
            assert abs(out[r, h] - sum(a[i] * w2[h, i] for i in range(inter))) < 1e-12


def test_spread():
    s = np.array([[1.0, 2.0], [3.0, 4.0]])
    v = OF.spread(s, 128)
    assert v.shape == (256, 256) and v[127, 127] == 1 and v[127, 128] == 2 and v[128, 127] == 3 and v[255, 255] == 4
    assert OF.spread(s).shape == (2, 256)
