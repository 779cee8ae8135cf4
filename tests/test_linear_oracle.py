"""Pins of the fp64 oracle of linear attention with a decay per head (CPU)."""
import numpy as np
import pytest

from oracle import linear_ref as R


def _inputs(T, H, dk, dv, seed):
    r = np.random.default_rng(seed)
    g = -np.abs(r.standard_normal((T, H))) * 0.5
    return (r.standard_normal((T, H, dk)), r.standard_normal((T, H, dk)), r.standard_normal((T, H, dv)), g,
            r.standard_normal((H, dk, dv)))


def test_two_tokens_by_hand():
    # S_0 = 4; a = (1/2, 1/4); k v = 3 * 5, 2 * 7; q = 1, 10
    a = np.log([[0.5], [0.25]])
    one = lambda x: np.array(x, np.float64).reshape(2, 1, 1)  # noqa: E731
    o, S = R.forward(one([1, 10]), one([3, 2]), one([5, 7]), a, np.full((1, 1, 1), 4.0), scale=2.0)
    assert np.allclose(o[:, 0, 0], [2 * 17, 2 * 10 * (17 / 4 + 14)], rtol=1e-15)
    assert np.allclose(S, 17 / 4 + 14, rtol=1e-15)


@pytest.mark.parametrize("T", [1, 2, 7])
def test_forward_is_masked_attention_with_decays(T):
    q, k, v, g, S0 = _inputs(T, 2, 3, 4, T)
    o, S = R.forward(q, k, v, g, S0, 0.7)
    G = np.cumsum(g, 0)
    for h in range(2):
        D = np.tril(np.exp(G[:, None, h] - G[None, :, h]))
        want = 0.7 * ((q[:, h] @ k[:, h].T * D) @ v[:, h] + np.exp(G[:, h, None]) * (q[:, h] @ S0[h]))
        assert np.allclose(o[:, h], want, rtol=1e-12, atol=1e-12)
        f = np.exp(G[-1, h] - G[:, h])
        assert np.allclose(S[h], np.exp(G[-1, h]) * S0[h] + (k[:, h] * f[:, None]).T @ v[:, h], rtol=1e-12, atol=1e-12)


def test_erasing_decay():
    q, k, v, g, S0 = _inputs(5, 1, 2, 2, 3)
    g[3] = -np.inf
    o, S = R.forward(q, k, v, g, S0)
    o2, S2 = R.forward(q[3:], k[3:], v[3:], g[3:], np.zeros_like(S0))
    assert np.array_equal(o[3:], o2) and np.array_equal(S, S2)


def test_gradients_are_central_differences():
    T, H, dk, dv = 5, 2, 3, 2
    q, k, v, g, S0 = _inputs(T, H, dk, dv, 11)
    r = np.random.default_rng(12)
    do, dS = r.standard_normal((T, H, dv)), r.standard_normal((H, dk, dv))
    x = {"q": q, "k": k, "v": v, "g": g, "initial_state": S0}

    def loss():
        o, S = R.forward(x["q"], x["k"], x["v"], x["g"], x["initial_state"], 0.6)
        return (o * do).sum() + (S * dS).sum()

    d = R.backward(q, k, v, g, S0, do, dS, 0.6)
    e = 1e-6
    for name, t in x.items():
        num = np.zeros_like(t)
        for i in np.ndindex(t.shape):
            keep = t[i]
            t[i] = keep + e
            up = loss()
            t[i] = keep - e
            num[i] = (up - loss()) / (2 * e)
            t[i] = keep
        # differences: e^2 / 6 times a third derivative of order 1e2, and 1e-16 * |loss| / e
        assert np.allclose(d[name], num, rtol=1e-6, atol=1e-7), name


def test_shared_heads():
    x = np.arange(12.0).reshape(1, 2, 6)
    r = R.repeat_heads(x, 6)
    assert r.shape == (1, 6, 6) and np.array_equal(r[0, 2], x[0, 0]) and np.array_equal(r[0, 3], x[0, 1])
    assert np.array_equal(R.sum_heads(r, 2), 3 * x)
