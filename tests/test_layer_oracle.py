"""Pins of oracle/layer_ref.py: values worked by hand and central differences of its gradients (fp64, CPU)."""
import numpy as np
import pytest

from oracle import layer_ref as R

GATES, INPUTS = ("lower_bound", "softplus", "sigmoid", "log"), ("none", "complement", "norm")


def _differences(value, x, grad, step=1e-6):
    """Central differences of value() in every element of the array x, which value reads."""
    # value is of the order of 10: its rounding is 1e-15, over 2 * step 1e-9; the third derivative's term is 1e-12
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + step
        up = value()
        x[i] = keep - step
        down = value()
        x[i] = keep
        assert abs((up - down) / (2 * step) - grad[i]) <= 1e-7 * max(1.0, abs(grad[i])), (i, (up - down) / (2 * step), grad[i])


def test_scan_by_hand():
    one = np.ones((2, 1))
    h, before, S = R.scan(one * 3, np.log(0.5) * one, None, 0, 0, np.array([4.0]), gate="log")
    assert np.allclose(h[:, 0], [5.0, 5.5]) and np.allclose(before[:, 0], [4.0, 5.0]) and np.allclose(S, 5.5)
    h, _, _ = R.scan(one * 3, np.log(0.5) * one, 0 * one, 0, 0, np.array([4.0]), gate="log", input_scale="complement")
    assert np.allclose(h[:, 0], [2.75, 2.125])  # 0.5 * 4 + 0.5 * 0.5 * 3
    h, _, _ = R.scan(one, np.log(0.6) * one, None, 0, 0, np.zeros(1), gate="log", input_scale="norm")
    assert np.allclose(h[:, 0], [0.8, 1.28])
    g, _, _ = R.decay(np.zeros((1, 1)), 0.0, 0.0, "softplus", 0)
    assert np.allclose(g, -np.log(2))
    assert np.allclose(R.decay(np.zeros((1, 1)), 0.0, 0.0, "lower_bound", -5.0)[0], -2.5)
    assert np.allclose(R.decay(np.zeros((1, 1)), np.log(3.0), 0.0, "sigmoid", 0)[0], -1.5)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("kind", INPUTS)
@pytest.mark.parametrize("gated", [True, False])
def test_scan_differences(gate, kind, gated):
    g = np.random.default_rng(3)
    x, i, h0, dh, dhT = g.normal(size=(4, 2)), g.normal(size=(4, 2)) if gated else None, g.normal(size=2), g.normal(size=(4, 2)), g.normal(size=2)
    z = g.normal(size=(4, 2)) if gate != "log" else -g.uniform(0.1, 2, size=(4, 2))
    A, b = (0.3 * g.normal(size=2), 0.3 * g.normal(size=2)) if gate != "log" else (np.zeros(2), np.zeros(2))

    def value():
        h, _, S = R.scan(x, z, i, A, b, h0, gate, -5.0, kind)
        return (h * dh).sum() + (S * dhT).sum()

    d = R.scan_grads(x, z, i, A, b, h0, dh, dhT, gate, -5.0, kind)
    for v, n in ((x, "x"), (z, "z"), (h0, "h0")) + (((i, "i"),) if gated else ()) + (((A, "A"), (b, "b")) if gate != "log" else ()):
        _differences(value, v, d[n])


def test_conv_by_hand():
    x, hist = np.array([[1.0], [2.0], [3.0]]), np.array([[10.0], [20.0]])
    y, tail = R.conv(x, hist, np.array([[100.0, 10.0, 1.0]]), 0.5, act="none")
    assert np.allclose(y[:, 0], [1201.5, 2012.5, 123.5]) and np.allclose(tail[:, 0], [2, 3])
    y, tail = R.conv(x[:1], hist, np.array([[0.0, 0.0, 1.0]]), 0.0)
    assert np.allclose(y, 1 / (1 + np.exp(-1.0))) and np.allclose(tail[:, 0], [20, 1])
    y, _ = R.conv(np.array([[3.0, 4.0]]), np.zeros((1, 2)), np.array([[0.0, 1.0]] * 2), 0.0, act="none", norm=2, eps=0.0)
    assert np.allclose(y, [[0.6, 0.8]])


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("norm", [0, 2])
@pytest.mark.parametrize("T", [0, 1, 5])
def test_conv_differences(act, norm, T):
    g = np.random.default_rng(4)
    K, D = 3, 4
    x, hist, w, b = g.normal(size=(T, D)), g.normal(size=(K - 1, D)), g.normal(size=(D, K)), g.normal(size=D)
    dy, dtail = g.normal(size=(T, D)), g.normal(size=(K - 1, D))

    def value():
        y, tail = R.conv(x, hist, w, b, act, norm, 0.01)
        return (y * dy).sum() + (tail * dtail).sum()

    d = R.conv_grads(x, hist, w, b, dy, dtail, act, norm, 0.01)
    for v, n in ((x, "x"), (hist, "hist"), (w, "w"), (b, "b")):
        _differences(value, v, d[n])


def test_block_norm_by_hand():
    r, n = R.block_norm(np.array([[3.0, 4.0]]), np.array([[1.0, 1.0]]), np.zeros(1), 2.0, np.array([1.0, 2.0]), np.ones(2), 0.0)
    k = 1 / np.sqrt(12.5)
    assert np.allclose(r, [[1 + 3 * k, 1 + 8 * k]])
    assert np.allclose(n, r / np.sqrt((r ** 2).mean()))


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_block_norm_differences(gate, post, pre):
    g = np.random.default_rng(5)
    T, D = 3, 4
    y, r, s = g.normal(size=(T, D)), g.normal(size=(T, D)), g.normal(size=D)
    gt = {"none": None, "channel": g.normal(size=(T, D)), "token": g.normal(size=T)}[gate]
    wp, wn = g.normal(size=D) if post else None, g.normal(size=D) if pre else None
    dr, dn = g.normal(size=(T, D)), g.normal(size=(T, D))

    def value():
        a, n = R.block_norm(y, r, gt, s, wp, wn, 0.01)
        return (a * dr).sum() + (0.0 if n is None else (n * dn).sum())

    d = R.block_norm_grads(y, r, gt, s, wp, wn, dr, dn, 0.01)
    for v, n in ((y, "y"), (r, "r"), (s, "scale"), (gt, "gate"), (wp, "post"), (wn, "pre")):
        if v is not None:
            _differences(value, v, d[n])
