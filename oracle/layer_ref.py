"""fp64 definitions of what stands around a recurrence in a layer, one sequence at a time, in NumPy: the gated
recurrence over channels, the short causal convolution, the norms around a block, and their gradients."""
import numpy as np


def sigmoid(y):
    e = np.exp(-np.abs(y))
    return np.where(y >= 0, 1.0, e) / (1.0 + e)


def decay(z, A, b, gate, g_min):
    """Log-decay g of the logits z, dg/dz and dg/dA (A: log-scale, b: bias, per channel)."""
    if gate == "log":
        return z, np.ones_like(z), np.zeros_like(z)
    y, r = z + b, np.exp(A)
    if gate == "lower_bound":
        s, n = sigmoid(r * y), sigmoid(-r * y)
        return g_min * s, g_min * s * n * r, g_min * s * n * r * y
    s, n = sigmoid(y), sigmoid(-y)
    if gate == "sigmoid":
        return -r * s, -r * s * n, -r * s
    soft = np.maximum(y, 0.0) + np.log1p(np.exp(-np.abs(y)))
    return -r * soft, -r * s, -r * soft


def input_factor(g, kind):
    """c and dc/dg."""
    a = np.exp(g)
    if kind == "none":
        return np.ones_like(g), np.zeros_like(g)
    if kind == "complement":
        return -np.expm1(g), -a
    c = np.sqrt(np.maximum(-np.expm1(2 * g), 0.0))
    return c, np.where(c > 0, -a * a / np.where(c > 0, c, 1.0), 0.0)


def scan(x, z, i, A, b, h0, gate="softplus", g_min=-5.0, input_scale="none"):
    """(h [T, D], the state before each token [T, D], the final state [D])."""
    g, _, _ = decay(z, A, b, gate, g_min)
    a, c = np.exp(g), input_factor(g, input_scale)[0]
    u = c * x if i is None else c * sigmoid(i) * x
    h, before, S = np.zeros_like(x), np.zeros_like(x), h0.copy()
    for t in range(x.shape[0]):
        before[t] = S
        S = np.where(a[t] == 0, 0.0, a[t] * S) + u[t]
        h[t] = S
    return h, before, S


def scan_grads(x, z, i, A, b, h0, dh, dhT, gate="softplus", g_min=-5.0, input_scale="none", magnitudes=False):
    """Gradients as a dict x, z, i, A, b (sums over tokens), h0.  With magnitudes, of absolute values: what the
    roundings of an element's terms scale with."""
    f = np.abs if magnitudes else (lambda v: v)
    g, gz, gA = decay(z, A, b, gate, g_min)
    a = np.exp(g)
    c, slope = input_factor(g, input_scale)
    _, before, _ = scan(f(x), z, i, A, b, f(h0), gate, g_min, input_scale)
    s, n = (np.ones_like(x), np.zeros_like(x)) if i is None else (sigmoid(i), sigmoid(-i))
    lam, L = np.zeros_like(x), f(dhT).copy()
    for t in range(x.shape[0] - 1, -1, -1):
        lam[t] = f(dh[t]) + L
        L = np.where(a[t] == 0, 0.0, a[t] * lam[t])
    dg = (a * before + f(slope) * s * f(x)) * lam
    dz, dA = dg * f(gz), dg * f(gA)
    return {"x": c * s * lam, "z": dz, "i": c * f(x) * s * n * lam, "A": dA.sum(0), "b": dz.sum(0), "h0": L}


def conv_rows(x, hist):
    return np.concatenate((hist, x))


def conv(x, hist, w, b, act="silu", norm=0, eps=1e-6):
    """(y [T, D], the new history [K - 1, D])."""
    p, s, _, r = _conv_parts(x, hist, w, b, act, norm, eps)
    rows = conv_rows(x, hist)
    return s * r, rows[rows.shape[0] - w.shape[1] + 1:]


def _conv_parts(x, hist, w, b, act, norm, eps):
    """Sums p, activations s, ds/dp, and 1 / the heads' norms (1 without) per channel."""
    rows, K, T = conv_rows(x, hist), w.shape[1], x.shape[0]
    p = np.zeros_like(x) + b
    for j in range(K):
        p = p + w[:, j] * rows[j:j + T]
    if act == "none":
        s, ds = p, np.ones_like(p)
    else:
        q, n = sigmoid(p), sigmoid(-p)
        s, ds = p * q, q * (1.0 + p * n)
    r = np.ones_like(p)
    if norm:
        r = 1.0 / np.sqrt(np.square(s).reshape(T, x.shape[1] // norm, norm).sum(-1) + eps)
        r = np.repeat(r, norm, axis=1)
    return p, s, ds, r


def conv_grads(x, hist, w, b, dy, dtail, act="silu", norm=0, eps=1e-6, magnitudes=False):
    """Gradients as a dict x, w, b, hist; with magnitudes, of absolute values (the terms' sizes)."""
    f = np.abs if magnitudes else (lambda v: v)
    rows, K, T = conv_rows(x, hist), w.shape[1], x.shape[0]
    _, s, ds, r = _conv_parts(x, hist, w, b, act, norm, eps)
    d = f(dy)
    if norm:
        y = f(s * r)
        dot = np.repeat((d * y).reshape(T, x.shape[1] // norm, norm).sum(-1), norm, axis=1)
        d = r * (d + y * dot if magnitudes else d - y * dot)
    d = d * f(ds)
    drows = np.zeros_like(rows)
    dw = np.zeros_like(w)
    for j in range(K):
        drows[j:j + T] += f(w[:, j]) * d
        dw[:, j] = (d * f(rows[j:j + T])).sum(0)
    drows[T:] += f(dtail)
    return {"x": drows[K - 1:], "hist": drows[:K - 1], "w": dw, "b": d.sum(0)}


def block_norm(y, r, gate, scale, post, pre, eps=1e-6):
    """(r', n).  y None: no block; gate: logits [T, D], [T] or None; post, pre: weights [D] or None (no norm)."""
    if y is not None:
        p = y if post is None else post * y / np.sqrt(np.square(y).mean(-1, keepdims=True) + eps)
        s = 1.0 if gate is None else sigmoid(gate if gate.ndim == 2 else gate[:, None])
        r = r + scale * s * p
    return r, (None if pre is None else pre * r / np.sqrt(np.square(r).mean(-1, keepdims=True) + eps))


def block_norm_grads(y, r, gate, scale, post, pre, dr, dn, eps=1e-6, magnitudes=False):
    """Gradients as a dict y, r, gate, post, pre, scale ([D] each for the last three); with magnitudes, the sizes of
    the terms."""
    f = np.abs if magnitudes else (lambda v: v)
    sub = (lambda u, v: u + v) if magnitudes else (lambda u, v: u - v)
    out, d = {}, f(dr)
    if pre is not None:
        rn, _ = block_norm(y, r, gate, scale, post, None, eps)
        k = 1.0 / np.sqrt(np.square(rn).mean(-1, keepdims=True) + eps)
        rh, e = f(rn * k), f(dn) * f(pre)
        out["pre"] = (f(dn) * rh).sum(0)
        d = d + k * sub(e, rh * (e * rh).mean(-1, keepdims=True))
    out["r"] = d
    if y is None:
        return out
    s = np.ones((1, 1)) if gate is None else sigmoid(gate if gate.ndim == 2 else gate[:, None])
    k = np.ones((1, 1)) if post is None else 1.0 / np.sqrt(np.square(y).mean(-1, keepdims=True) + eps)
    w = np.ones(y.shape[1]) if post is None else post
    yh = f(y) * k
    p = f(w) * yh
    out["scale"] = (d * s * p).sum(0)
    ds = d * f(scale)
    if gate is not None:
        dg = ds * p * s * (1.0 - s)
        out["gate"] = dg if gate.ndim == 2 else dg.sum(-1)
    dp = ds * s
    out["post"] = (dp * yh).sum(0)
    e = dp * f(w)
    out["y"] = e if post is None else k * sub(e, yh * (e * yh).mean(-1, keepdims=True))
    return out
