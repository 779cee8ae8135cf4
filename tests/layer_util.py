"""Helpers of the tests of the gated recurrence, the short convolution and the block norm: seeded inputs, fp64 results
and elementwise error bounds.

A bound is n u (sum of the magnitudes of an element's terms) plus half a step of the output's type, u = 2^-24 and n the
roundings that a term goes through; the sums of magnitudes come from the oracle on absolute values."""
import numpy as np
import torch

from oracle import layer_ref as R

U32 = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
LENS = [130, 0, 1, 63, 64, 65, 127, 128, 129, 300]
GATES, INPUTS = ("lower_bound", "softplus", "sigmoid", "log"), ("none", "complement", "norm")


def cu(lens):
    return torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32)


def to(d, dev="cuda"):
    return {n: x.to(dev) if isinstance(x, torch.Tensor) else x for n, x in d.items()}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def close(name, got, want, terms, n, half):
    got, want, terms = f64(got), np.asarray(want), np.asarray(terms)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bound = n * U32 * terms + half * np.abs(want) + 1e-37
    bad = ~(np.abs(got - want) <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isnan(got), np.inf, np.abs(got - want) / bound)), got.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} out of bounds, worst at {i}: {got[i]} for {want[i]}, bound {bound[i]}")


# ---------------------------------------------------------------- scan
def scan_batch(lens, D, dtype, seed, *, gate="softplus", input_scale="none", gated=True, params=True, state=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    T, N = sum(lens), len(lens)
    rate = torch.exp(torch.linspace(np.log(1e-3), np.log(0.7), D))
    z = rn(T, D)
    d = dict(lens=list(lens), D=D, dtype=dtype, gate=gate, input_scale=input_scale, A_log=None, dt_bias=None)
    if gate == "log":
        z = -rate * torch.nn.functional.softplus(z)
    elif params:
        d["A_log"], d["dt_bias"] = (0.3 * rn(D) if gate == "lower_bound" else torch.log(rate)), 0.5 * rn(D)
    d.update(x=rn(T, D).to(DT[dtype]), z=z.to(DT[dtype]), input_gate=rn(T, D).to(DT[dtype]) if gated else None, grad_h=rn(T, D).to(DT[dtype]),
             initial_state=rn(N, D) if state else None, grad_final_state=rn(N, D) if state else None, cu_seqlens=cu(lens))
    return d


def _scan_args(d):
    zero = np.zeros(d["D"])
    x, z, i = f64(d["x"]), f64(d["z"]), f64(d["input_gate"])
    A, b = (zero if d[k] is None else f64(d[k]) for k in ("A_log", "dt_bias"))
    st = lambda k: np.zeros((len(d["lens"]), d["D"])) if d[k] is None else f64(d[k])  # noqa: E731
    return x, z, i, A, b, st("initial_state"), st("grad_final_state")


def scan_ref(d, magnitudes=False):
    """(h, final states, checkpoints [T // 64 + N, D] with NaN in rows that hold none)"""
    x, z, i, A, b, h0, _ = _scan_args(d)
    f = np.abs if magnitudes else (lambda v: v)
    h, last = np.zeros_like(x), np.zeros_like(h0)
    keep = np.full((x.shape[0] // 64 + len(d["lens"]), d["D"]), np.nan)
    at = 0
    for n, m in enumerate(d["lens"]):
        s = slice(at, at + m)
        h[s], before, last[n] = R.scan(f(x[s]), z[s], None if i is None else i[s], A, b, f(h0[n]), d["gate"], -5.0, d["input_scale"])
        k = -(-m // 64)
        keep[at // 64 + n:at // 64 + n + k] = before[::64]
        at += m
    return h, last, keep


def scan_grads_ref(d, magnitudes=False):
    x, z, i, A, b, h0, dhT = _scan_args(d)
    dh = f64(d["grad_h"])
    out = {"x": np.zeros_like(x), "z": np.zeros_like(x), "input_gate": np.zeros_like(x), "A_log": np.zeros(d["D"]), "dt_bias": np.zeros(d["D"]),
           "initial_state": np.zeros_like(h0)}
    at = 0
    for n, m in enumerate(d["lens"]):
        s = slice(at, at + m)
        r = R.scan_grads(x[s], z[s], None if i is None else i[s], A, b, h0[n], dh[s], dhT[n], d["gate"], -5.0, d["input_scale"], magnitudes)
        out["x"][s], out["z"][s], out["input_gate"][s], out["initial_state"][n] = r["x"], r["z"], r["i"], r["h0"]
        out["A_log"] += r["A"]
        out["dt_bias"] += r["b"]
        at += m
    return out


def scan_roundings(d):
    """A state's term goes through two roundings a token; its decay's exponent, at most 104 where anything is left, is a sum
    over the tokens of log-decays with a few roundings each (relative to a sum of one sign) and goes through one
    exponential per run of tokens; and a few dozen for the gates themselves (logits up to 6: their exponentials are off by up to 10 u)."""
    return 2 * max(d["lens"], default=0) + 4 * 104 + 100


# ---------------------------------------------------------------- convolution
def conv_batch(lens, D, K, dtype, seed, *, act="silu", norm=0, bias=True, state=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    T, N, dt = sum(lens), len(lens), DT[dtype]
    return dict(lens=list(lens), D=D, K=K, dtype=dtype, activation=act, norm_dim=norm, x=rn(T, D).to(dt), weight=rn(D, K) / K ** 0.5,
                bias=0.3 * rn(D) if bias else None, grad_y=rn(T, D).to(dt), initial_state=rn(N, K - 1, D).to(dt) if state else None,
                grad_final_state=rn(N, K - 1, D).to(dt) if state else None, cu_seqlens=cu(lens))


def _conv_args(d):
    hist = np.zeros((len(d["lens"]), d["K"] - 1, d["D"]))
    st = lambda k: hist if d[k] is None else f64(d[k])  # noqa: E731
    return f64(d["x"]), f64(d["weight"]), (np.zeros(d["D"]) if d["bias"] is None else f64(d["bias"])), st("initial_state"), st("grad_final_state")


def conv_ref(d):
    x, w, b, hist, _ = _conv_args(d)
    y, tail, at = np.zeros_like(x), np.zeros_like(hist), 0
    for n, m in enumerate(d["lens"]):
        y[at:at + m], tail[n] = R.conv(x[at:at + m], hist[n], w, b, d["activation"], d["norm_dim"])
        at += m
    return y, tail


def conv_sizes(d):
    """Bound of |error of y| / u: the sum's magnitude through the activation (slope at most 1.1) and the norm."""
    x, w, b, hist, _ = _conv_args(d)
    out, at = np.zeros_like(x), 0
    for n, m in enumerate(d["lens"]):
        p, s, ds, r = R._conv_parts(x[at:at + m], hist[n], w, b, d["activation"], d["norm_dim"], 1e-6)
        mag = R._conv_parts(np.abs(x[at:at + m]), np.abs(hist[n]), np.abs(w), np.abs(b), "none", 0, 1e-6)[0]
        e = 1.1 * mag + np.abs(s)
        if d["norm_dim"]:  # y = s r, dr / r = -r^2 sum s ds
            y = np.abs(s * r)
            dot = (y * (e * r)).reshape(m, d["D"] // d["norm_dim"], d["norm_dim"]).sum(-1)
            e = e * r + y * (np.repeat(dot, d["norm_dim"], axis=1) + 1.0)
        out[at:at + m] = e
        at += m
    return out


def conv_grads_ref(d, magnitudes=False):
    x, w, b, hist, dtail = _conv_args(d)
    dy = f64(d["grad_y"])
    out = {"x": np.zeros_like(x), "weight": np.zeros_like(w), "bias": np.zeros(d["D"]), "initial_state": np.zeros_like(hist)}
    at = 0
    for n, m in enumerate(d["lens"]):
        s = slice(at, at + m)
        r = R.conv_grads(x[s], hist[n], w, b, dy[s], dtail[n], d["activation"], d["norm_dim"], magnitudes=magnitudes)
        out["x"][s], out["initial_state"][n] = r["x"], r["hist"]
        out["weight"] += r["w"]
        out["bias"] += r["b"]
        at += m
    return out


# ---------------------------------------------------------------- block norm
def norm_batch(T, D, dtype, seed, *, res=None, gate="channel", post=True, pre=True, vec=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    dt, rt = DT[dtype], DT[res or dtype]
    return dict(T=T, D=D, dtype=dtype, res=res or dtype, y=rn(T, D).to(dt), residual=(2 * rn(T, D)).to(rt),
                gate=None if gate == "none" else rn(T, D).to(dt) if gate == "channel" else rn(T).to(dt),
                scale=0.2 + 0.8 * torch.rand((D,), generator=g) if vec else 0.5, post_weight=1 + 0.2 * rn(D) if post else None,
                pre_weight=1 + 0.2 * rn(D) if pre else None, grad_residual=rn(T, D).to(rt), grad_normed=rn(T, D).to(dt) if pre else None)


def norm_args(d):
    s = f64(d["scale"]) if isinstance(d["scale"], torch.Tensor) else d["scale"]
    return f64(d["y"]), f64(d["residual"]), f64(d["gate"]), s, f64(d["post_weight"]), f64(d["pre_weight"])


def norm_options(d):
    return dict(post_weight=d["post_weight"], pre_weight=d["pre_weight"], scale=d["scale"], post_norm=d["post_weight"] is not None,
                pre_norm=d["pre_weight"] is not None)
