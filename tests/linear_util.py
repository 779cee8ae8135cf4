"""Helpers of the linear-attention tests: seeded batches, their fp64 results and elementwise error bounds.

Every bound is n * u * (sum of the magnitudes of an element's terms), the sum taken from the oracle on absolute
values, plus half a step of the output's type.  u = 2^-24 for what is computed in fp32; where the tensor-core path
rounds an operand to bf16 once, that operand's terms are off by 2^-8 of themselves at most (EPS_BF16)."""
import numpy as np
import torch

from oracle import linear_ref as R

U32, EPS_BF16 = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
LENS = [130, 0, 1, 63, 64, 65, 127, 128, 129, 300]


def batch(lens, H, dk, dv, dtype, seed, *, Hq=None, Hk=None, Hv=None, decay="token", state=True):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)  # noqa: E731
    d = {"q": unit(rn(T, Hq or H, dk)).to(DT[dtype]), "k": unit(rn(T, Hk or H, dk)).to(DT[dtype]),
         "v": rn(T, Hv or H, dv).to(DT[dtype]), "grad_o": rn(T, H, dv).to(DT[dtype])}
    rate = torch.exp(torch.linspace(np.log(2e-3), np.log(0.7), H))
    d["g"] = None if decay == "none" else -rate if decay == "head" else -rate * torch.nn.functional.softplus(rn(T, H))
    d["initial_state"] = rn(N, H, dk, dv) if state else None
    d["grad_final_state"] = rn(N, H, dk, dv) if state else None
    d["cu_seqlens"] = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32)
    d.update(H=H, lens=list(lens), scale=0.75)
    return d


def to(d, dev):
    return {n: x.to(dev) if isinstance(x, torch.Tensor) else x for n, x in d.items()}


def _np(d):
    H, T = d["H"], d["q"].shape[0]
    x = {n: R.repeat_heads(d[n].double().numpy(), H) for n in ("q", "k", "v")}
    g = torch.zeros(H) if d["g"] is None else d["g"]
    x["g"] = g.double().expand(T, H).numpy()
    x["do"] = d["grad_o"].double().numpy()
    return x


def _states(d, name):
    N, H = len(d["lens"]), d["H"]
    x = d[name]
    return np.zeros((N, H, d["q"].shape[2], d["v"].shape[2])) if x is None else x.double().numpy()


def forward_ref(d, magnitudes=False):
    """(o, final states) in fp64; on absolute values with magnitudes=True."""
    x, S0 = _np(d), _states(d, "initial_state")
    f = np.abs if magnitudes else (lambda y: y)
    o, S = np.zeros(x["do"].shape), np.zeros_like(S0)
    at = 0
    for n, m in enumerate(d["lens"]):
        s = slice(at, at + m)
        o[s], S[n] = R.forward(f(x["q"][s]), f(x["k"][s]), f(x["v"][s]), x["g"][s], f(S0[n]), d["scale"])
        at += m
    return o, S


def backward_ref(d, magnitudes=False):
    """Gradients in fp64 (dict), g's per token under "g_tokens" and, on absolute values, what its sums inside
    one chunk (of 64 or 128 tokens) can hold under "g_terms"."""
    x, S0, dS = _np(d), _states(d, "initial_state"), _states(d, "grad_final_state")
    f = np.abs if magnitudes else (lambda y: y)
    parts = {n: [] for n in ("q", "k", "v", "g", "terms")}
    dS0 = np.zeros_like(S0)
    at = 0
    for n, m in enumerate(d["lens"]):
        s = slice(at, at + m)
        r = R.backward(f(x["q"][s]), f(x["k"][s]), f(x["v"][s]), x["g"][s], f(S0[n]), f(x["do"][s]), f(dS[n]), d["scale"])
        for name in ("q", "k", "v", "g"):
            parts[name].append(r[name])
        if magnitudes:
            per = (np.abs(x["q"][s]) * r["q"]).sum(-1) + (np.abs(x["k"][s]) * r["k"]).sum(-1)
            terms = np.zeros_like(per)
            for b in range(0, m, 128):
                terms[b:b + 128] = per[b:b + 128].sum(0) + r["g"][b:b + 128].max(0)
            parts["terms"].append(terms)
        dS0[n] = r["initial_state"]
        at += m
    cat = lambda name, like: np.concatenate(parts[name]) if parts[name] else like  # noqa: E731
    out = {n: R.sum_heads(cat(n, None), d[n].shape[1]) for n in ("q", "k", "v")}
    out["g_tokens"] = cat("g", None)
    if magnitudes:
        out["g_terms"] = cat("terms", None)
    out["initial_state"] = dS0
    return out


def ops(d):
    """Roundings an fp32 term can go through: sums over channels and tokens of a chunk and over the chunks before
    it, the decay's argument (up to 104, three roundings) and its exponential."""
    return 2 * (128 + max(d["q"].shape[2], d["v"].shape[2])) + 4 * (max(d["lens"], default=0) // 64 + 1) + 3 * 104 + 40


def close(name, got, want, terms, per_term, step):
    """|got - want| <= per_term * terms + step * |want| elementwise (and nothing but numbers where want is one)."""
    got, want = got.double().cpu().numpy(), np.asarray(want)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bound = per_term * terms + step * np.abs(want) + 1e-37
    bad = ~(np.abs(got - want) <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isnan(got), np.inf, np.abs(got - want) / bound)), got.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} out of bounds, worst at {i}: {got[i]} for {want[i]}, bound {bound[i]}")
