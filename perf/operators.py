"""Cases and plain forms of the operators beside Kimi Delta Attention: linear attention with a decay per head
(prompts, gradients, single tokens), copies between the slots of a state pool, and rotary positions.

  fwd   S_t = e^{g_t} S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t       over whole sequences (packed, [T, heads, d])
  bwd   the gradients of fwd: q, k, v, g and the initial state, from dL/do and dL/dS_T
  step  one token of every sequence, the states updated in place in the slots of a pool
  copy  slot-to-slot copies of a pool applied in the order given: forks, compaction, clearing
  rope  the rotation of pairs of channels by position * frequency, applied to q and k

`own` chooses between the plain forms (elementary torch operations in fp32, sums of log-decays and angles in fp64)
and the framework's calls.  `exact` evaluates the definitions token by token in fp64.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_C = 64  # chunk of the plain form


# ----------------------------------------------------------------------------------------------- cases
def listed():
    lin = dict(hq=0, hk=0, hv=0, decay="token", state=True)  # 0: as many as there are heads
    return [
        # one short fp32 prompt, the smallest prefill: latency counts
        dict(lin, name="fwd_f32_T256_H2_d64", op="fwd", dtype="f32", h=2, dk=64, dv=64, n=1, lo=256, hi=256, len_seed=0, state=False),
        # one 4096-token prompt, the prefill of a request
        dict(lin, name="fwd_bf16_T4096_H32_d128", op="fwd", dtype="bf16", h=32, dk=128, dv=128, n=1, lo=4096, hi=4096, len_seed=0, state=False),
        # a ragged batch of 32 prompts with states in and out, the throughput of a prefill server
        dict(lin, name="fwd_bf16_varlen32_H32_d128", op="fwd", dtype="bf16", h=32, dk=128, dv=128, n=32, lo=512, hi=8192, len_seed=3),
        # a small fp32 gradient, as a numerical check of a training run takes it
        dict(lin, name="bwd_f32_T257_H2_d64", op="bwd", dtype="f32", h=2, dk=64, dv=64, n=1, lo=257, hi=257, len_seed=0),
        # a training step's sequence with a fixed decay per head
        dict(lin, name="bwd_bf16_T4096_H32_d128", op="bwd", dtype="bf16", h=32, dk=128, dv=128, n=1, lo=4096, hi=4096, len_seed=0, decay="head", state=False),
        # packed documents of odd lengths, narrow values, q and k shared by groups of four heads
        dict(lin, name="bwd_bf16_varlen12_H32_g8_dv64", op="bwd", dtype="bf16", h=32, hq=8, hk=8, dk=128, dv=64, n=12, lo=700, hi=5000, len_seed=5),
        # one token of one sequence: the latency of decoding
        dict(op="step", name="step_bf16_N1_H32_d128", dtype="bf16", h=32, hq=0, hk=0, hv=0, dk=128, dv=128, n=1, slots=8, decay="token"),
        # one token of each of 256 sequences in a larger pool
        dict(op="step", name="step_bf16_N256_H32_d128", dtype="bf16", h=32, hq=0, hk=0, hv=0, dk=128, dv=128, n=256, slots=300, decay="token"),
        # one prompt's state forked into four continuations
        dict(op="copy", name="copy_fork4_H32_d128", h=32, d=128, slots=8, pairs=4, kind="fork"),
        # a pool of 300 slots compacted after a third of its sequences ended
        dict(op="copy", name="copy_compact300_H32_d128", h=32, d=128, slots=300, pairs=150, kind="compact"),
        # the decoded tokens of 256 sequences at positions up to a million, every channel rotated
        dict(op="rope", name="rope_bf16_T256_H32_d128", dtype="bf16", t=256, hq=32, hk=32, d=128, rot=128, layout="half", top=1 << 20, inverse=False),
        # the prompts of a prefill batch, a part of the channels, neighbouring pairs
        dict(op="rope", name="rope_bf16_T131071_H32_d128_r64", dtype="bf16", t=131071, hq=32, hk=8, d=128, rot=64, layout="interleaved", top=131072, inverse=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "fwd", "bwd", "step", "copy", "rope"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("fwd", "bwd"):
        h = rng.choice([1, 2, 3, 6, 8, 12, 32])
        shared = rng.choice([0, 0, 0, 1])
        div = rng.choice([x for x in range(1, h + 1) if h % x == 0]) if shared else 0
        n = _log_int(rng, 1, 32)
        most = 100000 * 32 if dtype == "bf16" else 1 << 19
        if op == "bwd":
            most = 30000 * 32 if dtype == "bf16" else 1 << 18
        hi = max(1, min(8192, most // (h * n)))
        hi = _log_int(rng, min(hi, 33), hi)
        lo = _log_int(rng, 1, hi)
        shared_qk = rng.choice([True, False])  # heads of q and k, or of k and v, serve several states each
        return dict(op=op, dtype=dtype, h=h, hq=div if shared_qk else 0, hk=div, hv=0 if shared_qk else div, dk=rng.choice([64, 128]),
                    dv=rng.choice([64, 128]), n=n, lo=lo, hi=hi, len_seed=rng.randrange(1 << 20),
                    decay=rng.choice(["token", "token", "head", "none"]), state=rng.choice([True, False]))
    if op == "step":
        h = rng.choice([1, 3, 8, 32])
        n = _log_int(rng, 1, 256)
        div = rng.choice([0, 0, 1])
        return dict(op=op, dtype=dtype, h=h, hq=div, hk=div, hv=0, dk=rng.choice([64, 128]), dv=rng.choice([64, 128]), n=n,
                    slots=n + rng.randrange(0, 40), decay=rng.choice(["token", "head", "none"]))
    if op == "copy":
        slots = _log_int(rng, 4, 256)
        return dict(op=op, h=rng.choice([1, 3, 8, 32]), d=rng.choice([64, 128]), slots=slots, pairs=_log_int(rng, 1, max(1, slots // 2)),
                    kind=rng.choice(["fork", "compact", "mixed"]))
    d = rng.choice([64, 80, 128, 192])
    return dict(op=op, dtype=dtype, t=_log_int(rng, 1, 100000), hq=rng.choice([1, 8, 24, 32]), hk=rng.choice([1, 4, 8]), d=d,
                rot=rng.choice([r for r in (32, 40, 64, 128) if r <= d]), layout=rng.choice(["half", "interleaved"]), top=_log_int(rng, 2048, 1 << 20),
                inverse=rng.choice([False, True]))


def _lengths(c):
    g = torch.Generator().manual_seed(7919 + c["len_seed"])
    return [int(x) for x in torch.randint(c["lo"], c["hi"] + 1, (c["n"],), generator=g)]


def _heads(c):
    return tuple(c[x] or c["h"] for x in ("hq", "hk", "hv"))


# ----------------------------------------------------------------------------------------------- inputs
def _unit(shape, gen, dt):
    x = torch.randn(shape, generator=gen, device="cuda")
    return (x / x.norm(dim=-1, keepdim=True)).to(dt)


def _decay(kind, rows, h, gen):
    """Log-decays as a gate -rate_h softplus(x) gives them, rates from 1e-3 to 0.3 a token; or one rate per head."""
    rate = torch.exp(torch.rand((h,), generator=gen, device="cuda") * (math.log(0.3) - math.log(1e-3)) + math.log(1e-3))
    if kind == "none":
        return None
    if kind == "head":
        return -rate
    return -rate * torch.nn.functional.softplus(torch.randn((rows, h), generator=gen, device="cuda"))


def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    if c["op"] in ("fwd", "bwd"):
        dt, (hq, hk, hv), h, n = _DT[c["dtype"]], _heads(c), c["h"], c["n"]
        lens = _lengths(c)
        T = sum(lens)
        s["q"], s["k"] = _unit((T, hq, c["dk"]), gen, dt), _unit((T, hk, c["dk"]), gen, dt)
        s["v"] = torch.randn((T, hv, c["dv"]), generator=gen, device="cuda").to(dt)
        s["g"] = _decay(c["decay"], T, h, gen)
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["state"] = torch.randn((n, h, c["dk"], c["dv"]), generator=gen, device="cuda") if c["state"] else None
        if c["op"] == "bwd":
            s["grad_o"] = torch.randn((T, h, c["dv"]), generator=gen, device="cuda").to(dt)
            s["grad_state"] = torch.randn((n, h, c["dk"], c["dv"]), generator=gen, device="cuda") if c["state"] else None
        # token of each place of each chunk (T where there is none) and the chunks' sequences
        at = [torch.full((-(-x // _C) * _C,), T, dtype=torch.int64) for x in lens]
        for a, b, x in zip(at, cu, lens):
            a[:x] = torch.arange(b, b + x)
        s["at"] = torch.cat(at).view(-1, _C).cuda()
        s["seq"] = torch.repeat_interleave(torch.arange(n), torch.tensor([-(-x // _C) for x in lens])).cuda()
    elif c["op"] == "step":
        dt, (hq, hk, hv), h, n = _DT[c["dtype"]], _heads(c), c["h"], c["n"]
        s["q"], s["k"] = _unit((n, hq, c["dk"]), gen, dt), _unit((n, hk, c["dk"]), gen, dt)
        s["v"] = torch.randn((n, hv, c["dv"]), generator=gen, device="cuda").to(dt)
        s["g"] = _decay(c["decay"], n, h, gen)
        s["pool"] = torch.randn((c["slots"], h, c["dk"], c["dv"]), generator=gen, device="cuda")
        s["slots"] = torch.randperm(c["slots"], generator=gen, device="cuda")[:n].to(torch.int32)
    elif c["op"] == "copy":
        S, P = c["slots"], c["pairs"]
        s["pool"] = torch.randn((S, c["h"], c["d"], c["d"]), generator=gen, device="cuda")
        perm = torch.randperm(S, generator=gen, device="cuda")
        if c["kind"] == "fork":  # one state to P others (as many as there are)
            dst = perm[1:P + 1]
            src = perm[:1].expand(dst.numel())
        elif c["kind"] == "compact":  # the last slots move into holes before them
            dst = torch.sort(perm[:P]).values
            src = torch.arange(S - P, S, device="cuda")
        else:  # chains of copies, cleared slots (-1 as source) and unused entries (-1 as target)
            src = torch.randint(-1, S, (P,), generator=gen, device="cuda")
            dst = torch.randint(-1, S, (P,), generator=gen, device="cuda")
        s["src"], s["dst"] = src.to(torch.int32).contiguous(), dst.to(torch.int32).contiguous()
        # the same for the plain form, which copies all at once: the slot whose first contents each slot ends with
        last = list(range(S))
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            if b >= 0:
                last[b] = last[a] if a >= 0 else -1
        s["dst_at_once"] = torch.tensor([i for i in range(S) if last[i] != i], dtype=torch.int64, device="cuda")
        s["src_at_once"] = torch.tensor([last[i] for i in range(S) if last[i] != i], dtype=torch.int64, device="cuda")
    else:
        dt = _DT[c["dtype"]]
        s["q"] = torch.randn((c["t"], c["hq"], c["d"]), generator=gen, device="cuda").to(dt)
        s["k"] = torch.randn((c["t"], c["hk"], c["d"]), generator=gen, device="cuda").to(dt)
        s["positions"] = torch.randint(0, c["top"], (c["t"],), generator=gen, device="cuda").to(torch.int32)
        s["freqs"] = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])  # radians a position, on the host
        s["freqs_cuda"] = s["freqs"].cuda()
    return s


# ----------------------------------------------------------------------------------------------- plain forms
def _chunks(x, at, h):
    """[T, heads, d] -> [h, chunks, C, d] in fp32, zeros in the places behind a sequence's end, shared heads repeated."""
    x = torch.cat((x, x.new_zeros((1,) + x.shape[1:])))[at].float()
    return x.permute(2, 0, 1, 3).repeat_interleave(h // x.shape[2], 0)


def _log_decays(s, h):
    """Cumulative log-decays inside the chunks, and over the chunks up to each one's end, in fp64."""
    at, g = s["at"], s["g"]
    if g is None:
        g = torch.zeros((h,), device=at.device)
    T = s["q"].shape[0]
    g = g.double().expand(T, h)
    g = torch.cat((g, g.new_zeros((1, h))))[at].permute(2, 0, 1)
    G = g.cumsum(-1)
    return G, G[..., -1].cumsum(-1)


def _across(P, first, to, frm, keep):
    """exp(P[to] - P[frm]) where `keep`, 0 elsewhere: how much of what leaves chunk `frm` reaches chunk `to`."""
    d = P[..., to, None] - P[..., None, frm]
    return torch.where(keep, torch.exp(torch.where(keep, d, torch.zeros_like(d))), torch.zeros_like(d)).float()


def _entering(s, U, P, h, n):
    """States entering every chunk, and the final ones, from the chunks' own sums U."""
    seq, nc = s["seq"], U.shape[1]
    i = torch.arange(nc, device=seq.device)
    same = seq[:, None] == seq[None, :]
    Pz = torch.cat((torch.zeros_like(P[:, :1]), P), -1)  # up to each chunk's first token
    M = _across(Pz, 0, i, i + 1, same & (i[:, None] > i[None, :]))
    flat = U.reshape(h, nc, -1)
    S = M @ flat
    ns = torch.arange(n, device=seq.device)
    begin, end = torch.searchsorted(seq, ns), torch.searchsorted(seq, ns, right=True)
    last = _across(Pz, 0, end, i + 1, ns[:, None] == seq[None, :]) @ flat
    if s["state"] is not None:
        S0 = s["state"].permute(1, 0, 2, 3).reshape(h, n, -1)
        S = S + torch.exp(Pz[:, i] - Pz[:, begin[seq]]).float()[..., None] * S0[:, seq]
        last = last + torch.exp(Pz[:, end] - Pz[:, begin]).float()[..., None] * S0
    return S.view(U.shape), last.view(h, n, *U.shape[2:]), Pz, begin, end


def _rows(x, s, heads, dt):
    """[h, chunks, C, ...] back to token rows, summed over the heads that share one."""
    T = s["q"].shape[0]
    x = x.permute(1, 2, 0, *range(3, x.dim()))
    out = x.new_empty((T + 1,) + x.shape[2:])
    out[s["at"].reshape(-1)] = x.reshape((-1,) + x.shape[2:])
    out = out[:T]
    if out.shape[1] != heads:
        out = out.view(T, heads, out.shape[1] // heads, *out.shape[2:]).sum(2)
    return out.to(dt)


def _plain_fwd(s):
    c = s["case"]
    h, n = c["h"], c["n"]
    q, k, v = (_chunks(s[x], s["at"], h) for x in "qkv")
    G, P = _log_decays(s, h)
    low = torch.ones((_C, _C), dtype=torch.bool, device=q.device).tril()
    D = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill_(~low, -math.inf)).float()
    U = (k * torch.exp(G[..., -1:] - G).float()[..., None]).transpose(-1, -2) @ v
    S, last, _, _, _ = _entering(s, U, P, h, n)
    o = ((q @ k.transpose(-1, -2)) * D) @ v + torch.exp(G).float()[..., None] * (q @ S)
    return _rows(o, s, h, s["q"].dtype), last.permute(1, 0, 2, 3).contiguous()


def _plain_bwd(s):
    c = s["case"]
    h, n, (hq, hk, hv), dt = c["h"], c["n"], _heads(c), s["q"].dtype
    q, k, v, do = (_chunks(s[x], s["at"], h) for x in ("q", "k", "v", "grad_o"))
    G, P = _log_decays(s, h)
    low = torch.ones((_C, _C), dtype=torch.bool, device=q.device).tril()
    D = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill_(~low, -math.inf)).float()
    f, e = torch.exp(G[..., -1:] - G).float()[..., None], torch.exp(G).float()[..., None]
    U = (k * f).transpose(-1, -2) @ v
    S, last, Pz, begin, end = _entering(s, U, P, h, n)
    # the adjoint of the state leaving each chunk, from the chunks' own sums R
    R = (q * e).transpose(-1, -2) @ do
    seq, nc = s["seq"], U.shape[1]
    i = torch.arange(nc, device=seq.device)
    keep = (seq[:, None] == seq[None, :]) & (i[:, None] > i[None, :])
    flat = R.reshape(h, nc, -1)
    L = _across(Pz, 0, i, i + 1, keep).transpose(-1, -2) @ flat
    dS0 = torch.exp(torch.where(seq[None, :] == torch.arange(n, device=seq.device)[:, None], Pz[:, None, i] - Pz[:, begin, None], -math.inf)).float() @ flat
    dS0 = dS0.view(h, n, *U.shape[2:])
    if s["grad_state"] is not None:
        dST = s["grad_state"].permute(1, 0, 2, 3)
        L = L + torch.exp(Pz[:, end[seq]] - Pz[:, i + 1]).float()[..., None] * dST.reshape(h, n, -1)[:, seq]
        dS0 = dS0 + torch.exp(Pz[:, end] - Pz[:, begin]).float()[..., None, None] * dST
    L = L.view(U.shape)
    qk, dA = q @ k.transpose(-1, -2), (do @ v.transpose(-1, -2)) * D
    q_in, k_out = e * (do @ S.transpose(-1, -2)), f * (v @ L.transpose(-1, -2))
    dq, dk = dA @ k + q_in, dA.transpose(-1, -2) @ q + k_out
    dv = (qk * D).transpose(-1, -2) @ do + f * (k @ L)
    grads = {"q": _rows(dq, s, hq, dt), "k": _rows(dk, s, hk, dt), "v": _rows(dv, s, hv, dt)}
    if s["g"] is not None:
        # dL/dG inside each chunk; g_t is part of every G_r, r >= t, of its chunk
        W = qk * dA
        ko = (k * k_out).double().sum(-1)
        dG = W.double().sum(-1) - W.double().sum(-2) + (q * q_in).double().sum(-1) - ko
        dG[..., -1] += ko.sum(-1) + torch.exp(G[..., -1]) * (S * L).flatten(2).double().sum(-1)
        dg = _rows(dG.flip(-1).cumsum(-1).flip(-1), s, h, torch.float64)
        grads["g"] = (dg if s["g"].dim() == 2 else dg.sum(0)).float()
    if s["state"] is not None:
        grads["initial_state"] = dS0.permute(1, 0, 2, 3).contiguous()
    return grads


def _per_head(x, h):
    return x.repeat_interleave(h // x.shape[1], 1)


def _plain_step(s):
    h = s["case"]["h"]
    q, k, v = (_per_head(s[x], h).float() for x in "qkv")
    at = s["slots"].long()
    S = s["pool"][at]
    if s["g"] is not None:
        S = S * torch.exp(s["g"])[..., None, None]
    S = S + k[..., :, None] * v[..., None, :]
    s["pool"][at] = S
    return (q[..., :, None] * S).sum(-2).to(s["q"].dtype), s["pool"]


def _plain_copy(s):
    src, pool = s["src_at_once"], s["pool"]
    moved = pool[src.clamp_min(0)] * (src >= 0)[:, None, None, None]
    pool[s["dst_at_once"]] = moved
    return pool


def _plain_rope(s):
    c = s["case"]
    rot = c["rot"]
    turns = s["positions"].double()[:, None] * s["freqs_cuda"]
    cos, sin = torch.cos(turns).float()[:, None], torch.sin(turns).float()[:, None]
    if c["inverse"]:
        sin = -sin

    def turn(x):
        y = x.float()
        if c["layout"] == "half":
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        return torch.cat((r, y[..., rot:]), -1).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from linear_attention_kda_gb300 import kda
        if op == "fwd":
            return kda.linear_chunk_fwd(s["q"], s["k"], s["v"], s["g"], cu_seqlens=s["cu_seqlens"], initial_state=s["state"], output_final_state=True)
        if op == "bwd":
            return kda.linear_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["grad_o"], cu_seqlens=s["cu_seqlens"], initial_state=s["state"],
                                        grad_final_state=s["grad_state"], state_grad=s["state"] is not None)
        if op == "step":
            return kda.linear_recurrent_step(s["q"], s["k"], s["v"], s["g"], s["pool"], state_indices=s["slots"]), s["pool"]
        if op == "copy":
            return kda.state_copy(s["pool"], s["src"], s["dst"])
        c = s["case"]
        return kda.rope(s["q"], s["k"], s["positions"], s["freqs"], layout=c["layout"], inverse=c["inverse"])
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "copy": _plain_copy, "rope": _plain_rope}[op](s)


def work(case):
    c, op = case, case["op"]
    if op in ("fwd", "bwd"):
        T, h, (hq, hk, hv) = sum(_lengths(c)), c["h"], _heads(c)
        b, dk, dv = (2 if c["dtype"] == "bf16" else 4), c["dk"], c["dv"]
        rows = T * (hq * dk + hk * dk + hv * dv)
        states = c["n"] * h * dk * dv * 4
        g = {"token": T * h * 4, "head": h * 4, "none": 0}[c["decay"]]
        if op == "fwd":
            return {"bytes": b * (rows + T * h * dv) + g + states * (2 if c["state"] else 1), "flops": T * h * 4 * dk * dv}
        return {"bytes": b * (2 * rows + T * h * dv) + 2 * g + states * (3 if c["state"] else 0), "flops": T * h * 10 * dk * dv}
    if op == "step":
        hq, hk, hv = _heads(c)
        b = 2 if c["dtype"] == "bf16" else 4
        state = c["n"] * c["h"] * c["dk"] * c["dv"]
        rows = c["n"] * (hq * c["dk"] + hk * c["dk"] + hv * c["dv"] + c["h"] * c["dv"])
        return {"bytes": 8 * state + b * rows, "flops": 5 * state}
    if op == "copy":
        slot = c["h"] * c["d"] * c["d"] * 4
        n = min(c["pairs"], c["slots"] - 1)
        return {"bytes": slot * (n + (1 if c["kind"] == "fork" else n)), "flops": 0}
    b = 2 if c["dtype"] == "bf16" else 4
    return {"bytes": 2 * b * c["t"] * (c["hq"] + c["hk"]) * c["d"], "flops": 3 * c["t"] * (c["hq"] + c["hk"]) * c["rot"]}


# ----------------------------------------------------------------------------------------------- definitions in 64 bits
def _steps(x, s, h, per_token=True):
    """[T, heads, ...] as fp64 [longest, n, h, ...]: token t of every sequence (zeros behind its end)."""
    lens = _lengths(s["case"])
    x = x.double().repeat_interleave(h // x.shape[1], 1)
    out = x.new_zeros((max(lens), len(lens)) + x.shape[1:])
    for n, (a, m) in enumerate(zip(s["cu_seqlens"].tolist(), lens)):
        out[:m, n] = x[a:a + m]
    return out


def _packed(x, s):
    return torch.cat([x[:m, n] for n, m in enumerate(_lengths(s["case"]))])


def _exact_lin(s):
    c = s["case"]
    h, n, T = c["h"], c["n"], s["q"].shape[0]
    # (steps x states) fp64 values touched; leave out what would take too long
    if max(_lengths(c)) * (20e-6 + n * h * c["dk"] * c["dv"] * 8 * 16 / 4e12) > 15:
        return None
    q, k, v = (_steps(s[x], s, h) for x in "qkv")
    g = torch.zeros((h,), device="cuda") if s["g"] is None else s["g"]
    a = torch.exp(_steps(g.double().expand(T, h).contiguous(), s, h))[..., None, None]  # 1 behind a sequence's end
    S = torch.zeros((n, h, c["dk"], c["dv"]), dtype=torch.float64, device="cuda")
    if s["state"] is not None:
        S = s["state"].double()
    steps = q.shape[0]
    if c["op"] == "fwd":
        o = v.new_empty((steps, n, h, c["dv"]))
        for t in range(steps):
            S = torch.addcmul(S * a[t], k[t][..., None], v[t][..., None, :])
            o[t] = (q[t][..., None, :] @ S)[..., 0, :]
        return _packed(o, s), S
    do = _steps(s["grad_o"], s, h)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(steps):
        S = torch.addcmul(S * a[t], k[t][..., None], v[t][..., None, :])
        dq[t] = (S @ do[t][..., None])[..., 0]
    L = torch.zeros_like(S) if s["grad_state"] is None else s["grad_state"].double()
    whole = (S * L).sum((-1, -2))
    for t in range(steps - 1, -1, -1):  # L: the adjoint of S_t
        L = torch.addcmul(L, q[t][..., None], do[t][..., None, :])
        dk[t] = (L @ v[t][..., None])[..., 0]
        dv[t] = (k[t][..., None, :] @ L)[..., 0, :]
        L = L * a[t]
    hq, hk, hv = _heads(c)

    def shared(x, heads):
        x = _packed(x, s)
        return x.view(x.shape[0], heads, h // heads, x.shape[-1]).sum(2)

    grads = {"q": shared(dq, hq), "k": shared(dk, hk), "v": shared(dv, hv)}
    if s["g"] is not None:
        # g_t scales all that passes from before t to t or later: the outputs' share of it less the keys' own
        dg = ((q * dq).sum(-1) - (k * dk).sum(-1)).flip(0).cumsum(0).flip(0) + whole
        dg = _packed(dg, s)
        grads["g"] = dg if s["g"].dim() == 2 else dg.sum(0)
    if s["state"] is not None:
        grads["initial_state"] = L
    return grads


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op in ("fwd", "bwd"):
        return _exact_lin(s)
    if op == "step":
        h, pool, at = c["h"], s["pool"].double(), s["slots"].long()
        q, k, v = (_per_head(s[x], h).double() for x in "qkv")
        a = torch.ones((1, h), dtype=torch.float64, device="cuda") if s["g"] is None else torch.exp(s["g"].double())
        S = a.expand(c["n"], h)[..., None, None] * pool[at] + torch.einsum("nhi,nhj->nhij", k, v)
        pool[at] = S
        return torch.einsum("nhi,nhij->nhj", q, S), pool
    if op == "copy":
        pool = s["pool"].double()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            if b >= 0:
                pool[b] = pool[a] if a >= 0 else 0.0
        return pool
    rot, half = c["rot"], c["rot"] // 2
    turned = torch.polar(torch.ones((c["t"], half), dtype=torch.float64, device="cuda"), s["positions"].double()[:, None] * s["freqs_cuda"])
    if c["inverse"]:
        turned = turned.conj()
    out = []
    for x in (s["q"], s["k"]):
        y = x.double()
        first, second = (y[..., :half], y[..., half:rot]) if c["layout"] == "half" else (y[..., 0:rot:2], y[..., 1:rot:2])
        z = torch.complex(first, second) * turned[:, None]
        if c["layout"] == "half":
            y[..., :half], y[..., half:rot] = z.real, z.imag
        else:
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        out.append(y)
    return tuple(out)
