"""Cases and plain forms of what stands around a recurrence in a layer: the gated linear recurrence over channels,
the short causal convolution in front of it, and the norms before and after a block with its gate and residual scale.

  scan_fwd   h_t = a_t h_{t-1} + c(a_t) sigmoid(i_t) x_t per channel, over whole sequences (packed, [T, D])
  scan_bwd   its gradients: x, z (the decay's logit), i, A_log, dt_bias and the initial state, from dL/dh and dL/dh_T
  scan_step  one token of every sequence, the states updated in place in the slots of a pool
  conv_fwd   y_t = N(act(bias + sum_j w_j x_{t-K+1+j})), act SiLU or none, N an L2 norm over each head or none
  conv_bwd   its gradients: x, weight, bias and the initial history
  conv_step  one token of every sequence, the histories shifted in place in the slots of a pool
  norm_fwd   r' = r + s sigmoid(gate) RMSNorm(y),  n = RMSNorm(r')
  norm_bwd   its gradients: y, r, gate, both norms' weights and s

`own` chooses between the plain forms (elementary torch operations in fp32, sums over tokens and scans in fp64) and the
framework's calls.  `exact` evaluates the definitions in fp64: token by token, or by differentiating them.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_C = 64  # tokens from one checkpoint of a scan to the next, and the plain form's chunks


# ----------------------------------------------------------------------------------------------- cases
def listed():
    scan = dict(dtype="bf16", n=1, len_seed=0, gated=True, params=True, state=True)
    conv = dict(dtype="bf16", n=1, len_seed=0, K=4, act="silu", bias=False, state=True)
    norm = dict(dtype="bf16", res="bf16", gate="channel", vec_scale=True, post=True, pre=True)
    return [
        # one short fp32 sequence of odd sizes, the smallest scan: latency counts
        dict(scan, name="scan_fwd_f32_T257_D96", op="scan_fwd", dtype="f32", d=96, lo=257, hi=257, gate="softplus", cscale="none", gated=False, state=False, keep=False),
        # one 4096-token prompt through a gated recurrent layer, as wide as 32 heads of 128
        dict(scan, name="scan_fwd_bf16_T4096_D4096", op="scan_fwd", d=4096, lo=4096, hi=4096, gate="sigmoid", cscale="norm", state=False, keep=False),
        # one very long sequence of few channels: the scan's own latency
        dict(scan, name="scan_fwd_bf16_T131072_D256", op="scan_fwd", d=256, lo=131072, hi=131072, gate="lower_bound", cscale="complement", gated=False, keep=False),
        # the forward pass of a training batch of 32 ragged sequences, checkpoints kept
        dict(scan, name="scan_fwd_bf16_varlen32_D4096", op="scan_fwd", d=4096, n=32, lo=512, hi=8192, len_seed=3, gate="softplus", cscale="norm", keep=True),
        # the gradients of packed documents of odd lengths
        dict(scan, name="scan_bwd_bf16_varlen12_D4096", op="scan_bwd", d=4096, n=12, lo=700, hi=5000, len_seed=5, gate="sigmoid", cscale="norm"),
        # one decoded token of each of 256 sequences
        dict(scan, name="scan_step_bf16_N256_D4096", op="scan_step", d=4096, n=256, slots=300, gate="softplus", cscale="complement"),
        # q's or k's convolution in front of a prefill of 32 ragged prompts, SiLU and the L2 norm of each head
        dict(conv, name="conv_fwd_bf16_varlen32_H32_d128", op="conv_fwd", d=4096, head=128, n=32, lo=512, hi=8192, len_seed=3),
        # the same in a training step of one 4096-token sequence
        dict(conv, name="conv_bwd_bf16_T4096_H32_d128", op="conv_bwd", d=4096, head=128, lo=4096, hi=4096, state=False),
        # v's convolution of one decoded token of 64 sequences
        dict(conv, name="conv_step_bf16_N64_D4096", op="conv_step", d=4096, head=0, n=64, slots=70, bias=True),
        # one decoded token between two blocks
        dict(norm, name="norm_fwd_bf16_T1_D4096", op="norm_fwd", t=1, d=4096, gate="channel"),
        # a prefill batch between two blocks, the residual stream in fp32
        dict(norm, name="norm_fwd_bf16_T65535_D4096", op="norm_fwd", res="f32", t=65535, d=4096),
        # a training step's gradients between two blocks
        dict(norm, name="norm_bwd_bf16_T16384_D4096", op="norm_bwd", t=16384, d=4096),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_lengths(rng, most):
    """(n, lo, hi) of a ragged batch of at most `most` tokens."""
    most = max(1, most)
    n = _log_int(rng, 1, min(64, most))
    hi = _log_int(rng, 1, max(1, min(131072, most // n)))
    return n, rng.choice([0, 1, hi, _log_int(rng, 1, hi)]), hi


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "conv_fwd", "conv_bwd", "conv_step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, dtype=dtype)
    if op.startswith("scan"):
        d = rng.choice([_log_int(rng, 1, 8192), 8 * _log_int(rng, 1, 1024), rng.choice([256, 1024, 4096])])
        gate = rng.choice(["softplus", "sigmoid", "lower_bound", "log"])
        c.update(d=d, gate=gate, cscale=rng.choice(["none", "complement", "norm"]), gated=rng.choice([True, True, False]),
                 params=gate != "log" and rng.choice([True, True, False]))
        if op == "scan_step":
            n = _log_int(rng, 1, 1024)
            return dict(c, n=n, slots=n + rng.randrange(0, 40), state=True)
        most = min(131072, (1 << 28 if op == "scan_fwd" else 1 << 26) // (d * (2 if dtype == "f32" else 1)))
        n, lo, hi = _draw_lengths(rng, most)
        c.update(n=n, lo=lo, hi=hi, len_seed=rng.randrange(1 << 20), state=rng.choice([True, False]))
        if op == "scan_fwd":
            c["keep"] = rng.choice([True, False])
        return c
    if op.startswith("conv"):
        head = rng.choice([0, 0, 32, 64, 128, 256])
        d = head * _log_int(rng, 1, 8192 // head) if head else rng.choice([_log_int(rng, 1, 8192), 8 * _log_int(rng, 1, 1024)])
        c.update(d=d, head=head, K=rng.choice([2, 3, 4, 4]), act=rng.choice(["silu", "silu", "none"]), bias=rng.choice([True, False]))
        if op == "conv_step":
            n = _log_int(rng, 1, 1024)
            return dict(c, n=n, slots=n + rng.randrange(0, 40), state=True)
        most = min(131072, (1 << 28 if op == "conv_fwd" else 1 << 24) // (d * (2 if dtype == "f32" else 1)))
        n, lo, hi = _draw_lengths(rng, most)
        return dict(c, n=n, lo=lo, hi=hi, len_seed=rng.randrange(1 << 20), state=rng.choice([True, False]))
    d = rng.choice([_log_int(rng, 16, 8192), 8 * _log_int(rng, 2, 1024), rng.choice([1024, 2048, 4096, 7168])])
    res = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
    post, pre = rng.choice([(True, True), (True, True), (True, False), (False, True)])
    most = max(1, min(131072, (1 << 27 if op == "norm_fwd" else 1 << 25) // (d * (2 if dtype == "f32" else 1))))
    return dict(c, res=res, d=d, t=_log_int(rng, 1, most), gate=rng.choice(["channel", "channel", "token", "none"]),
                vec_scale=rng.choice([True, False]), post=post, pre=pre)


def _lengths(c):
    g = torch.Generator().manual_seed(104729 + c["len_seed"])
    return [c["hi"]] + [int(x) for x in torch.randint(c["lo"], c["hi"] + 1, (c["n"] - 1,), generator=g)]


def _starts(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu


# ----------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    dt, d = _DT[c["dtype"]], c["d"]

    def rn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if not c["op"].startswith("norm"):
        step = c["op"].endswith("step")
        lens = [1] * c["n"] if step else _lengths(c)
        cu, T = _starts(lens), sum(lens)
        s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["x"] = rn(T, d).to(dt)
    if c["op"].startswith("scan"):
        # decays from 1e-3 to 0.5 a token, as trained recurrent layers spread them over their channels
        rate = torch.exp(torch.rand((d,), generator=gen, device="cuda") * (math.log(0.5) - math.log(1e-3)) + math.log(1e-3))
        z = rn(T, d)
        s["A_log"] = s["dt_bias"] = None
        if c["gate"] == "log":
            z = -rate * torch.nn.functional.softplus(z)
        elif c["gate"] == "lower_bound":
            z = z - 2.0
        if c["params"]:
            s["A_log"] = 0.3 * rn(d) if c["gate"] == "lower_bound" else torch.log(rate)
            s["dt_bias"] = 0.5 * rn(d)
        s["z"] = z.to(dt)
        s["input_gate"] = rn(T, d).to(dt) if c["gated"] else None
        if step:
            s["pool"] = rn(c["slots"], d)
        else:
            s["state"] = rn(c["n"], d) if c["state"] else None
            # token of each place of each chunk (T where there is none), the chunks' sequences and rows in the list of checkpoints
            at = [torch.full((-(-m // _C) * _C,), T, dtype=torch.int64) for m in lens]
            for a, b, m in zip(at, cu, lens):
                a[:m] = torch.arange(b, b + m)
            s["at"] = torch.cat(at).view(-1, _C).cuda()
            nc = torch.tensor([-(-m // _C) for m in lens])
            s["seq"] = torch.repeat_interleave(torch.arange(c["n"]), nc).cuda()
            rows = [torch.arange(b // _C + n, b // _C + n + int(k)) for n, (b, k) in enumerate(zip(cu, nc))]
            s["rows"] = torch.cat(rows).cuda()
            if c["op"] == "scan_bwd":
                s["grad_h"] = rn(T, d).to(dt)
                s["grad_state"] = rn(c["n"], d) if c["state"] else None
                s["checkpoints"] = torch.zeros((T // _C + c["n"], d), device="cuda")
                _plain_scan_fwd(s)  # a training step has them from its forward pass
            else:
                s["checkpoints"] = torch.zeros((T // _C + c["n"], d), device="cuda") if c["keep"] else None
    elif c["op"].startswith("conv"):
        K = c["K"]
        s["weight"] = rn(d, K) / math.sqrt(K)
        s["bias"] = 0.2 * rn(d) if c["bias"] else None
        if step:
            s["pool"] = rn(c["slots"], K - 1, d).to(dt)
        else:
            s["state"] = rn(c["n"], K - 1, d).to(dt) if c["state"] else None
            if c["op"] == "conv_bwd":
                s["grad_y"] = rn(T, d).to(dt)
                s["grad_state"] = rn(c["n"], K - 1, d).to(dt) if c["state"] else None
            # rows of the histories and tokens of all sequences one after the other: each sequence's first, each token's first tap
            first = torch.tensor(cu[:-1]) + (K - 1) * torch.arange(c["n"])
            s["taps"] = (torch.arange(T) + (K - 1) * torch.repeat_interleave(torch.arange(c["n"]), torch.tensor(lens))).cuda()
            s["hist"] = (first[:, None] + torch.arange(K - 1)).cuda()
            s["tail"] = (first[:, None] + torch.tensor(lens)[:, None] + torch.arange(K - 1)).cuda()
    else:
        t, rt = c["t"], _DT[c["res"]]
        s["y"] = rn(t, d).to(dt)
        s["residual"] = (2.0 * rn(t, d)).to(rt)
        s["gate"] = None if c["gate"] == "none" else rn(t, d).to(dt) if c["gate"] == "channel" else rn(t).to(dt)
        s["scale"] = 0.2 + 0.8 * torch.rand((d,), generator=gen, device="cuda") if c["vec_scale"] else 0.5
        s["post_weight"] = 1.0 + 0.2 * rn(d) if c["post"] else None
        s["pre_weight"] = 1.0 + 0.2 * rn(d) if c["pre"] else None
        if c["op"] == "norm_bwd":
            s["grad_residual"] = rn(t, d).to(rt)
            s["grad_normed"] = rn(t, d).to(dt) if c["pre"] else None
    if c["op"].endswith("step"):
        s["slots"] = torch.randperm(c["slots"], generator=gen, device="cuda")[:c["n"]].to(torch.int32)
    return s


# ----------------------------------------------------------------------------------------------- plain forms
_GMIN = -5.0


def _decay(s, z):
    """Log-decay g of logits z, and what its derivatives need: sigmoid of the gate's argument, that argument, e^A."""
    kind = s["case"]["gate"]
    if kind == "log":
        return z, None, None, None
    zb = z if s["dt_bias"] is None else z + s["dt_bias"]
    eA = torch.ones_like(zb[:1]) if s["A_log"] is None else torch.exp(s["A_log"])
    if kind == "lower_bound":
        sg = torch.sigmoid(eA * zb)
        return _GMIN * sg, sg, zb, eA
    sg = torch.sigmoid(zb)
    if kind == "sigmoid":
        return -eA * sg, sg, zb, eA
    return -eA * (torch.clamp_min(zb, 0.0) + torch.log1p(torch.exp(-zb.abs()))), sg, zb, eA


def _inject(s, g):
    """c(a) for a = e^g."""
    kind = s["case"]["cscale"]
    return None if kind == "none" else -torch.expm1(g) if kind == "complement" else torch.sqrt(-torch.expm1(2.0 * g))


def _terms(s):
    """a and u of h = a h + u, per token in fp64: a decay near 1 acts over thousands of tokens."""
    g = _decay(s, s["z"].float())[0].double()
    u = s["x"].double()
    if s["input_gate"] is not None:
        u = u * torch.sigmoid(s["input_gate"].float())
    c = _inject(s, g)
    return torch.exp(g), (u if c is None else u * c)


def _doubling(a, u, dim, size):
    """a, u become the decay and the value of the recurrence h = a h + u from the first of `size` steps along dim."""
    k = 1
    while k < size:
        here, before = (slice(None),) * dim + (slice(k, None),), (slice(None),) * dim + (slice(0, size - k),)
        u_new, a_new = u.clone(), a.clone()
        u_new[here] += a[here] * u[before]
        a_new[here] *= a[before]
        a, u, k = a_new, u_new, 2 * k
    return a, u


def _entering(A, U, seq, state, n):
    """States entering every chunk, and those behind each sequence's last, from the chunks' decays A and values U."""
    nc, D = U.shape
    if nc:
        first = torch.ones_like(seq, dtype=torch.bool)
        first[1:] = seq[1:] != seq[:-1]
        start = torch.zeros_like(U) if state is None else state[seq].to(U.dtype)
        U = torch.where(first[:, None], A * start + U, U)
        A = torch.where(first[:, None], torch.zeros_like(A), A)
        _, U = _doubling(A, U, 0, nc)
        S = torch.where(first[:, None], start, torch.cat((U[:1], U[:-1])))
    else:
        S = U
    last = torch.zeros((n, D), device=U.device) if state is None else state.clone()
    if nc:
        end = torch.ones_like(first)
        end[:-1] = first[1:]
        last[seq[end]] = U[end].to(last.dtype)
    return S, last


def _padded(x, at, fill):
    return torch.cat((x, x.new_full((1,) + x.shape[1:], fill)))[at]


def _packed(x, at, T):
    out = x.new_empty((T + 1, x.shape[-1]))
    out[at.reshape(-1)] = x.reshape(-1, x.shape[-1])
    return out[:T]


def _plain_scan_fwd(s):
    c, at, T = s["case"], s["at"], s["x"].shape[0]
    a, u = _terms(s)
    A, U = _doubling(_padded(a, at, 1.0), _padded(u, at, 0.0), 1, _C)
    S, last = _entering(A[:, -1], U[:, -1], s["seq"], s["state"], c["n"])
    if s["checkpoints"] is not None:
        s["checkpoints"][s["rows"]] = S.float()
    return _packed(U + A * S[:, None], at, T).to(s["x"].dtype), last, s["checkpoints"]


def _plain_scan_bwd(s):
    c, at, T, dt = s["case"], s["at"], s["x"].shape[0], s["x"].dtype
    a, u = _terms(s)
    ap = _padded(a, at, 1.0)
    A, U = _doubling(ap, _padded(u, at, 0.0), 1, _C)
    S, _ = _entering(A[:, -1], U[:, -1], s["seq"], s["state"], c["n"])
    h = _packed(torch.cat((S[:, None], U[:, :-1] + A[:, :-1] * S[:, None]), 1), at, T)  # h_{t-1}
    # M_t = a_t (dh_t + M_{t+1}) is the adjoint of h_{t-1}: the same recurrence backwards
    dh = s["grad_h"].double()
    A, U = _doubling(ap.flip(1), _padded(a * dh, at, 0.0).flip(1), 1, _C)
    gs = s["grad_state"]
    M, last = _entering(A[:, -1].flip(0), U[:, -1].flip(0), s["seq"].flip(0), gs, c["n"])
    M = M.flip(0)
    M = _packed(torch.cat((M[:, None], U[:, :-1] + A[:, :-1] * M[:, None]), 1).flip(1), at, T)  # M_{t+1}
    lam = dh + M
    z = s["z"].float()
    g, sg, zb, eA = _decay(s, z)
    g = g.double()
    ci, x = _inject(s, g), s["x"].float()
    si = None if s["input_gate"] is None else torch.sigmoid(s["input_gate"].float())
    xi = x if si is None else x * si
    dg = a * h * lam
    if ci is not None:
        # dc/dg: -a of 1 - a, -a^2 / c of sqrt(1 - a^2)
        dg = dg - (a if c["cscale"] == "complement" else a * a / ci) * xi * lam
        lam = ci * lam
    out = {"x": (lam if si is None else si * lam).to(dt)}
    if si is not None:
        out["input_gate"] = (x * si * (1.0 - si) * lam).to(dt)
    if sg is None:
        out["z"] = dg.to(dt)
    else:
        dz = dg * (_GMIN * eA * sg * (1.0 - sg) if c["gate"] == "lower_bound" else -eA * sg * (1.0 - sg) if c["gate"] == "sigmoid" else -eA * sg)
        out["z"] = dz.to(dt)
        if c["params"]:
            out["A_log"] = ((dz * zb) if c["gate"] == "lower_bound" else dg * g).double().sum(0).float()
            out["dt_bias"] = dz.double().sum(0).float()
    if c["state"]:
        out["initial_state"] = last
    return out


def _plain_scan_step(s):
    a, u = _terms(s)
    at = s["slots"].long()
    h = (a * s["pool"][at] + u).float()
    s["pool"][at] = h
    return h.to(s["x"].dtype), s["pool"]


def _silu(c, v):
    return v if c["act"] == "none" else v * torch.sigmoid(v)


def _normed(c, v):
    """v and 1 / its heads' norms (1 where there is no norm)."""
    if not c["head"]:
        return v, None
    y = v.view(-1, c["d"] // c["head"], c["head"])
    r = torch.rsqrt((y * y).sum(-1, keepdim=True) + 1e-6)
    return (y * r).view_as(v), r


def _rows(s):
    """Histories and tokens of all sequences, one after the other."""
    x, K, n = s["x"], s["case"]["K"], s["case"]["n"]
    rows = x.new_zeros((x.shape[0] + n * (K - 1), x.shape[1]))
    if s["state"] is not None:
        rows[s["hist"]] = s["state"]
    rows[s["taps"] + K - 1] = x
    return rows


def _mix(s, rows, taps):
    pre = 0.0 if s["bias"] is None else s["bias"]
    for j in range(s["case"]["K"]):
        pre = pre + s["weight"][:, j] * rows[taps + j].float()
    return pre


def _plain_conv_fwd(s):
    c, rows = s["case"], _rows(s)
    y, _ = _normed(c, _silu(c, _mix(s, rows, s["taps"])))
    return y.to(s["x"].dtype), rows[s["tail"]]


def _plain_conv_bwd(s):
    c, rows, dt, K = s["case"], _rows(s), s["x"].dtype, s["case"]["K"]
    pre = _mix(s, rows, s["taps"])
    y, r = _normed(c, _silu(c, pre))
    d = s["grad_y"].float()
    if r is not None:
        dv, yv = d.view(r.shape[0], r.shape[1], -1), y.view(r.shape[0], r.shape[1], -1)
        d = (r * (dv - yv * (dv * yv).sum(-1, keepdim=True))).view_as(d)
    if c["act"] != "none":
        sg = torch.sigmoid(pre)
        d = d * sg * (1.0 + pre * (1.0 - sg))
    drows = torch.zeros(rows.shape, device="cuda")
    dw = []
    for j in range(K):
        drows[s["taps"] + j] += s["weight"][:, j] * d
        dw.append((d * rows[s["taps"] + j].float()).double().sum(0))
    if s["grad_state"] is not None:
        drows[s["tail"]] += s["grad_state"].float()
    out = {"x": drows[s["taps"] + K - 1].to(dt), "weight": torch.stack(dw, 1).float()}
    if c["bias"]:
        out["bias"] = d.double().sum(0).float()
    if c["state"]:
        out["initial_state"] = drows[s["hist"]].to(dt)
    return out


def _plain_conv_step(s):
    c, at = s["case"], s["slots"].long()
    rows = torch.cat((s["pool"][at], s["x"][:, None]), 1)
    pre = (rows.float() * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    s["pool"][at] = rows[:, 1:]
    return _normed(c, _silu(c, pre))[0].to(s["x"].dtype), s["pool"]


def _rms(v):
    return torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6)


def _gate_of(s):
    if s["gate"] is None:
        return None
    g = torch.sigmoid(s["gate"].float())
    return g if g.dim() == 2 else g[:, None]


def _plain_norm_fwd(s):
    c, y = s["case"], s["y"].float()
    if c["post"]:
        y = y * _rms(y) * s["post_weight"]
    g = _gate_of(s)
    r = s["residual"].float() + s["scale"] * (y if g is None else g * y)
    n = (r * _rms(r) * s["pre_weight"]).to(s["y"].dtype) if c["pre"] else None
    return r.to(s["residual"].dtype), n


def _plain_norm_bwd(s):
    c, y, g = s["case"], s["y"].float(), _gate_of(s)
    ry = _rms(y) if c["post"] else None
    p = y * ry * s["post_weight"] if c["post"] else y
    gp = p if g is None else g * p
    dr = s["grad_residual"].float()
    out = {}
    if c["pre"]:
        r = s["residual"].float() + s["scale"] * gp
        rr = _rms(r)
        dn, nh = s["grad_normed"].float(), r * rr
        out["pre_weight"] = (dn * nh).double().sum(0).float()
        dn = dn * s["pre_weight"]
        dr = dr + rr * (dn - nh * (dn * nh).mean(-1, keepdim=True))
    out["residual"] = dr.to(s["residual"].dtype)
    if c["vec_scale"]:
        out["scale"] = (dr * gp).double().sum(0).float()
    dgp = dr * s["scale"]
    if g is not None:
        dg = dgp * p * g * (1.0 - g)
        out["gate"] = (dg if s["gate"].dim() == 2 else dg.sum(-1)).to(s["gate"].dtype)
        dgp = dgp * g
    if c["post"]:
        yh = y * ry
        out["post_weight"] = (dgp * yh).double().sum(0).float()
        dgp = dgp * s["post_weight"]
        dgp = ry * (dgp - yh * (dgp * yh).mean(-1, keepdim=True))
    out["y"] = dgp.to(s["y"].dtype)
    return out


def run(state):
    s, c, op = state, state["case"], state["case"]["op"]
    if not own:
        return {"scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step, "conv_fwd": _plain_conv_fwd,
                "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step, "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}[op](s)
    from linear_attention_kda_gb300 import kda
    if op.startswith("scan"):
        how = dict(A_log=s["A_log"], dt_bias=s["dt_bias"], gate=c["gate"], input_scale=c["cscale"])
        if op == "scan_step":
            return kda.scan_step(s["x"], s["z"], s["input_gate"], s["pool"], state_indices=s["slots"], **how), s["pool"]
        if op == "scan_fwd":
            h, last = kda.scan_fwd(s["x"], s["z"], s["input_gate"], cu_seqlens=s["cu_seqlens"], initial_state=s["state"], output_final_state=True,
                                   checkpoints=s["checkpoints"], **how)
            return h, last, s["checkpoints"]
        return kda.scan_bwd(s["x"], s["z"], s["input_gate"], s["grad_h"], s["checkpoints"], cu_seqlens=s["cu_seqlens"],
                            grad_final_state=s["grad_state"], param_grads=c["params"], state_grad=c["state"], **how)
    if op.startswith("conv"):
        how = dict(activation=c["act"], norm_dim=c["head"])
        if op == "conv_step":
            return kda.short_conv_step(s["x"], s["weight"], s["bias"], s["pool"], state_indices=s["slots"], **how), s["pool"]
        if op == "conv_fwd":
            return kda.short_conv_fwd(s["x"], s["weight"], s["bias"], cu_seqlens=s["cu_seqlens"], initial_state=s["state"], output_final_state=True, **how)
        return kda.short_conv_bwd(s["x"], s["weight"], s["bias"], s["grad_y"], cu_seqlens=s["cu_seqlens"], initial_state=s["state"],
                                  grad_final_state=s["grad_state"], state_grad=c["state"], **how)
    how = dict(post_weight=s["post_weight"], pre_weight=s["pre_weight"], scale=s["scale"], post_norm=c["post"], pre_norm=c["pre"])
    if op == "norm_fwd":
        return kda.block_norm_fwd(s["y"], s["residual"], s["gate"], **how)
    return kda.block_norm_bwd(s["y"], s["residual"], s["gate"], s["grad_residual"], s["grad_normed"], **how)


def work(case):
    c, op, d, b = case, case["op"], case["d"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("norm"):
        t, e, r = c["t"], c["t"] * c["d"], 2 if c["res"] == "bf16" else 4
        gate = {"channel": e, "token": t, "none": 0}[c["gate"]] * b
        w = 4 * d * (c["post"] + c["pre"] + c["vec_scale"])
        if op == "norm_fwd":
            return {"bytes": e * (b + 2 * r + (b if c["pre"] else 0)) + gate + w, "flops": 14 * e}
        return {"bytes": e * (2 * b + 3 * r + (b if c["pre"] else 0)) + 2 * gate + 2 * w, "flops": 40 * e}
    step = op.endswith("step")
    T = c["n"] if step else sum(_lengths(c))
    if op.startswith("scan"):
        ins, st, w = 2 + c["gated"], c["n"] * d * 4, 8 * d * c["params"]
        kept = (T // _C + c["n"]) * d * 4
        if step:
            return {"bytes": T * d * b * (ins + 1) + 2 * st + w, "flops": 20 * T * d}
        if op == "scan_fwd":
            return {"bytes": T * d * b * (ins + 1) + st * (2 if c["state"] else 1) + w + (kept if c["keep"] else 0), "flops": 20 * T * d}
        return {"bytes": T * d * b * (2 * ins + 1) + st * (2 if c["state"] else 0) + 2 * w + kept, "flops": 45 * T * d}
    K, hist = c["K"], c["n"] * (c["K"] - 1) * d * b
    w = 4 * d * (K + c["bias"])
    if op == "conv_bwd":
        return {"bytes": 3 * T * d * b + hist * (3 if c["state"] else 0) + 2 * w, "flops": T * d * (6 * K + 20)}
    return {"bytes": 2 * T * d * b + hist * (2 if c["state"] else 1) + w, "flops": T * d * (2 * K + 8)}


# ----------------------------------------------------------------------------------------------- definitions in 64 bits
def _exact_gate(s, z, A, b):
    """a and c(a) from logits z, differentiable."""
    c = s["case"]
    if c["gate"] == "log":
        g = z
    else:
        y = z if b is None else z + b
        e = 1.0 if A is None else torch.exp(A)
        g = {"lower_bound": lambda: _GMIN * torch.sigmoid(e * y), "sigmoid": lambda: -e * torch.sigmoid(y),
             "softplus": lambda: -e * torch.nn.functional.softplus(y, threshold=1e9)}[c["gate"]]()
    return torch.exp(g), {"none": lambda: torch.ones_like(g), "complement": lambda: -torch.expm1(g),
                          "norm": lambda: torch.sqrt(-torch.expm1(2 * g))}[c["cscale"]]()


def _exact_scan(s):
    c, x, cu = s["case"], s["x"].double(), s["cu_seqlens"].tolist()
    T, d, lens = x.shape[0], c["d"], [b - a for a, b in zip(cu, cu[1:])]
    if max(lens) * (12e-6 + c["n"] * d * 8 * 6 / 4e12) * (2 if c["op"] == "scan_bwd" else 1) > 15:
        return None
    f64 = lambda v: None if v is None else v.double()  # noqa: E731
    z, A, b, i = (f64(s[k]) for k in ("z", "A_log", "dt_bias", "input_gate"))
    with torch.no_grad():
        a, cs = _exact_gate(s, z, A, b)
        u = cs * x if i is None else cs * torch.sigmoid(i) * x
    order = sorted(range(c["n"]), key=lambda n: -lens[n])
    start = torch.tensor([cu[n] for n in order], device="cuda")
    count = [sum(m > t for m in lens) for t in range(max(lens))]  # sequences with a token t: the first of `order`
    h = torch.zeros((c["n"], d), dtype=torch.float64, device="cuda") if s["state"] is None else s["state"].double()[order]
    before = torch.empty((T, d), dtype=torch.float64, device="cuda")
    keep = torch.zeros((T // _C + c["n"], d), dtype=torch.float64, device="cuda")
    rows = torch.tensor([cu[n] // _C + n for n in order], device="cuda")
    one = c["n"] == 1
    for t, m in enumerate(count):
        at = slice(cu[0] + t, cu[0] + t + 1) if one else start[:m] + t
        before[at] = h[:m]
        if t % _C == 0:
            keep[rows[:m] + t // _C] = h[:m]
        h[:m] = a[at] * h[:m] + u[at]
    if c["op"] == "scan_fwd":
        last = torch.empty_like(h)
        last[order] = h
        return a * before + u, last, (keep if s["checkpoints"] is not None else None)
    lam = torch.empty((T, d), dtype=torch.float64, device="cuda")
    dh = s["grad_h"].double()
    M = torch.zeros_like(h) if s["grad_state"] is None else s["grad_state"].double()[order]
    for t in range(len(count) - 1, -1, -1):
        m = count[t]
        at = slice(cu[0] + t, cu[0] + t + 1) if one else start[:m] + t
        v = dh[at] + M[:m]
        lam[at] = v
        M[:m] = a[at] * v
    # everything else is local to a token: d(sum lam (a h_{t-1} + c sigmoid(i) x)), some tokens at a time
    out = {"x": torch.empty_like(x), "z": torch.empty_like(x)}
    if i is not None:
        out["input_gate"] = torch.empty_like(x)
    if c["params"]:
        out["A_log"], out["dt_bias"] = (torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(2))
    block = max(1, (1 << 24) // d)
    for t0 in range(0, T, block):
        r = slice(t0, t0 + block)
        leaf = {"x": x[r], "z": z[r]}
        if i is not None:
            leaf["input_gate"] = i[r]
        if c["params"]:
            leaf["A_log"], leaf["dt_bias"] = A, b
        leaf = {k: v.detach().clone().requires_grad_() for k, v in leaf.items()}
        av, cv = _exact_gate(s, leaf["z"], leaf.get("A_log"), leaf.get("dt_bias"))
        uv = cv * leaf["x"] if i is None else cv * torch.sigmoid(leaf["input_gate"]) * leaf["x"]
        gr = torch.autograd.grad((lam[r] * (av * before[r] + uv)).sum(), list(leaf.values()))
        for k, v in zip(leaf, gr):
            if k in ("A_log", "dt_bias"):
                out[k] += v
            else:
                out[k][r] = v
    if c["state"]:
        out["initial_state"] = torch.empty_like(M)
        out["initial_state"][order] = M
    return out


def _exact_mix(c, rows, w, b):
    """The convolution, activation and norm of one sequence; rows: its history, then its tokens."""
    K, m = c["K"], rows.shape[0] - c["K"] + 1
    v = sum(w[:, j] * rows[j:j + m] for j in range(K))
    if b is not None:
        v = v + b
    if c["act"] != "none":
        v = torch.nn.functional.silu(v)
    if c["head"]:
        v = v.unflatten(-1, (-1, c["head"]))
        v = (v / torch.sqrt(v.square().sum(-1, keepdim=True) + 1e-6)).flatten(-2)
    return v


def _exact_conv(s):
    c, cu = s["case"], s["cu_seqlens"].tolist()
    K, d, T = c["K"], c["d"], s["x"].shape[0]
    f64 = dict(dtype=torch.float64, device="cuda")
    w, b = s["weight"].double(), None if s["bias"] is None else s["bias"].double()
    state = torch.zeros((c["n"], K - 1, d), **f64) if s["state"] is None else s["state"].double()
    if c["op"] == "conv_fwd":
        y, last = torch.empty((T, d), **f64), torch.empty((c["n"], K - 1, d), **f64)
        for n in range(c["n"]):
            rows = torch.cat((state[n], s["x"][cu[n]:cu[n + 1]].double()))
            y[cu[n]:cu[n + 1]] = _exact_mix(c, rows, w, b)
            last[n] = rows[rows.shape[0] - K + 1:]
        return y, last
    out = {"x": torch.empty((T, d), **f64), "weight": torch.zeros_like(w)}
    if c["bias"]:
        out["bias"] = torch.zeros(d, **f64)
    if c["state"]:
        out["initial_state"] = torch.empty((c["n"], K - 1, d), **f64)
    for n in range(c["n"]):
        rows = torch.cat((state[n], s["x"][cu[n]:cu[n + 1]].double())).requires_grad_()
        wl = w.clone().requires_grad_()
        leaves = [rows, wl] + ([b.clone().requires_grad_()] if c["bias"] else [])
        total = (_exact_mix(c, rows, wl, leaves[2] if c["bias"] else None) * s["grad_y"][cu[n]:cu[n + 1]].double()).sum()
        if s["grad_state"] is not None:
            total = total + (rows[rows.shape[0] - K + 1:] * s["grad_state"][n].double()).sum()
        gr = torch.autograd.grad(total, leaves)
        out["x"][cu[n]:cu[n + 1]] = gr[0][K - 1:]
        out["weight"] += gr[1]
        if c["bias"]:
            out["bias"] += gr[2]
        if c["state"]:
            out["initial_state"][n] = gr[0][:K - 1]
    return out


def _exact_norm(s):
    c = s["case"]
    f64 = lambda v: v.double() if isinstance(v, torch.Tensor) else v  # noqa: E731
    par = {k: f64(s[k]) for k in ("post_weight", "pre_weight", "scale")}
    rows = {k: s[k] for k in ("y", "residual", "gate") if s[k] is not None}

    def value(p, x):
        y = x["y"]
        if c["post"]:
            y = p["post_weight"] * y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6)
        if "gate" in x:
            g = torch.sigmoid(x["gate"])
            y = y * (g if g.dim() == 2 else g[:, None])
        r = x["residual"] + p["scale"] * y
        return r, (p["pre_weight"] * r / torch.sqrt(r.square().mean(-1, keepdim=True) + 1e-6) if c["pre"] else None)

    block = max(1, (1 << 24) // c["d"])
    whole = {k: torch.empty(v.shape, dtype=torch.float64, device="cuda") for k, v in rows.items()}
    sums = {k: torch.zeros_like(v) for k, v in par.items() if isinstance(v, torch.Tensor)}
    r_out, n_out = [], []
    for t0 in range(0, c["t"], block):
        at = slice(t0, t0 + block)
        x = {k: v[at].double() for k, v in rows.items()}
        if c["op"] == "norm_fwd":
            r, n = value(par, x)
            r_out.append(r)
            n_out.append(n)
            continue
        x = {k: v.requires_grad_() for k, v in x.items()}
        p = {k: v.clone().requires_grad_() if k in sums else v for k, v in par.items()}
        r, n = value(p, x)
        total = (r * s["grad_residual"][at].double()).sum()
        if c["pre"]:
            total = total + (n * s["grad_normed"][at].double()).sum()
        for k, g in zip(list(x) + list(sums), torch.autograd.grad(total, list(x.values()) + [p[k] for k in sums])):
            if k in sums:
                sums[k] += g
            else:
                whole[k][at] = g
    if c["op"] == "norm_fwd":
        return torch.cat(r_out), (torch.cat(n_out) if c["pre"] else None)
    return {**whole, **sums}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "scan_step":
        f64 = lambda v: None if v is None else v.double()  # noqa: E731
        a, c = _exact_gate(s, s["z"].double(), f64(s["A_log"]), f64(s["dt_bias"]))
        pool, at = s["pool"].double(), s["slots"].long()
        u = c * s["x"].double()
        if s["input_gate"] is not None:
            u = u * torch.sigmoid(s["input_gate"].double())
        pool[at] = a * pool[at] + u
        return pool[at], pool
    if op == "conv_step":
        pool, at = s["pool"].double(), s["slots"].long()
        rows = torch.cat((pool[at], s["x"].double()[:, None]), 1)
        b = None if s["bias"] is None else s["bias"].double()
        y = torch.cat([_exact_mix(case, rows[n], s["weight"].double(), b) for n in range(case["n"])])
        pool[at] = rows[:, 1:]
        return y, pool
    if op.startswith("scan"):
        return _exact_scan(s)
    return _exact_conv(s) if op.startswith("conv") else _exact_norm(s)
