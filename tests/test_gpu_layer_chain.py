"""The calls around a recurrence together, as a recurrent layer uses them: the norm in front, the short convolution, the
gated recurrence and the norm behind with its gate and scale into the residual stream; prefill, padded decode steps from
pools, and a training step's gradients through all of them; and the convolution with its norm in front of KDA itself."""
import numpy as np
import pytest
import torch

from linear_attention_kda_gb300 import kda
from oracle import c_ref, layer_ref as R
from tests import layer_util as U

pytestmark = pytest.mark.gpu
D = 96


def _params(seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(pre=1 + 0.2 * rn(D), post=1 + 0.2 * rn(D), scale=0.3 + 0.5 * torch.rand((D,), generator=g), w=rn(D, 4) / 2, b=0.2 * rn(D),
                A=torch.linspace(np.log(2e-3), np.log(0.5), D), dt=0.5 * rn(D))


def _tokens(n, seed):
    g = torch.Generator().manual_seed(seed)
    return dict(zip(("r", "z", "i", "gate"), (torch.randn((n, D), generator=g) for _ in range(4))))


def _cat(*ts):
    return {k: torch.cat([t[k] for t in ts]) for k in ts[0]}


def _layer(p, t, cu=None, conv=None, state=None, keep=None):
    """One layer on packed tokens; (what the next block reads, the residual stream, what a gradient needs)."""
    _, n = kda.block_norm_fwd(None, t["r"], pre_weight=p["pre"])
    c, _ = kda.short_conv_fwd(n, p["w"], p["b"], cu_seqlens=cu, initial_state=conv, final_state=conv)
    h, _ = kda.scan_fwd(c, t["z"], t["i"], A_log=p["A"], dt_bias=p["dt"], input_scale="norm", cu_seqlens=cu, initial_state=state, final_state=state,
                        checkpoints=keep)
    r, y = kda.block_norm_fwd(h, t["r"], t["gate"], post_weight=p["post"], pre_weight=p["pre"], scale=p["scale"])
    return y, r, (n, c, h)


def _reference(p, t):
    """The layer on one sequence from empty states, fp64: (y, r', history, state)."""
    q = {k: v.double().numpy() for k, v in p.items()}
    x = {k: v.double().numpy() for k, v in t.items()}
    _, n = R.block_norm(None, x["r"], None, 1.0, None, q["pre"])
    c, hist = R.conv(n, np.zeros((3, D)), q["w"], q["b"])
    h, _, S = R.scan(c, x["z"], x["i"], q["A"], q["dt"], np.zeros(D), input_scale="norm")
    r, y = R.block_norm(h, x["r"], x["gate"], q["scale"], q["post"], q["pre"])
    return y, r, hist, S


def _near(got, want, tol=1e-5):
    # fp32 throughout: each call's own tests bound its elements by a few hundred u = 6e-8 of their terms at the very worst, the
    # typical error of a row's norm through the four of them is below 1e-6
    got = got.double().cpu().numpy()
    err = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-30)
    assert err <= tol, err


def test_serving():
    p = _params(1)
    q = U.to(p)
    prompts = [_tokens(201, 1), _tokens(2, 2), _tokens(70, 3)]
    batch = U.to(_cat(*prompts))
    conv, state = torch.zeros((3, 3, D), device="cuda"), torch.zeros((3, D), device="cuda")
    y, r, _ = _layer(q, batch, U.cu([201, 2, 70]).cuda(), conv, state)
    torch.cuda.synchronize()
    at = 0
    for n, t in enumerate(prompts):
        m, want = t["r"].shape[0], _reference(p, t)
        for got, ref in ((y[at:at + m], want[0]), (r[at:at + m], want[1]), (conv[n], want[2]), (state[n], want[3])):
            _near(got, ref)
        at += m
    # slots 5, 1 and 3 of the pools; the first prompt is forked into slot 0
    idx = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    pools = [torch.full((7, 3, D), float("nan"), device="cuda"), torch.full((7, D), float("nan"), device="cuda")]
    for a, b in zip((conv, state), pools):
        kda.state_copy(a, idx(0, 1, 2), idx(5, 1, 3), out_pool=b)
        kda.state_copy(b, idx(5), idx(0))
    slots = [3, -1, 0, 5, 1, -1]
    seqs = {5: [prompts[0]], 0: [prompts[0]], 1: [prompts[1]], 3: [prompts[2]]}
    for step in range(4):
        new = _tokens(6, 50 + step)
        x = U.to(new)
        _, n = kda.block_norm_fwd(None, x["r"], pre_weight=q["pre"])
        c = kda.short_conv_step(n, q["w"], q["b"], pools[0], state_indices=idx(*slots))
        h = kda.scan_step(c, x["z"], x["i"], pools[1], A_log=q["A"], dt_bias=q["dt"], input_scale="norm", state_indices=idx(*slots))
        r, y = kda.block_norm_fwd(h, x["r"], x["gate"], post_weight=q["post"], pre_weight=q["pre"], scale=q["scale"])
        torch.cuda.synchronize()
        for row, s in enumerate(slots):
            if s >= 0:
                seqs[s].append({k: v[row:row + 1] for k, v in new.items()})
                want = _reference(p, _cat(*seqs[s]))
                for got, ref in ((y[row], want[0][-1]), (r[row], want[1][-1]), (pools[0][s], want[2]), (pools[1][s], want[3])):
                    _near(got, ref)
    assert kda.get_device_error() == 0


def _torch_layer(p, t, lens):
    rms = lambda v: v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    out, at = [], 0
    for m in lens:
        x = {k: v[at:at + m] for k, v in t.items()}
        n = torch.cat((torch.zeros((3, D), dtype=torch.float64), p["pre"] * rms(x["r"])))
        c = torch.nn.functional.silu(p["b"] + sum(p["w"][:, j] * n[j:j + m] for j in range(4)))
        g = -torch.exp(p["A"]) * torch.nn.functional.softplus(x["z"] + p["dt"], threshold=1e9)
        u, a = torch.sqrt(-torch.expm1(2 * g)) * torch.sigmoid(x["i"]) * c, torch.exp(g)
        h, hs = torch.zeros(D, dtype=torch.float64), []
        for k in range(m):
            h = a[k] * h + u[k]
            hs.append(h)
        r = x["r"] + p["scale"] * torch.sigmoid(x["gate"]) * p["post"] * rms(torch.stack(hs))
        out.append(torch.cat((r, p["pre"] * rms(r)), -1))
        at += m
    return torch.cat(out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_step(dtype):
    """Gradients of sum(r' w1 + y w2) with regard to every input and parameter, against autograd in fp64."""
    p, lens = _params(2), [130, 3, 67]
    t = {k: v.to(U.DT[dtype]) for k, v in _tokens(200, 4).items()}
    g = torch.Generator().manual_seed(9)
    w1, w2 = (torch.randn((200, D), generator=g).to(U.DT[dtype]) for _ in range(2))
    q, x, cu = U.to(p), U.to(t), U.cu(lens).cuda()
    keep = kda.scan_checkpoints(200, 3, D)
    _, _, (n, c, h) = _layer(q, x, cu, keep=keep)
    how = dict(post_weight=q["post"], pre_weight=q["pre"], scale=q["scale"])
    b1 = kda.block_norm_bwd(h, x["r"], x["gate"], w1.cuda(), w2.cuda(), **how)
    b2 = kda.scan_bwd(c, x["z"], x["i"], b1["y"], keep, A_log=q["A"], dt_bias=q["dt"], input_scale="norm", cu_seqlens=cu, state_grad=False)
    b3 = kda.short_conv_bwd(n, q["w"], q["b"], b2["x"], cu_seqlens=cu, state_grad=False)
    b4 = kda.block_norm_bwd(None, x["r"], None, b1["residual"], b3["x"], pre_weight=q["pre"])
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0
    got = dict(r=b4["residual"], z=b2["z"], i=b2["input_gate"], gate=b1["gate"], pre=b1["pre_weight"] + b4["pre_weight"], post=b1["post_weight"],
               scale=b1["scale"], w=b3["weight"], b=b3["bias"], A=b2["A_log"], dt=b2["dt_bias"])
    leaf = {k: v.double().requires_grad_() for k, v in {**p, **t}.items()}
    (_torch_layer({k: leaf[k] for k in p}, {k: leaf[k] for k in t}, lens) * torch.cat((w1, w2), -1).double()).sum().backward()
    # Relative 2-norms.  fp32: as _near, through eight calls.  bf16: up to eight roundings of 2^-9 on the way to a gradient (n, c, h
    # forwards, their gradients backwards and the result), errors of mixed sign; parameters' sums cancel to a fraction (counted twice).
    for k, v in got.items():
        want = leaf[k].grad.numpy()
        err = np.linalg.norm(v.double().cpu().numpy() - want) / np.linalg.norm(want)
        assert err <= (2e-5 if dtype == "f32" else (8 if k in t else 16) * 2.0 ** -9), (k, err)


def test_convolution_in_front_of_kda():
    """Eq. 2 without projections: q and k through the convolution, SiLU and the heads' L2 norm, v without the norm, then the
    prefill and its output between two blocks, against the oracles."""
    T, H, d = 130, 2, 64
    g = torch.Generator().manual_seed(5)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    fused, w = rn(T, 3 * H * d), rn(3, H * d, 4) / 2
    z, beta = rn(T, H, d), torch.sigmoid(rn(T, H))
    qkv = []
    x = fused.cuda()
    for j in range(3):
        y, _ = kda.short_conv_fwd(x[:, j * H * d:(j + 1) * H * d], w[j].cuda(), norm_dim=d if j < 2 else 0)
        qkv.append(y.view(T, H, d))
    o, _ = kda.chunk_fwd(*qkv[:2], qkv[2], z.cuda(), beta.cuda())
    r0, gate = rn(T, H * d), rn(T, H * d)
    r, n = kda.block_norm_fwd(o.view(T, H * d), r0.cuda(), gate.cuda())
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0
    ref = []
    for j in range(3):
        y, _ = R.conv(fused[:, j * H * d:(j + 1) * H * d].double().numpy(), np.zeros((3, H * d)), w[j].double().numpy(), 0.0,
                      norm=d if j < 2 else 0)
        ref.append(torch.from_numpy(y).view(T, H, d))
    res, _ = c_ref.forward(*ref[:2], ref[2], z.double(), beta.double(), torch.zeros((H, d)), torch.zeros(H), torch.tensor([0, T]), S0=None,
                           g_min=-5.0, scale=1.0)
    want = np.stack([res[(0, h)][0] for h in range(H)], 1).reshape(T, H * d)
    a, b = R.block_norm(want, r0.double().numpy(), gate.double().numpy(), 1.0, np.ones(H * d), np.ones(H * d))
    _near(o.view(T, H * d), want, 1e-4)  # (the prefill's own tolerance)
    _near(r, a, 1e-4)
    _near(n, b, 1e-4)
