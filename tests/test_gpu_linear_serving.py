"""The linear-attention calls together, as a server and a training step use them: rotary positions, prefill, slots of
a state pool saved, forked and compacted, padded decode batches, the output gate; gradients through rope and prefill."""
import numpy as np
import pytest
import torch

from linear_attention_kda_gb300 import kda
from oracle import linear_ref as R, numpy_ref
from tests import linear_util as LU

pytestmark = pytest.mark.gpu
H, D = 3, 64
FREQS = kda.rope_frequencies(32, 5e4, "yarn", 8.0, original_length=4096)
SCALE = kda.rope_attention_scale(8.0)


def _turn(x, positions, inverse=False):
    """kda.rope's "interleaved" rotation in fp64."""
    x = x.double().clone()
    a = positions.double()[:, None] * FREQS
    c, s = torch.cos(a)[:, None] * SCALE, torch.sin(a)[:, None] * SCALE * (-1 if inverse else 1)
    u, v = x[..., 0:32:2].clone(), x[..., 1:32:2].clone()
    x[..., 0:32:2], x[..., 1:32:2] = u * c - v * s, v * c + u * s
    return x


def _tokens(n, seed):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn((n, H, D), generator=g) for _ in range(3))
    rate = torch.tensor([0.003, 0.05, 0.4])
    return dict(q=q / q.norm(dim=-1, keepdim=True), k=k / k.norm(dim=-1, keepdim=True), v=v,
                g=-rate * torch.nn.functional.softplus(torch.randn((n, H), generator=g)), gate=torch.randn((n, H, D), generator=g))


def _rope(t, positions):
    return kda.rope(t["q"].cuda(), t["k"].cuda(), positions.cuda(), FREQS, layout="interleaved", scale=SCALE)


def _cat(*ts):
    return {n: torch.cat([t[n] for t in ts]) for n in ts[0]}


def _reference(t, first=0):
    """Outputs behind the gate and the final state of one sequence, fp64, from a zero state."""
    pos = torch.arange(first, first + t["q"].shape[0])
    o, S = R.forward(_turn(t["q"], pos).numpy(), _turn(t["k"], pos).numpy(), t["v"].double().numpy(), t["g"].double().numpy(),
                     np.zeros((H, D, D)))
    return numpy_ref.output_gate(o, t["gate"].double().numpy(), np.ones((1, H, D)), 1e-6), S


def _near(got, want, tol=2e-5):
    # fp32 throughout; a chain of rope (6e-7), prefill and steps (their own tests bound each element) and the norm, whose
    # division can raise an element's relative error but not the row's: rows of about 1, errors below 1e-6 each
    err = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
    assert err <= tol, err


def test_serving():
    prompts = [_tokens(201, 1), _tokens(64, 2), _tokens(7, 3)]
    lens = [p["q"].shape[0] for p in prompts]
    cu = torch.tensor([0, 201, 265, 272], dtype=torch.int32).cuda()
    batch = _cat(*prompts)
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
    q, k = _rope(batch, pos)
    o, S = kda.linear_chunk_fwd(q, k, batch["v"].cuda(), batch["g"].cuda(), cu_seqlens=cu, output_final_state=True)
    y = kda.output_gate(o, batch["gate"].cuda(), eps=1e-6)
    torch.cuda.synchronize()
    at = 0
    for p, n in zip(prompts, lens):
        _near(y[at:at + n], _reference(p)[0])
        at += n
    # the prompts' states go into slots 9, 4 and 6 of the pool; prompt 0 is forked into slots 1 and 7, slot 4 is cleared
    idx = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    pool = torch.full((10, H, D, D), float("nan"), device="cuda")
    kda.state_copy(S, idx(0, 1, 2), idx(9, 4, 6), out_pool=pool)
    kda.state_copy(pool, idx(9, 9, -1), idx(1, 7, 4))
    seqs = {9: [prompts[0]], 1: [prompts[0]], 7: [prompts[0]], 6: [prompts[2]]}
    # decode: a padded batch of six rows, four of them in use
    slots = [7, -1, 6, 9, 1, -1]
    for step in range(4):
        new = _tokens(6, 100 + step)
        pos = torch.tensor([sum(t["q"].shape[0] for t in seqs[s]) if s >= 0 else 0 for s in slots], dtype=torch.int32)
        q, k = _rope(new, pos)
        o = kda.linear_recurrent_step(q, k, new["v"].cuda(), new["g"].cuda(), pool, state_indices=idx(*slots))
        y = kda.output_gate(o, new["gate"].cuda(), eps=1e-6)
        torch.cuda.synchronize()
        for row, s in enumerate(slots):
            if s >= 0:
                seqs[s].append({n: t[row:row + 1] for n, t in new.items()})
                _near(y[row:row + 1], _reference(_cat(*seqs[s]))[0][-1:])
        if step == 1:  # compaction: slots 9, 7 and 6 move down into holes, one of them onto a slot that has just moved
            kda.state_copy(pool, idx(6, 9, 7), idx(0, 6, 2))
            seqs = {0: seqs[6], 6: seqs[9], 2: seqs[7], 1: seqs[1]}
            slots = [2, -1, 0, 6, 1, -1]
    # one more prompt for two of the sequences, entering from their slots and going back there
    more = [_tokens(130, 7), _tokens(33, 8)]
    batch, n0 = _cat(*more), [sum(t["q"].shape[0] for t in seqs[s]) for s in (2, 0)]
    pos = torch.cat([torch.arange(a, a + t["q"].shape[0]) for a, t in zip(n0, more)]).to(torch.int32)
    entering = torch.empty((2, H, D, D), device="cuda")
    kda.state_copy(pool, idx(2, 0), idx(0, 1), out_pool=entering)
    q, k = _rope(batch, pos)
    o, S = kda.linear_chunk_fwd(q, k, batch["v"].cuda(), batch["g"].cuda(), cu_seqlens=idx(0, 130, 163), initial_state=entering,
                                final_state=entering)
    kda.state_copy(entering, idx(0, 1), idx(2, 0), out_pool=pool)
    y = kda.output_gate(o, batch["gate"].cuda(), eps=1e-6)
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0
    for (a, b), s, t in zip(((0, 130), (130, 163)), (2, 0), more):
        want, state = _reference(_cat(*seqs[s], t))
        _near(y[a:b], want[-(b - a):])
        _near(pool[s], state)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_step(dtype):
    """Gradients of sum(prefill(rope(q), rope(k), v, g) * w) against autograd of the formulas in fp64."""
    t, lens = _tokens(200, 5), [137, 63]
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
    w = torch.randn((200, H, D), generator=torch.Generator().manual_seed(6)).to(LU.DT[dtype])
    x = {n: t[n].to(LU.DT[dtype]) if n != "g" else t[n] for n in ("q", "k", "v", "g")}
    cu = torch.tensor([0, 137, 200], dtype=torch.int32).cuda()
    q, k = kda.rope(x["q"].cuda(), x["k"].cuda(), pos.cuda(), FREQS, layout="interleaved", scale=SCALE)
    r = kda.linear_chunk_bwd(q, k, x["v"].cuda(), x["g"].cuda(), w.cuda(), cu_seqlens=cu, state_grad=False)
    dq, dk = kda.rope(r["q"], r["k"], pos.cuda(), FREQS, layout="interleaved", scale=SCALE, inverse=True)
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0
    leaf = {n: v.double().requires_grad_() for n, v in x.items()}
    a = pos.double()[:, None] * FREQS
    c, s = (torch.cos(a) * SCALE)[:, None], (torch.sin(a) * SCALE)[:, None]

    def turn(y):
        u, v = y[..., 0:32:2], y[..., 1:32:2]
        return torch.cat((torch.stack((u * c - v * s, v * c + u * s), -1).flatten(-2), y[..., 32:]), -1)

    qr, kr, loss = turn(leaf["q"]), turn(leaf["k"]), 0.0
    for b, n in ((0, 137), (137, 63)):
        G = leaf["g"][b:b + n].cumsum(0)
        D_ = torch.exp((G[:, None] - G[None]).masked_fill(~torch.ones((n, n), dtype=torch.bool).tril()[..., None], -np.inf))
        A = torch.einsum("rhd,thd->rth", qr[b:b + n], kr[b:b + n]) * D_
        loss = loss + (torch.einsum("rth,thd->rhd", A, leaf["v"][b:b + n]) * w[b:b + n].double()).sum()
    loss.backward()
    # Relative 2-norms.  fp32: the calls' own elementwise bounds are a few 1e-5 of an element's terms at the very worst.
    # bf16: q and k rounded behind rope, A or dA and the results, rope's result: five roundings of 2^-8 at most each.
    # g's gradient is made from the rounded q and k: two of them, in sums whose terms partly cancel (counted as four).
    for name, got in (("q", dq), ("k", dk), ("v", r["v"]), ("g", r["g"])):
        want = leaf[name].grad.numpy()
        err = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
        assert err <= (5e-5 if dtype == "f32" else (5 if name != "g" else 8) * 2.0 ** -8), (name, err)
