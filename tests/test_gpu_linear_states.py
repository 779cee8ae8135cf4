"""GPU tests of what the linear-attention calls hold in their states: sums over many tokens, and what an erasing decay
leaves of values that are no numbers."""
import numpy as np
import pytest
import torch

from linear_attention_kda_gb300 import kda
from tests import linear_util as LU

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,T,dk,dv", [(77, 16384, 64, 64), (77, 8192, 128, 128), (5, 40000, 64, 128)])
def test_bf16_state_of_many_tokens_has_no_drift(H, T, dk, dv):
    """Positive terms without decay: whatever a sum loses at every step in one direction shows in the mean of the error.

    A chunk's 128 terms are exact products, summed in 8 steps of 16 that may each cut below the last bit of an fp32
    (2^-23 of the sum); chunks are added with rounding to nearest, which has no direction.  8 * 2^-23 bounds the drift
    at any length; an accumulator that ran through all T / 16 steps, half full on average, would lose about
    T / 16 / 2 * 2^-24, 1.5e-5 at 8192 tokens."""
    gen = torch.Generator(device="cuda").manual_seed(T + dk)
    k, v = (torch.rand((T, H, d), generator=gen, device="cuda").add_(0.25).bfloat16() for d in (dk, dv))
    q = torch.zeros_like(k)
    _, S = kda.linear_chunk_fwd(q, k, v, None, output_final_state=True)
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0
    want = torch.stack([k[:, h].double().T @ v[:, h].double() for h in range(H)])
    drift = float(((S[0].double() - want) / want).mean())
    assert abs(drift) <= 8 * 2.0 ** -23, drift


LENS = {"short": [1, 0, 5, 40], "ragged": [300, 130, 0, 128, 1], "few_long": [3000, 700]}


def _erasing(lens, H, dk, dv, dtype, seed, at):
    """A batch whose decay erases the state at token `at` of every sequence (-1: the last one) that has it."""
    d = LU.batch(lens, H, dk, dv, dtype, seed)
    cu = d["cu_seqlens"].tolist()
    rows = [a + (at if at >= 0 else b - a + at) for a, b in zip(cu, cu[1:]) if b - a > (at if at >= 0 else 0)]
    d["g"][rows[::2]] = -np.inf
    d["g"][rows[1::2]] = -104.0
    return d, cu


def _tokens_from(cu, at):
    keep = torch.zeros(cu[-1], dtype=torch.bool, device="cuda")
    for a, b in zip(cu, cu[1:]):
        keep[min(a + at, b):b] = True
    return keep


def _fwd(d, state):
    x = LU.to(d, "cuda")
    r = kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], scale=d["scale"], cu_seqlens=x["cu_seqlens"], initial_state=state.cuda(),
                             output_final_state=True)
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0
    return r


def _bwd(d, state, grad_state):
    x = LU.to(d, "cuda")
    r = kda.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["grad_o"], scale=d["scale"], cu_seqlens=x["cu_seqlens"],
                             initial_state=state.cuda(), grad_final_state=grad_state.cuda())
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0
    return r


def _no_numbers(like):
    x = torch.full_like(like, float("nan"))
    x.view(-1)[::3] = float("inf")
    x.view(-1)[1::5] = -float("inf")
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("at,dk,dv", [(0, 128, 128), (0, 64, 128), (70, 128, 64), (200, 128, 128), (1000, 64, 64)])
def test_prefill_from_a_state_that_is_erased(dtype, lens, at, dk, dv):
    """Tokens from the erasing one on, and the final states, are those of a call that began from zeros."""
    d, cu = _erasing(LENS[lens], 2, dk, dv, dtype, 60 + at, at)
    o, S = _fwd(d, _no_numbers(d["initial_state"]))
    zo, zS = _fwd(d, torch.zeros_like(d["initial_state"]))
    keep = _tokens_from(cu, at)
    assert torch.equal(o[keep], zo[keep]) and torch.isfinite(o[keep]).all()
    erased = torch.tensor([b - a > at for a, b in zip(cu, cu[1:])], device="cuda")
    assert torch.equal(S[erased], zS[erased]) and torch.isfinite(S[erased]).all()
    # (the second head's decays of 700 tokens, 0.7 * 0.8 each on average, come to e^-390, which is 0 as well)
    assert not torch.isfinite(S[~erased, 0]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_token_prefill_and_step_erase_alike(dtype):
    d = LU.batch([1] * 7, 2, 64, 128, dtype, 70)
    d["g"][:] = -np.inf
    x, bad = LU.to(d, "cuda"), _no_numbers(d["initial_state"]).cuda()
    o, S = kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], scale=0.75, cu_seqlens=x["cu_seqlens"], initial_state=bad,
                                output_final_state=True)
    so = kda.linear_recurrent_step(x["q"], x["k"], x["v"], x["g"], bad, scale=0.75)
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0
    d["initial_state"] = torch.zeros_like(d["initial_state"])
    (ro, rS), (ao, aS) = LU.forward_ref(d), LU.forward_ref(d, True)
    # one product for a state's element (bf16 operands: an exact one), 64 of them and a rounding or two for an output's
    step = LU.U32 if dtype == "f32" else LU.EPS_BF16
    for got_o, got_S in ((o, S), (so, bad)):
        LU.close("o", got_o, ro, ao, 104 * LU.U32 + (0 if dtype == "f32" else LU.EPS_BF16), step)
        LU.close("state", got_S, rS, aS, 8 * LU.U32, LU.U32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", sorted(LENS) + ["one_long"])
@pytest.mark.parametrize("dk,dv,heads", [(128, 128, {}), (64, 128, dict(Hq=1, Hk=1)), (128, 64, dict(Hk=1, Hv=1))])
def test_gradients_from_a_state_that_is_erased(dtype, lens, dk, dv, heads):
    """The first token erases the state that a sequence begins with: all gradients are those of zeros."""
    n = LENS.get(lens, [9000])
    d = LU.batch(n, 2, dk, dv, dtype, 80, **heads)
    cu = d["cu_seqlens"].tolist()
    d["g"][[a for a, b in zip(cu, cu[1:]) if b > a]] = -np.inf
    zero = torch.zeros_like(d["initial_state"])
    r, z = _bwd(d, _no_numbers(d["initial_state"]), d["grad_final_state"]), _bwd(d, zero, d["grad_final_state"])
    for x in r:
        assert torch.isfinite(r[x]).all() and torch.equal(r[x], z[x]), x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", sorted(LENS) + ["one_long"])
@pytest.mark.parametrize("dk,dv,heads", [(128, 128, {}), (64, 128, dict(Hq=1, Hk=1)), (128, 64, dict(Hk=1, Hv=1))])
def test_gradients_of_a_final_state_that_was_erased(dtype, lens, dk, dv, heads):
    """The last token erases what came before: only its own k and v meet the final state's gradient."""
    d, cu = _erasing(LENS.get(lens, [9000]), 2, dk, dv, dtype, 90, -1)
    for n, h in heads.items():
        x = n[1].lower()
        d[x] = d[x][:, :h].contiguous()
    zero = torch.zeros_like(d["grad_final_state"])
    r, z = _bwd(d, d["initial_state"], _no_numbers(zero)), _bwd(d, d["initial_state"], zero)
    keep = torch.ones(cu[-1], dtype=torch.bool, device="cuda")
    keep[[b - 1 for a, b in zip(cu, cu[1:]) if b > a]] = False
    assert torch.equal(r["q"], z["q"])
    for x in ("k", "v"):
        assert torch.isfinite(r[x][keep]).all() and torch.equal(r[x][keep], z[x][keep]), x
    some = torch.tensor([b > a for a, b in zip(cu, cu[1:])], device="cuda")
    assert torch.equal(r["initial_state"][some], z["initial_state"][some]) and torch.isfinite(r["initial_state"][some]).all()
