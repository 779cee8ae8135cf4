"""GPU tests of what the linear-attention calls hold in their states: sums over many tokens."""
import pytest
import torch

from linear_attention_kda_gb300 import kda

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
