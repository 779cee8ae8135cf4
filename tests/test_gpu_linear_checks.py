"""GPU tests of the finite checks (kda_set_debug_checks) on decode steps of linear attention: they look at what the
call wrote, and at nothing else."""
import pytest
import torch

from linear_attention_kda_gb300 import kda
from tests import linear_util as LU

pytestmark = pytest.mark.gpu
NUMERIC = 12


@pytest.fixture
def checks():
    torch.cuda.synchronize()
    kda.get_device_error()
    kda.set_debug_checks(kda.CHECK_FINITE)
    yield
    kda.set_debug_checks(0)


def _step(d, pool, idx, out):
    x = LU.to(d, "cuda")
    kda.linear_recurrent_step(x["q"], x["k"], x["v"], x["g"], pool, scale=0.75, state_indices=idx, out=out)
    return kda.get_device_error()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H,dk,dv", [(5, 4, 128, 128), (40, 3, 64, 128), (300, 1, 128, 64)])
def test_padded_batch(checks, dtype, N, H, dk, dv):
    """Unused rows and slots hold NaN; every written row and slot is looked at."""
    d = LU.batch([1] * N, H, dk, dv, dtype, N)
    slots = 2 * N + 1
    idx = torch.randperm(slots, generator=torch.Generator().manual_seed(N))[:N].to(torch.int32)
    used = idx.long().clone()
    idx[1::3] = -1
    used = used[idx >= 0]

    def fresh():
        pool = torch.full((slots, H, dk, dv), float("nan"))
        pool[used] = 0.5
        out = torch.full((N, H, dv), float("nan"), dtype=LU.DT[dtype], device="cuda")
        return pool.cuda(), out

    pool, out = fresh()
    assert _step(d, pool, idx.cuda(), out) == 0
    for n in (0, N - 1 - (idx[N - 1] < 0).item()):
        # (one channel of the state: its row and the output's column of it)
        pool, out = fresh()
        pool[int(idx[n]), H - 1, dk - 1, dv - 1] = float("inf")
        assert _step(d, pool, idx.cuda(), out) == NUMERIC
        # a product too large for the output alone
        big = dict(d, q=d["q"].clone())
        big["q"][n] = 3e38
        pool, out = fresh()
        assert _step(big, pool, idx.cuda(), out) == NUMERIC
        assert torch.isfinite(pool[int(idx[n])]).all()


def test_without_indices_and_with_bad_ones(checks):
    N = 6
    d = LU.batch([1] * N, 2, 64, 64, "f32", 1)
    pool = torch.full((N + 2, 2, 64, 64), 0.25, device="cuda")
    pool[N:] = float("nan")  # behind the call's slots
    out = torch.zeros((N, 2, 64), device="cuda")
    assert _step(d, pool, None, out) == 0
    idx = torch.arange(N, dtype=torch.int32)
    idx[2], idx[4] = 9999, 0  # outside the pool, and the first row's slot: reported, not looked at
    out[[2, 4]] = float("nan")
    pool[[2, 4]] = float("nan")
    assert _step(d, pool, idx.cuda(), out) == 8
