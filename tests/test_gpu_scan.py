"""GPU tests of the gated recurrence over channels (sequences, gradients, single tokens) against the fp64 oracle."""
import numpy as np
import pytest
import torch

from linear_attention_kda_gb300 import kda
from oracle import layer_ref as R
from tests import layer_util as U

pytestmark = pytest.mark.gpu
DTYPES = ("f32", "bf16")


def _no_error():
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0


def _how(x):
    return dict(A_log=x["A_log"], dt_bias=x["dt_bias"], gate=x["gate"], input_scale=x["input_scale"], cu_seqlens=x["cu_seqlens"])


def _fwd(d, **kw):
    x = U.to(d)
    keep = torch.full((d["x"].shape[0] // 64 + len(d["lens"]), d["D"]), float("nan"), device="cuda")
    h, last = kda.scan_fwd(x["x"], x["z"], x["input_gate"], initial_state=x["initial_state"], output_final_state=True, checkpoints=keep, **_how(x), **kw)
    return h, last, keep


def _bwd(d, keep, **kw):
    x = U.to(d)
    return kda.scan_bwd(x["x"], x["z"], x["input_gate"], x["grad_h"], keep, grad_final_state=x["grad_final_state"], **_how(x), **kw)


def _check_fwd(d, got):
    _no_error()
    want, size, n = U.scan_ref(d), U.scan_ref(d, True), U.scan_roundings(d)
    U.close("h", got[0], want[0], size[0], n, U.HALF[d["dtype"]])
    U.close("final_state", got[1], want[1], size[1], n, U.U32)
    held = ~np.isnan(want[2])
    assert (np.isnan(U.f64(got[2])) == ~held).all()  # rows without a checkpoint are left as they were
    U.close("checkpoints", got[2].cpu()[torch.from_numpy(held)], want[2][held], size[2][held], n, U.U32)


def _check_bwd(d, got):
    _no_error()
    # states and adjoints both carry a scan's roundings, parameters' gradients those of a sum over all tokens as well
    want, size, n = U.scan_grads_ref(d), U.scan_grads_ref(d, True), 2 * U.scan_roundings(d)
    assert set(got) == {"x", "z", "initial_state"} | ({"input_gate"} if d["input_gate"] is not None else set()) | (
        set() if d["gate"] == "log" else {"A_log", "dt_bias"})
    for k in got:
        par = k in ("A_log", "dt_bias")
        U.close(k, got[k], want[k], size[k], n + (d["x"].shape[0] if par else 0), U.U32 if par or k == "initial_state" else U.HALF[d["dtype"]])


CASES = [(t, g, i, {}) for t in DTYPES for g in U.GATES for i in U.INPUTS] + \
        [(t, "softplus", "norm", kw) for t in DTYPES for kw in (dict(gated=False), dict(params=False), dict(state=False))]


@pytest.mark.parametrize("dtype,gate,input_scale,kw", CASES)
def test_varlen(dtype, gate, input_scale, kw):
    d = U.scan_batch(U.LENS, 136, dtype, 1, gate=gate, input_scale=input_scale, **kw)
    r = _fwd(d)
    _check_fwd(d, r)
    _check_bwd(d, _bwd(d, r[2]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [1, 2, 3, 7, 8, 31, 33, 64, 100, 127, 130, 260, 1032])
def test_widths(dtype, D):
    d = U.scan_batch([70, 5, 129], D, dtype, D, gate="sigmoid", input_scale="norm")
    r = _fwd(d)
    _check_fwd(d, r)
    _check_bwd(d, _bwd(d, r[2]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[1], [20000], [1023, 1025], [1, 4097, 1024], [2] * 300, [64] * 40])
def test_lengths(dtype, lens):
    d = U.scan_batch(lens, 8, dtype, len(lens), gate="lower_bound", input_scale="complement")
    r = _fwd(d)
    _check_fwd(d, r)
    _check_bwd(d, _bwd(d, r[2]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("long", (0, 3000))
@pytest.mark.parametrize("N", (350, 700))
def test_many_sequences(dtype, N, long):
    """Tiles of 32 and of 64 channels, whole chains and (beside one long sequence) tiles that join others; the same bits from
    rows at odd elements."""
    lens = np.random.default_rng(N + long).integers(0, 520 if not long else 8, N).tolist()
    lens[N // 3] = long or lens[N // 3]
    d = U.scan_batch(lens, 36, dtype, N, gate="softplus" if long else "sigmoid", input_scale="norm")
    r = _fwd(d)
    g = _bwd(d, r[2])
    _check_fwd(d, r)
    _check_bwd(d, g)
    x = U.to(d)
    wide = torch.zeros((sum(lens), 3 * 36 + 1), dtype=U.DT[dtype], device="cuda")
    v = [wide[:, 1 + 36 * k:37 + 36 * k] for k in range(3)]
    for a, b in zip(v, ("x", "z", "input_gate")):
        a.copy_(x[b])
    keep = torch.full_like(r[2], float("nan"))
    h, last = kda.scan_fwd(*v, initial_state=x["initial_state"], output_final_state=True, checkpoints=keep, **_how(x))
    g2 = kda.scan_bwd(*v, x["grad_h"], keep, grad_final_state=x["grad_final_state"], **_how(x))
    _no_error()
    assert torch.equal(h, r[0]) and torch.equal(last, r[1]) and all(torch.equal(g2[k], g[k]) for k in g)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("long", (0, 3000))
@pytest.mark.parametrize("N", (350, 700))
def test_many_sequences_by_copies(dtype, N, long):
    """As above with rows of a multiple of 16 bytes, so that tiles of 32 and of 64 channels come by copies ahead of their use; infinite states too."""
    lens = np.random.default_rng(N + long).integers(0, 520 if not long else 8, N).tolist()
    lens[N // 3] = long or lens[N // 3]
    d = U.scan_batch(lens, 40, dtype, N, gate="softplus" if long else "sigmoid", input_scale="norm")
    r = _fwd(d)
    _check_fwd(d, r)
    _check_bwd(d, _bwd(d, r[2]))
    size, n = U.scan_ref(d, True), U.scan_roundings(d)
    for c, k in enumerate((5, N // 3, N - 1)):  # channels of slow decay, which never erases
        d["initial_state"][k, c] = float("inf")
    r, want = _fwd(d), U.scan_ref(d)
    _no_error()
    assert np.isinf(want[0]).sum() == sum(lens[k] for k in (5, N // 3, N - 1))
    _same("h", r[0], want[0], size[0], n, U.HALF[dtype])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[9000, 30, 500, 0, 77], [700, 0, 1500, 2000, 64, 1, 900, 1200, 333, 1800], [5, 3000]])
def test_few_sequences_of_many_channels(dtype, lens):
    """Large enough a call for its sequences to be taken in order of length: whole chains, and tiles that join others."""
    d = U.scan_batch(lens, 1040, dtype, 23, input_scale="complement")
    r = _fwd(d)
    _check_fwd(d, r)
    _check_bwd(d, _bwd(d, r[2]))


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_long_sequence(dtype):
    """More tiles than share the first two levels of what joins them."""
    d = U.scan_batch([140000, 5], 6, dtype, 18, gate="sigmoid")
    r = _fwd(d)
    _check_fwd(d, r)
    _check_bwd(d, _bwd(d, r[2]))


def test_tokens_behind_32_bits():
    """More than 2^31 elements: the last sequences against the oracle, the gradients of theirs too."""
    D, T = 8192, 264000
    d = U.scan_batch([130, 3, 70], D, "bf16", 17, gate="sigmoid", input_scale="norm")
    x, m = U.to(d), sum(d["lens"])
    big = {k: torch.zeros((T, D), dtype=torch.bfloat16, device="cuda") for k in ("x", "z", "input_gate", "grad_h")}
    for k in big:
        big[k][-m:] = x[k]
    lens = [T - m] + d["lens"]
    how = {**_how(x), "cu_seqlens": U.cu(lens).cuda()}
    state, tail = (torch.cat((torch.zeros((1, D), device="cuda"), x[k])) for k in ("initial_state", "grad_final_state"))
    keep = torch.empty((T // 64 + 4, D), device="cuda")
    h, last = kda.scan_fwd(big["x"], big["z"], big["input_gate"], initial_state=state, output_final_state=True, checkpoints=keep, **how)
    g = kda.scan_bwd(big["x"], big["z"], big["input_gate"], big["grad_h"], keep, grad_final_state=tail, **how)
    _no_error()
    want, size, n = U.scan_ref(d), U.scan_ref(d, True), U.scan_roundings(d)
    U.close("h", h[-m:], want[0], size[0], n, U.HALF["bf16"])
    U.close("final_state", last[1:], want[1], size[1], n, U.U32)
    assert (h[:-m:1000] == 0).all() and (g["x"][:-m:1000] == 0).all()
    _check_bwd(d, {k: v[-m:] if k in ("x", "z", "input_gate") else v[1:] if k == "initial_state" else v for k, v in g.items()})


def test_equal_lengths_without_cu_seqlens():
    d = U.scan_batch([50] * 6, 24, "f32", 2)
    r = _fwd(d)
    x = U.to(d)
    how = {**_how(x), "cu_seqlens": None, "n_seq": 6}
    h, last = kda.scan_fwd(x["x"], x["z"], x["input_gate"], initial_state=x["initial_state"], output_final_state=True, **how)
    _no_error()
    assert torch.equal(h, r[0]) and torch.equal(last, r[1])


@pytest.mark.parametrize("dtype", DTYPES)
def test_empty_batch(dtype):
    d = U.scan_batch([0, 0, 0], 40, dtype, 3)
    h, last, keep = _fwd(d)
    g = _bwd(d, keep)
    _no_error()
    assert h.shape == (0, 40) and torch.equal(last.cpu(), d["initial_state"]) and torch.equal(g["initial_state"].cpu(), d["grad_final_state"])
    assert (g["A_log"] == 0).all() and (g["dt_bias"] == 0).all()


def test_slow_decays_do_not_drift():
    """A state that remembers 10,000 tokens, fed a constant: 1 / (1 - a) in the end.  Every 8 tokens or more share one
    decay of the state before them, so it goes through 2 * 60000 / 8 roundings with weights that sum to 2 * 10000 / 8."""
    T, g = 60000, -1e-4
    z = torch.full((T, 16), g, device="cuda")
    _, last = kda.scan_fwd(torch.ones_like(z), z, gate="log", output_final_state=True)
    _no_error()
    a = np.exp(np.float64(np.float32(g)))
    want = (1 - a ** T) / (1 - a)
    assert abs(float(last[0, 0]) / want - 1) <= 2 * 10000 / 8 * U.U32, float(last[0, 0]) / want - 1
    assert (last == last[0, 0]).all()


def test_joined_tiles_keep_slow_decays():
    """A state with nothing entering, over 4096 tiles of 256 tokens that join others, forwards and backwards: exp(T g) of it.  Behind every 256
    tiles it goes through at most 16 groups', 15 tiles' and 8 warps' decays, a rounding each, and a decay's logarithm is a sum of roundings relative to
    itself.  (Decays joined as 1 + d lose up to 1e-4 of the state here.)"""
    T, rates = 1 << 20, [1e-10, 3e-10, 1e-9, 3e-9, 1e-8, 3e-8, 1e-7, 1e-6]
    z = -torch.tensor(rates, device="cuda").expand(T, len(rates)).contiguous()
    x, one, keep = torch.zeros_like(z), torch.ones((1, len(rates)), device="cuda"), kda.scan_checkpoints(T, 1, len(rates))
    _, last = kda.scan_fwd(x, z, gate="log", initial_state=one, output_final_state=True, checkpoints=keep)
    g = kda.scan_bwd(x, z, None, x, keep, gate="log", grad_final_state=one)
    _no_error()
    log = T * U.f64(z[0])
    for got in (last[0], g["initial_state"][0]):
        assert (abs(U.f64(got) / np.exp(log) - 1) <= (16 * 39 + 64 * abs(log)) * U.U32).all(), U.f64(got) / np.exp(log) - 1


@pytest.mark.parametrize("dtype", DTYPES)
def test_erasing_decays(dtype):
    """exp(g) = 0 leaves nothing of the state, infinities and NaN included; -inf and -200 are such decays."""
    d = U.scan_batch([100, 80], 24, dtype, 4, gate="log")
    d["z"][0, :] = -float("inf")
    d["z"][100, :] = -200.0
    d["z"][57, ::2] = -float("inf")
    clean = {**d, "initial_state": d["initial_state"].clone()}
    d["initial_state"][0, :8], d["initial_state"][1, 8:16] = float("nan"), float("inf")
    r = _fwd(d)
    _no_error()
    want, size, n = U.scan_ref(clean), U.scan_ref(clean, True), U.scan_roundings(d)
    U.close("h", r[0], want[0], size[0], n, U.HALF[dtype])
    U.close("final_state", r[1], want[1], size[1], n, U.U32)
    g = _bwd(clean, _fwd(clean)[2])
    _check_bwd(clean, g)
    assert (g["initial_state"] == 0).all()


def _same(name, got, want, size, n, half):
    """Infinities and NaN where the definition has them, the rest within its bound."""
    got, bad = U.f64(got), ~np.isfinite(want)
    assert np.array_equal(np.where(bad, got, 0), np.where(bad, want, 0), equal_nan=True), (name, np.argwhere(~((got == want) | np.isfinite(want) | np.isnan(got) & np.isnan(want)))[:9])
    U.close(name, torch.from_numpy(np.where(bad, 0, got)), np.where(bad, 0, want), np.where(bad, 0, size), n, half)


@pytest.mark.filterwarnings("ignore:invalid value")  # (the oracle's infinities times 0)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("input_scale", U.INPUTS)
@pytest.mark.parametrize("lens", [[150, 90], [60, 3000], [5000, 0, 17]])
def test_infinities_stay_infinities(dtype, input_scale, lens):
    """A state, an input or an adjoint of infinity is one from there on under decays above 0, and erased by one of 0."""
    inf, last, T = float("inf"), len(lens) - 1, sum(lens)
    d = U.scan_batch(lens, 40, dtype, 22, gate="log", input_scale=input_scale)
    d["z"] = (d["z"].float() * 0.02).to(U.DT[dtype])  # (whose sum over a sequence is nowhere below -80)
    d["z"][0, 5], d["z"][35, 14], d["z"][T - 1, 6] = -inf, -inf, -inf
    clean = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    n, size = U.scan_roundings(d), U.scan_ref(clean, True)
    d["initial_state"][0, :8], d["initial_state"][last, 4:9] = inf, -inf
    d["x"][40, 10], d["x"][lens[0] - 1, 11], d["x"][T - 9, 12], d["x"][20, 14] = inf, -inf, inf, inf
    r, want = _fwd(d), U.scan_ref(d)
    _no_error()
    _same("h", r[0], want[0], size[0], n, U.HALF[dtype])
    _same("final_state", r[1], want[1], size[1], n, U.U32)
    held = ~np.isnan(size[2][:, 0])
    _same("checkpoints", r[2].cpu()[torch.from_numpy(held)], want[2][held], size[2][held], n, U.U32)
    assert np.isinf(want[0]).sum() > 100
    # gradients: of infinite ones of the final state and of a token, and beside an infinite state
    for k in ("grads", "state"):
        e = {**clean, **{j: clean[j].clone() for j in ("grad_final_state", "grad_h", "initial_state")}}
        if k == "grads":
            e["grad_final_state"][last, :8], e["grad_h"][T - 9, 20] = inf, -inf
        else:
            e["initial_state"][0, :5] = inf  # (one that is erased leaves 0 here, 0 x infinity in the oracle)
        got, want, sizes = _bwd(e, _fwd(e)[2]), U.scan_grads_ref(e), U.scan_grads_ref(clean, True)
        _no_error()
        assert sum(np.isinf(want[j]).sum() for j in ("x", "z")) > 50
        for j in ("x", "z", "input_gate", "initial_state"):
            _same(j, got[j], want[j], sizes[j], 2 * n, U.U32 if j == "initial_state" else U.HALF[dtype])


@pytest.mark.filterwarnings("ignore:invalid value")
@pytest.mark.parametrize("dtype", DTYPES)
def test_step_keeps_infinities(dtype):
    d, pool, idx = _step_batch(3, 20, dtype, 5, 4, gate="log")
    pool[idx.long(), :4], d["z"][:, 2] = float("inf"), -float("inf")
    pool[idx[1].long(), 3] = -float("inf")
    d["initial_state"] = pool[idx.long()]
    p = pool.cuda()
    h = _step(d, p, idx)
    _no_error()
    want = U.scan_ref(d)[1]
    assert np.isinf(want).sum() == 9
    _same("h", h, want, abs(want), U.scan_roundings(d), U.HALF[dtype])
    _same("state", p[idx.long().cuda()], want, abs(want), U.scan_roundings(d), U.U32)


@pytest.mark.parametrize("dtype", DTYPES)
def test_nan_stays_in_its_channel(dtype):
    d = U.scan_batch([200, 150], 40, dtype, 5, gate="softplus", input_scale="norm")
    h0, last0, keep0 = _fwd(d)
    g0 = _bwd(d, keep0)
    d["x"][77, 13], d["z"][250, 20] = float("nan"), float("nan")
    h, last, keep = _fwd(d)
    g = _bwd(d, keep)
    _no_error()
    bad = torch.zeros((350, 40), dtype=torch.bool)
    bad[77:200, 13], bad[250:, 20] = True, True
    assert torch.equal(h.isnan().cpu(), bad) and torch.equal(h.cpu()[~bad], h0.cpu()[~bad])
    assert torch.equal(last.isnan().cpu(), torch.stack((bad[199], bad[349])))
    other = torch.ones(40, dtype=torch.bool)
    other[13] = other[20] = False
    for k in g:
        assert torch.equal(g[k].cpu()[..., other], g0[k].cpu()[..., other]), k


@pytest.mark.parametrize("dtype", DTYPES)
def test_views(dtype):
    """Slices of one projection, rows that begin at odd elements, the final state over the initial one."""
    d = U.scan_batch([90, 200], 64, dtype, 6)
    r = _fwd(d)
    g = _bwd(d, r[2])
    x = U.to(d)
    for pad in (0, 3):
        wide = torch.zeros((290, 3 * 64 + pad), dtype=U.DT[dtype], device="cuda")
        v = [wide[:, pad + 64 * k:pad + 64 * (k + 1)] for k in range(3)]
        for a, b in zip(v, ("x", "z", "input_gate")):
            a.copy_(x[b])
        state, keep = x["initial_state"].clone(), torch.full_like(r[2], float("nan"))
        h, last = kda.scan_fwd(*v, initial_state=state, final_state=state, checkpoints=keep, **_how(x))
        g2 = kda.scan_bwd(*v, x["grad_h"], keep, grad_final_state=x["grad_final_state"], **_how(x))
        _no_error()
        assert torch.equal(h, r[0]) and torch.equal(last, r[1]) and last is state
        assert all(torch.equal(g[k], g2[k]) for k in g)


@pytest.mark.parametrize("dtype", DTYPES)
def test_views_whose_rows_end_inside_a_copy(dtype):
    """100 of 104 channels: rows come by copies, whose last channels are others' (and NaN)."""
    d = U.scan_batch([90, 1, 200], 100, dtype, 24, input_scale="norm")
    r = _fwd(d)
    g = _bwd(d, r[2])
    x = U.to(d)
    for k in ("x", "z", "input_gate"):
        wide = torch.full((291, 104), float("nan"), dtype=U.DT[dtype], device="cuda")
        wide[:, :100] = x[k]
        x[k] = wide[:, :100]
    keep = torch.full_like(r[2], float("nan"))
    h, last = kda.scan_fwd(x["x"], x["z"], x["input_gate"], initial_state=x["initial_state"], output_final_state=True, checkpoints=keep, **_how(x))
    g2 = kda.scan_bwd(x["x"], x["z"], x["input_gate"], x["grad_h"], keep, grad_final_state=x["grad_final_state"], **_how(x))
    _no_error()
    assert torch.equal(h, r[0]) and torch.equal(last, r[1]) and all(torch.equal(g2[k], g[k]) for k in g)


def test_rows_far_apart():
    d = U.scan_batch([2, 1], 64, "bf16", 25)
    r = _fwd(d)
    g = _bwd(d, r[2])
    x = U.to(d)
    big = torch.empty((3, 1 << 29), dtype=torch.bfloat16, device="cuda")
    for i, k in enumerate(("x", "z", "input_gate")):
        big[:, 64 * i:64 * i + 64] = x[k]
        x[k] = big[:, 64 * i:64 * i + 64]
    h, last = kda.scan_fwd(x["x"], x["z"], x["input_gate"], initial_state=x["initial_state"], output_final_state=True, **_how(x))
    g2 = kda.scan_bwd(x["x"], x["z"], x["input_gate"], x["grad_h"], r[2], grad_final_state=x["grad_final_state"], **_how(x))
    _no_error()
    assert torch.equal(h, r[0]) and torch.equal(last, r[1]) and all(torch.equal(g2[k], g[k]) for k in g)


@pytest.mark.parametrize("dtype", DTYPES)
def test_another_lower_bound(dtype):
    """g_min: sequences, gradients and steps."""
    d = U.scan_batch([80], 48, dtype, 26, gate="lower_bound", input_scale="norm", state=False)
    x = U.to(d)
    keep = kda.scan_checkpoints(80, 1, 48)
    h, last = kda.scan_fwd(x["x"], x["z"], x["input_gate"], g_min=-0.5, checkpoints=keep, output_final_state=True, **_how(x))
    g = kda.scan_bwd(x["x"], x["z"], x["input_gate"], x["grad_h"], keep, g_min=-0.5, **_how(x))
    state, how = torch.zeros((1, 48), device="cuda"), {k: v for k, v in _how(x).items() if k != "cu_seqlens"}
    steps = torch.cat([kda.scan_step(x["x"][t:t + 1], x["z"][t:t + 1], x["input_gate"][t:t + 1], state, g_min=-0.5, **how) for t in range(80)])
    _no_error()
    a = [U.f64(d[k]) for k in ("x", "z", "input_gate", "A_log", "dt_bias")]
    want, size = (R.scan(f(a[0]), *a[1:], np.zeros(48), "lower_bound", -0.5, "norm") for f in (lambda v: v, np.abs))
    n, half = U.scan_roundings(d), U.HALF[dtype]
    U.close("h", h, want[0], size[0], n, half)
    U.close("final_state", last[0], want[2], size[2], n, U.U32)
    U.close("steps", steps, want[0], size[0], n, half)
    U.close("state", state[0], want[2], size[2], n, U.U32)
    want, size = (R.scan_grads(*a, np.zeros(48), U.f64(d["grad_h"]), np.zeros(48), "lower_bound", -0.5, "norm", magnitudes=m) for m in (False, True))
    for k, o in (("x", "x"), ("z", "z"), ("input_gate", "i"), ("A_log", "A"), ("dt_bias", "b")):
        U.close(k, g[k], want[o], size[o], 2 * n + 80, U.U32 if o in "Ab" else half)


def test_outputs_at_odd_elements():
    d = U.scan_batch([90, 200], 64, "bf16", 6)
    r = _fwd(d)
    buf = torch.zeros(290 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    for k in (1, 4):
        out = buf[k:k + 290 * 64].view(290, 64)
        buf.zero_()
        h = _fwd(d, out=out)[0]
        _no_error()
        assert h.data_ptr() == out.data_ptr() and torch.equal(h, r[0])
        assert (buf[:k] == 0).all() and (buf[k + 290 * 64:] == 0).all()


def test_same_bits_again():
    d = U.scan_batch([3000, 1, 700], 200, "bf16", 7, input_scale="norm")
    a = _fwd(d)
    g = _bwd(d, a[2])
    for _ in range(3):
        b = _fwd(d)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[2].nan_to_num(), b[2].nan_to_num())
        g2 = _bwd(d, a[2])
        assert all(torch.equal(g[k], g2[k]) for k in g)
    _no_error()


def test_a_sequence_does_not_depend_on_its_neighbours():
    """The same bits alone and in a batch whose tokens before it pass 2^32 elements."""
    D, T0, T1 = 8192, 530000, 200
    d = U.scan_batch([T1], D, "bf16", 8, gated=False)
    x = U.to(d)
    h1, last1 = kda.scan_fwd(x["x"], x["z"], initial_state=x["initial_state"], output_final_state=True, **_how(x))
    big = [torch.zeros((T0 + T1, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    big[0][T0:], big[1][T0:] = x["x"], x["z"]
    state = torch.cat((torch.zeros_like(x["initial_state"]), x["initial_state"]))
    how = {**_how(x), "cu_seqlens": U.cu([T0, T1]).cuda()}
    h2, last2 = kda.scan_fwd(*big, initial_state=state, output_final_state=True, **how)
    _no_error()
    assert torch.equal(h2[T0:], h1) and torch.equal(last2[1:], last1) and (h2[:T0:1000] == 0).all() and (last2[0] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,length", [(5, 320), (7, 127), (2, 512), (3, 1), (1, 1024), (400, 70)])
def test_the_same_bits_with_and_without_cu_seqlens(dtype, N, length):
    """Sequences of one length: their tiles are known before the call."""
    d = U.scan_batch([length] * N, 40, dtype, N, input_scale="norm")
    r = _fwd(d)
    g = _bwd(d, r[2])
    _check_fwd(d, r)
    _check_bwd(d, g)
    x = U.to(d)
    how = {**_how(x), "cu_seqlens": None, "n_seq": N}
    keep = torch.full_like(r[2], float("nan"))
    h, last = kda.scan_fwd(x["x"], x["z"], x["input_gate"], initial_state=x["initial_state"], output_final_state=True, checkpoints=keep, **how)
    g2 = kda.scan_bwd(x["x"], x["z"], x["input_gate"], x["grad_h"], keep, grad_final_state=x["grad_final_state"], **how)
    _no_error()
    assert torch.equal(h, r[0]) and torch.equal(last, r[1]) and torch.equal(keep.nan_to_num(7.0), r[2].nan_to_num(7.0))
    assert all(torch.equal(g2[k], g[k]) for k in g)


@pytest.mark.parametrize("T", (30, 700))
def test_bad_cu_seqlens_of_one_sequence(T):
    d = U.scan_batch([T], 24, "f32", 19)
    r = _fwd(d)
    for bad in ([0, T - 1], [1, T], [0, T + 1], [T, 0]):
        d["cu_seqlens"] = torch.tensor(bad, dtype=torch.int32)
        out, state = torch.full_like(r[0], 3.0), torch.full_like(r[1], 4.0)
        h, last, keep = _fwd(d, out=out, final_state=state)
        torch.cuda.synchronize()
        assert kda.get_device_error() == 7, bad
        assert h is out and (h == 3).all() and (state == 4).all() and keep.isnan().all()
        g = _bwd(d, r[2])
        torch.cuda.synchronize()
        assert kda.get_device_error() == 7, bad
        assert (g["A_log"] == 0).all() and (g["dt_bias"] == 0).all()


def test_two_calls_at_once():
    """Two streams, each with tensors and a workspace of its own; tiles that wait for one another."""
    ds = [U.scan_batch([4000, 100], 24, "bf16", 20), U.scan_batch([100, 6000, 3], 40, "bf16", 21, gate="sigmoid", input_scale="norm")]
    want = [_fwd(d) for d in ds]
    want = [(f, _bwd(d, f[2])) for d, f in zip(ds, want)]
    _no_error()
    streams, xs, got = [torch.cuda.Stream() for _ in ds], [U.to(d) for d in ds], [[] for _ in ds]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, x, d, f, o in zip(streams, xs, ds, [w[0] for w in want], got):
            with torch.cuda.stream(s):
                keep = torch.zeros_like(f[2])
                h, last = kda.scan_fwd(x["x"], x["z"], x["input_gate"], initial_state=x["initial_state"], output_final_state=True,
                                       checkpoints=keep, **_how(x))
                g = kda.scan_bwd(x["x"], x["z"], x["input_gate"], x["grad_h"], keep, grad_final_state=x["grad_final_state"], **_how(x))
                o.append((h, last, g))
    _no_error()
    for o, (f, g) in zip(got, want):
        for h, last, g2 in o:
            assert torch.equal(h, f[0]) and torch.equal(last, f[1]) and all(torch.equal(g2[k], g[k]) for k in g)


def test_bad_cu_seqlens():
    d = U.scan_batch([64, 100, 36], 40, "bf16", 9)
    x = U.to(d)
    good = _fwd(d)
    for bad in ([0, 64, 50, 200], [0, 64, 300, 200], [0, 64, 164, 190], [5, 64, 164, 200], [0, -7, 164, 200]):
        how = {**_how(x), "cu_seqlens": torch.tensor(bad, dtype=torch.int32).cuda()}
        out = torch.full_like(x["x"], 7.0)
        keep = torch.zeros((200 // 64 + 3, 40), device="cuda")
        kda.scan_fwd(x["x"], x["z"], x["input_gate"], initial_state=x["initial_state"], output_final_state=True, checkpoints=keep, out=out, **how)
        torch.cuda.synchronize()
        assert kda.get_device_error() == 7, bad
        if bad[1] == 64 and bad[0] == 0 and bad[2] >= 64:
            assert torch.equal(out[:64], good[0][:64])
        kda.scan_bwd(x["x"], x["z"], x["input_gate"], x["grad_h"], keep, **how)
        torch.cuda.synchronize()
        assert kda.get_device_error() == 7, bad


def test_streams_and_graphs():
    """Another stream; two captured graphs that share a workspace, replayed in turn with other contents."""
    d1, d2 = U.scan_batch([2000, 300], 72, "bf16", 10), U.scan_batch([700] * 3, 72, "bf16", 11, gate="sigmoid", input_scale="norm")
    want = [(_fwd(d), None) for d in (d1, d2)]
    want = [(f, _bwd(d, f[2])) for d, (f, _) in zip((d1, d2), want)]
    need = max(max(kda.scan_fwd_workspace_size(2300, 3, 72, torch.bfloat16), kda.scan_bwd_workspace_size(2300, 3, 72, torch.bfloat16)), 256)
    ws, stream, runs = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.cuda.Stream(), []
    torch.cuda.synchronize()
    for d in (d1, d2):
        x = U.to(d)
        src = {k: x[k].clone() for k in ("x", "z", "input_gate")}
        keep = torch.zeros((d["x"].shape[0] // 64 + len(d["lens"]), 72), device="cuda")

        def call(x=x, keep=keep):
            h, last = kda.scan_fwd(x["x"], x["z"], x["input_gate"], initial_state=x["initial_state"], output_final_state=True, checkpoints=keep,
                                   workspace=ws, **_how(x))
            return h, last, kda.scan_bwd(x["x"], x["z"], x["input_gate"], x["grad_h"], keep, grad_final_state=x["grad_final_state"], workspace=ws, **_how(x))

        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = call()
        runs.append((graph, x, src, out))
    for turn in range(3):
        for (graph, x, src, out), (f, g) in zip(runs, want):
            for k in src:
                x[k].copy_(src[k] if turn != 1 else torch.zeros_like(src[k]))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], f[0]) == (turn != 1)
            if turn != 1:
                assert torch.equal(out[1], f[1]) and all(torch.equal(out[2][k], g[k]) for k in g)
    _no_error()


def test_finite_checks():
    d = U.scan_batch([100, 30], 33, "bf16", 12)
    kda.set_debug_checks(kda.CHECK_FINITE)
    try:
        r = _fwd(d)
        assert kda.get_device_error() == 0
        _bwd(d, r[2])
        assert kda.get_device_error() == 0
        d["x"][120, 32] = float("inf")
        r = _fwd(d)
        assert kda.get_device_error() == 12
        _bwd(d, r[2])
        assert kda.get_device_error() == 12
    finally:
        kda.set_debug_checks(0)


# ---------------------------------------------------------------- single tokens
def _step_batch(N, D, dtype, seed, slots, **kw):
    d = U.scan_batch([1] * N, D, dtype, seed, **kw)
    g = torch.Generator().manual_seed(seed)
    pool = torch.randn((slots, D), generator=g)
    idx = torch.randperm(slots, generator=g)[:N].to(torch.int32)
    pool[idx.long()] = d["initial_state"]
    return d, pool, idx


def _step(d, pool, idx, **kw):
    x = U.to(d)
    how = _how(x)
    how.pop("cu_seqlens")
    return kda.scan_step(x["x"], x["z"], x["input_gate"], pool, state_indices=None if idx is None else idx.cuda(), **how, **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gate", U.GATES)
@pytest.mark.parametrize("N,D", [(1, 8), (5, 100), (3, 4096), (200, 33), (1, 1)])
def test_step(dtype, gate, N, D):
    d, pool, idx = _step_batch(N, D, dtype, N + D, N + 3, gate=gate, input_scale=U.INPUTS[N % 3], gated=N != 5)
    p = pool.cuda()
    h = _step(d, p, idx)
    _no_error()
    want, size, n = U.scan_ref(d), U.scan_ref(d, True), U.scan_roundings(d)
    U.close("h", h, want[0], size[0], n, U.HALF[dtype])
    U.close("state", p[idx.long().cuda()], want[1], size[1], n, U.U32)
    rest = torch.ones(N + 3, dtype=torch.bool)
    rest[idx.long()] = False
    assert torch.equal(p.cpu()[rest], pool[rest])
    q = pool[idx.long()].contiguous().cuda()
    assert torch.equal(_step(d, q, None), h) and torch.equal(q, p[idx.long().cuda()])


@pytest.mark.parametrize("dtype", DTYPES)
def test_step_padded_and_bad_rows(dtype):
    d, pool, idx = _step_batch(40, 50, dtype, 1, 60)
    want = _step(d, pool.cuda(), idx)
    bad = idx.clone()
    bad[[3, 17]] = -1
    bad[20], bad[30], bad[31] = 60, -5, bad[7]
    skipped = torch.tensor([3, 17, 20, 30, 31])
    p, out = pool.cuda(), torch.full((40, 50), 9.0, dtype=U.DT[dtype], device="cuda")
    h = _step(d, p, bad, out=out)
    torch.cuda.synchronize()
    assert kda.get_device_error() == 8 and h is out
    used = torch.ones(40, dtype=torch.bool)
    used[skipped] = False
    assert torch.equal(h.cpu()[used], want.cpu()[used]) and (h.cpu()[~used] == 9).all()
    untouched = torch.ones(60, dtype=torch.bool)
    untouched[idx.long()[used]] = False
    assert torch.equal(p.cpu()[untouched], pool[untouched])
    p = pool.cuda()
    _step(d, p, torch.full((40,), -1, dtype=torch.int32))
    _no_error()
    assert torch.equal(p.cpu(), pool)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad", (0, 3))
def test_step_views(dtype, pad):
    """Slices of one projection."""
    d, pool, idx = _step_batch(9, 64, dtype, 6, 12, input_scale="norm")
    p, q = pool.cuda(), pool.cuda()
    h = _step(d, p, idx)
    x = U.to(d)
    wide = torch.zeros((9, 3 * 64 + pad), dtype=U.DT[dtype], device="cuda")
    for i, k in enumerate(("x", "z", "input_gate")):
        v = wide[:, pad + 64 * i:pad + 64 * i + 64]
        v.copy_(x[k])
        x[k] = v
    h2 = _step(x, q, idx)
    _no_error()
    assert torch.equal(h2, h) and torch.equal(p, q)


def test_step_of_more_sequences_than_a_grid_is_high():
    N = 70000
    d, pool, idx = _step_batch(N, 5, "bf16", 12, N + 3)
    p = pool.cuda()
    h = _step(d, p, idx)
    _no_error()
    want, size, n = U.scan_ref(d), U.scan_ref(d, True), U.scan_roundings(d)
    U.close("h", h, want[0], size[0], n, U.HALF["bf16"])
    U.close("state", p[idx.long().cuda()], want[1], size[1], n, U.U32)


def test_step_slots_behind_32_bits():
    D, slots = 8192, 530000  # 4.3e9 elements
    d, pool, _ = _step_batch(2, D, "bf16", 3, 4)
    p = torch.empty((slots, D), device="cuda")
    idx = torch.tensor([slots - 1, 3], dtype=torch.int32)
    p[idx.long().cuda()] = d["initial_state"].cuda()
    h = _step(d, p, idx)
    _no_error()
    q = d["initial_state"].cuda()
    assert torch.equal(h, _step(d, q, None)) and torch.equal(p[idx.long().cuda()], q)


def test_step_finite_checks():
    d, pool, idx = _step_batch(6, 20, "bf16", 2, 9)
    idx[2] = -1
    rest = torch.ones(9, dtype=torch.bool)
    rest[idx[idx >= 0].long()] = False
    pool[rest] = float("nan")
    kda.set_debug_checks(kda.CHECK_FINITE)
    try:
        out = torch.full((6, 20), float("nan"), dtype=torch.bfloat16, device="cuda")
        p = pool.cuda()
        _step(d, p, idx, out=out)
        assert kda.get_device_error() == 0
        p[idx[5].long(), 19] = float("inf")
        _step(d, p, idx, out=out)
        assert kda.get_device_error() == 12
    finally:
        kda.set_debug_checks(0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [1, 3, 7])
def test_step_finite_checks_of_short_rows(dtype, D):
    d, pool, idx = _step_batch(3, D, dtype, 4, 5)
    kda.set_debug_checks(kda.CHECK_FINITE)
    try:
        p = pool.cuda()
        _step(d, p, idx)
        assert kda.get_device_error() == 0
        p[idx[2].long(), D - 1] = float("inf")
        _step(d, p, idx)
        assert kda.get_device_error() == 12
    finally:
        kda.set_debug_checks(0)


@pytest.mark.parametrize("gate,input_scale", [("softplus", "norm"), ("lower_bound", "complement")])
def test_steps_continue_a_prefill(gate, input_scale):
    """A prompt in two parts and then token by token, against one pass: fp32, each bound by the oracle."""
    d = U.scan_batch([150], 48, "f32", 13, gate=gate, input_scale=input_scale)
    x = U.to(d)
    how = _how(x)
    how.pop("cu_seqlens")
    at = lambda a, b: (x["x"][a:b], x["z"][a:b], x["input_gate"][a:b])  # noqa: E731
    h1, s = kda.scan_fwd(*at(0, 70), initial_state=x["initial_state"], output_final_state=True, **how)
    h2, s = kda.scan_fwd(*at(70, 140), initial_state=s, final_state=s, **how)
    rest = [kda.scan_step(*at(t, t + 1), s, **how) for t in range(140, 150)]
    _no_error()
    want, size, n = U.scan_ref(d), U.scan_ref(d, True), U.scan_roundings(d)
    U.close("h", torch.cat([h1, h2] + rest), want[0], size[0], n, U.U32)
    U.close("state", s, want[1], size[1], n, U.U32)
