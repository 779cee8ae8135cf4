"""GPU tests of linear attention with a decay per head (prefill, gradients, decode) against the fp64 oracle."""
import numpy as np
import pytest
import torch

from linear_attention_kda_gb300 import kda
from tests import linear_util as LU

pytestmark = pytest.mark.gpu
HEADS = {"all": {}, "shared_qk": dict(Hq=2, Hk=2), "shared_kv": dict(Hk=1, Hv=1), "mixed": dict(Hq=4, Hk=1, Hv=2)}


def _no_error():
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0


def _run_fwd(d, **kw):
    x = LU.to(d, "cuda")
    r = kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], scale=d["scale"], cu_seqlens=x["cu_seqlens"],
                             initial_state=x["initial_state"], output_final_state=True, **kw)
    _no_error()
    return r


def _run_bwd(d, **kw):
    x = LU.to(d, "cuda")
    r = kda.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["grad_o"], scale=d["scale"], cu_seqlens=x["cu_seqlens"],
                             initial_state=x["initial_state"], grad_final_state=x["grad_final_state"], **kw)
    _no_error()
    return r


# bf16 operands that the tensor-core path rounds: the masked products and the state of an output, dA or A and a state
# of a gradient (one rounding in each term); what goes into fp32 results is kept as two bf16 parts, 2^-16 of a term.
def _per_term(d, fp32_result):
    n = LU.ops(d) * LU.U32
    return n if d["q"].dtype == torch.float32 else n + (2.0 ** -15 if fp32_result else LU.EPS_BF16)


def _step(d):
    return LU.U32 if d["q"].dtype == torch.float32 else LU.EPS_BF16


def _check_fwd(d, o, S):
    (ro, rS), (ao, aS) = LU.forward_ref(d), LU.forward_ref(d, True)
    LU.close("o", o, ro, ao, _per_term(d, False), _step(d))
    LU.close("final_state", S, rS, aS, _per_term(d, True), LU.U32)


def _check_bwd(d, r):
    w, a = LU.backward_ref(d), LU.backward_ref(d, True)
    for n in ("q", "k", "v"):
        LU.close(n, r[n], w[n], a[n], _per_term(d, False), _step(d))
    LU.close("initial_state", r["initial_state"], w["initial_state"], a["initial_state"], _per_term(d, True), LU.U32)
    if d["g"] is not None:
        # two states are multiplied: both of their errors count
        if d["g"].dim() == 2:
            LU.close("g", r["g"], w["g_tokens"], a["g_terms"], 2 * _per_term(d, True), LU.U32)
        else:
            LU.close("g", r["g"], w["g_tokens"].sum(0), a["g_terms"].sum(0), 2 * _per_term(d, True), LU.U32)


CASES = [(t, dk, dv, "all", "token") for t in ("f32", "bf16") for dk in (64, 128) for dv in (64, 128)] + \
        [(t, 128, 128, h, "token") for t in ("f32", "bf16") for h in ("shared_qk", "shared_kv", "mixed")] + \
        [(t, 64, 128, "shared_qk", g) for t in ("f32", "bf16") for g in ("head", "none")]


@pytest.mark.parametrize("dtype,dk,dv,heads,decay", CASES)
def test_forward_varlen(dtype, dk, dv, heads, decay):
    d = LU.batch(LU.LENS, 4, dk, dv, dtype, 1, decay=decay, **HEADS[heads])
    _check_fwd(d, *_run_fwd(d))


@pytest.mark.parametrize("dtype,dk,dv,heads,decay", CASES)
def test_backward_varlen(dtype, dk, dv, heads, decay):
    d = LU.batch(LU.LENS, 4, dk, dv, dtype, 2, decay=decay, **HEADS[heads])
    _check_bwd(d, _run_bwd(d))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 128, 129, 255, 257, 640, 1500])
def test_one_sequence(dtype, T):
    """One sequence of one or three heads, without states or cu_seqlens."""
    d = LU.batch([T], 3 if T % 2 else 1, 128, 128, dtype, T, state=False)
    x = LU.to(d, "cuda")
    o, S = kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], scale=d["scale"], output_final_state=True)
    r = kda.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["grad_o"], scale=d["scale"])
    _no_error()
    _check_fwd(d, o, S)
    _check_bwd(d, r)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_lengths_without_cu_seqlens(dtype):
    d = LU.batch([77] * 5, 2, 64, 64, dtype, 9)
    x = LU.to(d, "cuda")
    o, S = kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], scale=d["scale"], n_seq=5,
                                initial_state=x["initial_state"], output_final_state=True)
    r = kda.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["grad_o"], scale=d["scale"], n_seq=5,
                             initial_state=x["initial_state"], grad_final_state=x["grad_final_state"])
    _no_error()
    _check_fwd(d, o, S)
    _check_bwd(d, r)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_short_sequences(dtype):
    """More sequences than one 32-way search step holds, most of them shorter than a chunk."""
    lens = [(7 * i) % 41 for i in range(70)]
    d = LU.batch(lens, 2, 64, 128, dtype, 4)
    _check_fwd(d, *_run_fwd(d))
    _check_bwd(d, _run_bwd(d))


@pytest.mark.parametrize("N,Hq,Hk,Hv,dk,dv,decay,state", [(770, 2, 2, 8, 64, 64, "token", True),
                                                         (770, 2, 1, 8, 64, 64, "head", False),
                                                         (390, 4, 1, 8, 64, 128, "none", True),
                                                         (390, 2, 4, 8, 128, 64, "token", False),
                                                         (770, 8, 2, 2, 64, 64, "token", True),
                                                         (770, 8, 1, 2, 64, 64, "head", False),
                                                         (390, 8, 2, 1, 64, 128, "token", True),
                                                         (390, 8, 4, 2, 128, 64, "none", False),
                                                         (200, 8, 2, 2, 128, 128, "token", True)])
def test_backward_many_chunks_of_shared_heads(N, Hq, Hk, Hv, dk, dv, decay, state):
    """Chunks enough that a block runs over several of the 8 heads that share a row of q and k, or of k and v: all of
    them, or some; ragged and whole chunks, sequences of one chunk and of several, with and without states at the ends."""
    lens = [300, 256, 0, 128, 130] + [(5 * i) % 11 for i in range(N - 5)]
    d = LU.batch(lens, 8, dk, dv, "bf16", N + Hq, Hq=Hq, Hk=Hk, Hv=Hv, decay=decay, state=state)
    r = _run_bwd(d)
    _check_bwd(d, r)
    again = _run_bwd(d)
    for n in r:
        assert r[n] is None or torch.equal(r[n], again[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_erasing_decays(dtype):
    """Log-decays of -inf, far below exp's range, and zero, alone and in runs."""
    d = LU.batch([300, 64, 5], 2, 128, 128, dtype, 6)
    g = d["g"]
    g[0] = -np.inf
    g[10:13] = -1e6
    g[70:200, 0] = -150.0
    g[70:200, 1] = 0.0
    g[200] = -np.inf
    g[301:304] = -104.0
    g[364:] = -np.inf
    _check_fwd(d, *_run_fwd(d))
    _check_bwd(d, _run_bwd(d))


def test_slow_decay_long_sum():
    """No decay at all over many chunks: every token stays in the state."""
    d = LU.batch([2048], 1, 64, 64, "f32", 8, decay="none")
    _check_fwd(d, *_run_fwd(d))
    _check_bwd(d, _run_bwd(d))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_decay_stays_in_its_sequence_and_head(dtype):
    d = LU.batch([100, 90, 80], 2, 64, 64, dtype, 10)
    ok, okS = _run_fwd(d)
    bad = dict(d, g=d["g"].clone())
    bad["g"][120, 1] = float("nan")
    o, S = _run_fwd(bad)
    assert torch.isnan(o[120:190, 1]).all() and torch.isnan(S[1, 1]).all()
    same = torch.ones(o.shape[:2], dtype=torch.bool, device="cuda")
    same[120:190, 1] = False
    assert torch.equal(o[same], ok[same])
    assert torch.equal(S[[0, 2]], okS[[0, 2]]) and torch.equal(S[1, 0], okS[1, 0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_no_number_stays_in_its_sequence(dtype, value):
    """The neighbours of a sequence full of NaN or infinities, ragged ends in its chunks, keep every bit."""
    d = LU.batch([100, 77, 130, 3], 2, 64, 128, dtype, 19)
    bad = dict(d)
    for n in ("q", "k", "v", "grad_o"):
        bad[n] = d[n].clone()
        bad[n][100:177] = value
    keep = torch.ones(310, dtype=torch.bool, device="cuda")
    keep[100:177] = False
    (o, S), (bo, bS), r, br = _run_fwd(d), _run_fwd(bad), _run_bwd(d), _run_bwd(bad)
    assert torch.equal(o[keep], bo[keep]) and torch.equal(S[[0, 2, 3]], bS[[0, 2, 3]])
    for n in ("q", "k", "v", "g"):
        assert torch.equal(r[n][keep], br[n][keep]), n
    assert torch.equal(r["initial_state"][[0, 2, 3]], br["initial_state"][[0, 2, 3]])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_batch_and_empty_sequences(dtype):
    d = LU.batch([0, 0, 0], 2, 128, 64, dtype, 3)
    x = LU.to(d, "cuda")
    o, S = _run_fwd(d)
    assert torch.equal(S, x["initial_state"]) and o.numel() == 0
    r = _run_bwd(d)
    assert torch.equal(r["initial_state"], x["grad_final_state"])
    d = LU.batch([0, 0, 0], 2, 128, 64, dtype, 3, decay="head")
    assert torch.equal(_run_bwd(d)["g"], torch.zeros(2, device="cuda"))
    d = LU.batch([0, 40, 0], 2, 128, 64, dtype, 3)
    S = _run_fwd(d)[1]
    assert torch.equal(S[[0, 2]].cpu(), d["initial_state"][[0, 2]])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeats_to_the_bit_on_a_dirty_workspace(dtype):
    d = LU.batch([200, 0, 331], 4, 128, 128, dtype, 12, decay="head", **HEADS["mixed"])
    N, T = 3, 531
    wf = kda.linear_chunk_fwd_workspace_size(T, N, 4, 128, 128, LU.DT[dtype])
    wb = kda.linear_chunk_bwd_workspace_size(T, N, 4, 128, 128, LU.DT[dtype], 4, 1, 2)
    nan = lambda n: torch.full((-(-max(n, 4) // 4),), float("nan"), device="cuda")  # noqa: E731
    o, S = _run_fwd(d)
    o2, S2 = _run_fwd(d, workspace=nan(wf))
    assert torch.equal(o, o2) and torch.equal(S, S2)
    r, r2 = _run_bwd(d), _run_bwd(d, workspace=nan(wb))
    for n in r:
        assert torch.equal(r[n], r2[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_final_state_over_initial_state(dtype):
    d = LU.batch([90, 200], 2, 128, 128, dtype, 13)
    o, S = _run_fwd(d)
    x = LU.to(d, "cuda")
    o2, S2 = kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], scale=d["scale"], cu_seqlens=x["cu_seqlens"],
                                  initial_state=x["initial_state"], final_state=x["initial_state"])
    _no_error()
    assert torch.equal(o, o2) and torch.equal(S, S2) and S2.data_ptr() == x["initial_state"].data_ptr()


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("lens", [[3000], [2500, 0, 130, 1], [1, 128, 4100]])
def test_few_long_sequences(dk, dv, lens):
    """Few chains of many chunks (cut into segments), the final states written over the initial ones."""
    d = LU.batch(lens, 2, dk, dv, "bf16", sum(lens))
    o, S = _run_fwd(d)
    _check_fwd(d, o, S)
    x = LU.to(d, "cuda")
    o2, S2 = kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], scale=d["scale"], cu_seqlens=x["cu_seqlens"],
                                  initial_state=x["initial_state"], final_state=x["initial_state"])
    _no_error()
    assert torch.equal(o, o2) and torch.equal(S, S2)
    _check_bwd(d, _run_bwd(d))


@pytest.mark.parametrize("lens,Hq,dk,dv,decay,state", [([1, 9000, 130, 0], 2, 64, 64, "token", True),
                                                     ([0, 129, 8000, 1], 1, 128, 64, "head", False),
                                                     ([9100], 2, 64, 128, "none", True)])
def test_gradients_of_few_chains_cut_into_segments(lens, Hq, dk, dv, decay, state):
    """Segments of a sequence that others stand beside, with and without states at its ends."""
    d = LU.batch(lens, 2, dk, dv, "bf16", len(lens), Hq=Hq, decay=decay, state=state)
    r = _run_bwd(d)
    _check_bwd(d, r)
    again = _run_bwd(d, workspace=torch.full((kda.linear_chunk_bwd_workspace_size(
        sum(lens), len(lens), 2, dk, dv, torch.bfloat16, Hq=Hq),), 255, dtype=torch.uint8, device="cuda"))
    _no_error()
    for n in r:
        assert torch.equal(r[n], again[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_split_prompt_equals_whole(dtype):
    """Two calls, the second from the first one's state, against the oracle of the whole."""
    d = LU.batch([333], 2, 128, 64, dtype, 14)
    x = LU.to(d, "cuda")
    S, outs = x["initial_state"], []
    for a, b in ((0, 101), (101, 333)):
        o, S = kda.linear_chunk_fwd(x["q"][a:b].contiguous(), x["k"][a:b].contiguous(), x["v"][a:b].contiguous(),
                                    x["g"][a:b].contiguous(), scale=d["scale"], initial_state=S, output_final_state=True)
        outs.append(o)
    _no_error()
    _check_fwd(d, torch.cat(outs), S)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cu", [[0, 60, 50, 120], [1, 60, 90, 120], [0, 60, 90, 119], [0, -5, 90, 120], [0, 60, 500, 120]])
def test_bad_cu_seqlens_is_reported(dtype, cu):
    d = LU.batch([60, 30, 30], 2, 64, 64, dtype, 15)
    x = LU.to(d, "cuda")
    bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
    kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], cu_seqlens=bad, output_final_state=True)
    assert kda.get_device_error() == 7
    kda.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["grad_o"], cu_seqlens=bad)
    assert kda.get_device_error() == 7
    assert kda.get_device_error() == 0


@pytest.mark.parametrize("H,N", [(1, 1), (5, 2), (64, 3), (7, 130)])
def test_batches_of_other_shapes(H, N):
    """One head, many heads, more sequences than are sorted by length; bf16 against the fp32 kernels on the same values
    (each is checked against the oracle elsewhere): the difference is both bounds'."""
    lens = [(37 * i + 5 * H) % 190 for i in range(N)]
    d = LU.batch(lens, H, 64, 64, "bf16", H + N)
    f = {n: x.float() if isinstance(x, torch.Tensor) and x.dtype == torch.bfloat16 else x for n, x in d.items()}
    (o, S), (fo, fS) = _run_fwd(d), _run_fwd(f)
    mo, mS = (torch.from_numpy(x).cuda() for x in LU.forward_ref(d, True))
    assert ((o.double() - fo.double()).abs() <= 2 * _per_term(d, False) * mo + LU.EPS_BF16 * fo.double().abs() + 1e-37).all()
    assert ((S.double() - fS.double()).abs() <= 2 * _per_term(d, True) * mS + 1e-37).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_behind_the_last_sequence_stay(dtype):
    d = LU.batch([60, 30, 30], 2, 64, 64, dtype, 16)
    x = LU.to(d, "cuda")
    short = torch.tensor([0, 60, 90, 90], dtype=torch.int32, device="cuda")
    out = torch.full((120, 2, 64), 7.0, dtype=LU.DT[dtype], device="cuda")
    kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], scale=d["scale"], cu_seqlens=short, out=out,
                         initial_state=x["initial_state"])
    assert kda.get_device_error() == 7  # sequence lengths do not add up to T
    assert (out[90:] == 7.0).all()
    ok, _ = _run_fwd(d)
    assert torch.equal(out[:90], ok[:90])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_and_replayed(dtype):
    """Forward and backward in one graph, replayed with other contents (lengths among them) in the same buffers."""
    d = LU.batch([130, 40, 200], 2, 128, 128, dtype, 17)
    e = LU.batch([10, 300, 60], 2, 128, 128, dtype, 18)
    x = LU.to(d, "cuda")

    def calls():
        o, S = kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], scale=d["scale"], cu_seqlens=x["cu_seqlens"],
                                    initial_state=x["initial_state"], output_final_state=True)
        return o, S, kda.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["grad_o"], scale=d["scale"],
                                          cu_seqlens=x["cu_seqlens"], initial_state=x["initial_state"],
                                          grad_final_state=x["grad_final_state"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, S, r = calls()
    for b in (d, e, d):
        for n, t in x.items():
            if isinstance(t, torch.Tensor):
                t.copy_(b[n])
        graph.replay()
        graph.replay()
        _no_error()
        _check_fwd(b, o, S)
        _check_bwd(b, r)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_streams_at_once(dtype):
    d = [LU.batch([500, 130], 4, 128, 128, dtype, 20 + i) for i in range(2)]
    want = [(_run_fwd(x), _run_bwd(x)) for x in d]
    xs, got = [LU.to(x, "cuda") for x in d], [None, None]
    streams = [torch.cuda.Stream() for _ in d]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (x, s) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(s):
                f = kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], scale=0.75, cu_seqlens=x["cu_seqlens"],
                                         initial_state=x["initial_state"], output_final_state=True)
                b = kda.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["grad_o"], scale=0.75,
                                         cu_seqlens=x["cu_seqlens"], initial_state=x["initial_state"],
                                         grad_final_state=x["grad_final_state"])
                got[i] = (f, b)
    _no_error()
    for (f, b), (wf, wb) in zip(got, want):
        assert torch.equal(f[0], wf[0]) and torch.equal(f[1], wf[1])
        assert all(torch.equal(b[n], wb[n]) for n in wb)


def test_gradients_against_differences():
    """The fp32 gradients against differences of the fp32 forward, one direction in all inputs."""
    d = LU.batch([150, 70], 2, 64, 64, "f32", 30, decay="token")
    r, x = _run_bwd(d), LU.to(d, "cuda")
    gen = torch.Generator().manual_seed(31)
    names = ("q", "k", "v", "g", "initial_state")
    move = {n: torch.randn(d[n].shape, generator=gen) * (0.1 if n == "g" else 1.0) for n in names}
    e = 2.0 ** -8

    def loss(sign):
        y = {n: x[n] + sign * e * move[n].cuda() for n in names}
        o, S = kda.linear_chunk_fwd(y["q"], y["k"], y["v"], y["g"], scale=0.75, cu_seqlens=x["cu_seqlens"],
                                    initial_state=y["initial_state"], output_final_state=True)
        return float((o.double() * x["grad_o"].double()).sum() + (S.double() * x["grad_final_state"].double()).sum())

    num = (loss(1) - loss(-1)) / (2 * e)
    ana = sum(float((r[n].double().cpu() * move[n].double()).sum()) for n in names)
    # the third derivative's part, e^2 / 6 = 2.5e-6 of it, and the forward's rounding: 1e5 outputs of size 10 with
    # errors of 1e-6 of themselves, independent, over 2 e: 1e-6 * 10 * 300 / (1 / 128) = 0.4 on sums of order 1e3
    assert abs(num - ana) <= 1e-3 * abs(ana) + 1.0


# ------------------------------------------------------------------------------------------------ decode
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv,heads,decay", [(64, 64, "all", "token"), (128, 64, "shared_qk", "head"), (64, 128, "shared_kv", "none"),
                                               (128, 128, "mixed", "token"), (128, 128, "all", "head")])
@pytest.mark.parametrize("N", [1, 5, 150])
def test_step(dtype, dk, dv, heads, decay, N):
    d = LU.batch([1] * N, 4, dk, dv, dtype, 40 + N, decay=decay, **HEADS[heads])
    (ro, rS), (ao, aS) = LU.forward_ref(d), LU.forward_ref(d, True)
    slots = N + 3
    gen = torch.Generator().manual_seed(1)
    at = torch.randperm(slots, generator=gen)[:N]
    pool = torch.randn((slots, 4, dk, dv), generator=gen)
    before = pool.clone()
    pool[at] = d["initial_state"]
    x, pool = LU.to(d, "cuda"), pool.cuda()
    o = kda.linear_recurrent_step(x["q"], x["k"], x["v"], x["g"], pool, scale=0.75, state_indices=at.to(torch.int32).cuda())
    _no_error()
    LU.close("o", o, ro, ao, (dk + 40) * LU.U32, _step(d))
    LU.close("state", pool.cpu()[at], rS, aS, 8 * LU.U32, LU.U32)
    rest = torch.ones(slots, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(pool.cpu()[rest], before[rest])


def test_step_without_indices_and_erasing():
    d = LU.batch([1] * 3, 2, 64, 64, "f32", 50)
    d["g"][1] = -np.inf
    (ro, rS), (ao, aS) = LU.forward_ref(d), LU.forward_ref(d, True)
    x = LU.to(d, "cuda")
    o = kda.linear_recurrent_step(x["q"], x["k"], x["v"], x["g"], x["initial_state"], scale=0.75)
    _no_error()
    LU.close("o", o, ro, ao, 104 * LU.U32, LU.U32)
    LU.close("state", x["initial_state"], rS, aS, 8 * LU.U32, LU.U32)


@pytest.mark.parametrize("N", [5, 600])
def test_step_padded_duplicate_and_bad_rows(N):
    """-1 rows leave everything alone; a slot given twice is the first row's; a slot outside the pool is reported."""
    d = LU.batch([1] * N, 1, 64, 64, "f32", 51)
    x = LU.to(d, "cuda")
    pool = torch.randn((N, 1, 64, 64), generator=torch.Generator().manual_seed(2)).cuda()
    idx = torch.arange(N, dtype=torch.int32)
    good, out = pool.clone(), torch.full((N, 1, 64), 7.0, device="cuda")
    want = kda.linear_recurrent_step(x["q"], x["k"], x["v"], x["g"], good)
    _no_error()
    idx[1] = -1
    p = pool.clone()
    kda.linear_recurrent_step(x["q"], x["k"], x["v"], x["g"], p, state_indices=idx.cuda(), out=out)
    _no_error()
    assert (out[1] == 7.0).all() and torch.equal(p[1], pool[1])
    assert torch.equal(out[2:], want[2:]) and torch.equal(p[2:], good[2:])
    for value in (0, N, -2):
        idx[N - 1] = value
        p, o = pool.clone(), out.clone()
        kda.linear_recurrent_step(x["q"], x["k"], x["v"], x["g"], p, state_indices=idx.cuda(), out=o)
        assert kda.get_device_error() == 8
        assert torch.equal(o[:N - 1], out[:N - 1]) and torch.equal(p[:N - 1][idx[:N - 1] >= 0], good[:N - 1][idx[:N - 1] >= 0])
        assert torch.equal(p[N - 1], pool[N - 1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steps_continue_a_prefill(dtype):
    d = LU.batch([97], 2, 128, 128, dtype, 52)
    x = LU.to(d, "cuda")
    cut = lambda n, a, b: x[n][a:b].contiguous()  # noqa: E731
    o, S = kda.linear_chunk_fwd(*(cut(n, 0, 90) for n in ("q", "k", "v", "g")), scale=0.75,
                                initial_state=x["initial_state"], output_final_state=True)
    outs = [o] + [kda.linear_recurrent_step(*(cut(n, t, t + 1) for n in ("q", "k", "v", "g")), S, scale=0.75)
                  for t in range(90, 97)]
    _no_error()
    _check_fwd(d, torch.cat(outs), S)


def test_debug_checks_see_the_linear_calls():
    d = LU.batch([40], 1, 64, 64, "f32", 53)
    x = LU.to(d, "cuda")
    kda.set_debug_checks(kda.CHECK_FINITE)
    try:
        kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], output_final_state=True)
        kda.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["grad_o"])
        _no_error()
        x["v"][3, 0, 0] = float("inf")
        kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], output_final_state=True)
        assert kda.get_device_error() == 12
        kda.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["grad_o"])
        assert kda.get_device_error() == 12
    finally:
        kda.set_debug_checks(0)
