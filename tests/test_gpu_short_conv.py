"""GPU tests of the short causal convolution (sequences, gradients, single tokens) against the fp64 oracle."""
import pytest
import torch

from linear_attention_kda_gb300 import kda
from oracle import layer_ref as R
from tests import layer_util as U

pytestmark = pytest.mark.gpu
DTYPES = ("f32", "bf16")
LENS = U.LENS + [2, 3, 4, 5]


def _no_error():
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0


def _fwd(d, **kw):
    x = U.to(d)
    kw = {**dict(cu_seqlens=x["cu_seqlens"], initial_state=x["initial_state"], output_final_state=True), **kw}
    return kda.short_conv_fwd(x["x"], x["weight"], x["bias"], activation=d["activation"], norm_dim=d["norm_dim"], **kw)


def _bwd(d, **kw):
    x = U.to(d)
    kw = {**dict(cu_seqlens=x["cu_seqlens"], initial_state=x["initial_state"], grad_final_state=x["grad_final_state"]), **kw}
    return kda.short_conv_bwd(x["x"], x["weight"], x["bias"], x["grad_y"], activation=d["activation"], norm_dim=d["norm_dim"], **kw)


# a sum of K terms, the activation's exponential (an argument up to 10 in size: 10 u), quotient and products, the sum
# of a head's squares (as a tree or in order, at most 256 terms), its root
def _roundings(d):
    return 40 + d["norm_dim"]


def _check_fwd(d, r):
    _no_error()
    y, tail = U.conv_ref(d)
    U.close("y", r[0], y, U.conv_sizes(d), _roundings(d), U.HALF[d["dtype"]])
    assert torch.equal(r[1].cpu().double(), torch.from_numpy(tail))  # histories are copies


def _check_bwd(d, g):
    _no_error()
    want, size = U.conv_grads_ref(d), U.conv_grads_ref(d, True)
    assert set(g) == {"x", "weight", "initial_state"} | ({"bias"} if d["bias"] is not None else set())
    for k in g:
        par = k in ("weight", "bias")
        # (s, ds and the norm are formed again: their errors come on top, relative to the same terms; the derivative of SiLU passes
        # through 0, where its error, a few u of 1, is one of what the oracle's size leaves out: |ds| + 0.1 covers it)
        sz = size[k] + 0.1 * abs(size[k]).max()
        U.close(k, g[k], want[k], sz, 4 * _roundings(d) + (d["x"].shape[0] if par else 0), U.U32 if par else U.HALF[d["dtype"]])


CASES = [(t, K, a, n) for t in DTYPES for K in (2, 3, 4) for a in ("silu", "none") for n in (0, 32, 128)] + \
        [(t, 4, "silu", n) for t in DTYPES for n in (64, 256)]


@pytest.mark.parametrize("dtype,K,act,norm", CASES)
def test_varlen(dtype, K, act, norm):
    d = U.conv_batch(LENS, 256 if norm else 136, K, dtype, K, act=act, norm=norm, bias=K != 3)
    _check_fwd(d, _fwd(d))
    _check_bwd(d, _bwd(d))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,norm", [(1, 0), (2, 0), (3, 0), (7, 0), (31, 0), (33, 0), (100, 0), (130, 0), (1032, 0), (32, 32), (96, 32), (64, 64), (192, 64),
                                    (384, 128), (768, 256), (4096, 128)])
def test_widths(dtype, D, norm):
    d = U.conv_batch([70, 2, 33], D, 4, dtype, D, norm=norm)
    _check_fwd(d, _fwd(d))
    _check_bwd(d, _bwd(d))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[1], [2], [5000], [1] * 200, [3] * 50, [0, 0, 7, 0]])
def test_lengths(dtype, lens):
    d = U.conv_batch(lens, 64, 4, dtype, len(lens), norm=64)
    _check_fwd(d, _fwd(d))
    _check_bwd(d, _bwd(d))


@pytest.mark.parametrize("dtype", DTYPES)
def test_without_history(dtype):
    d = U.conv_batch([40, 9], 64, 4, dtype, 1, state=False, bias=False)
    _check_fwd(d, _fwd(d))
    g = _bwd(d)
    _check_bwd(d, g)
    only = _bwd(d, param_grads=False, state_grad=False)
    assert set(only) == {"x"} and torch.equal(only["x"], g["x"])
    y, none = _fwd(d, output_final_state=False)
    assert none is None and torch.equal(y, _fwd(d)[0])
    e = U.conv_batch([50] * 4, 64, 4, dtype, 1, state=False, bias=False)
    assert torch.equal(_fwd(e)[0], _fwd(e, cu_seqlens=None, n_seq=4)[0])


@pytest.mark.parametrize("dtype", DTYPES)
def test_empty_batch(dtype):
    d = U.conv_batch([0, 0], 32, 3, dtype, 2)
    y, tail = _fwd(d)
    g = _bwd(d)
    _no_error()
    assert y.shape == (0, 32) and torch.equal(tail.cpu(), d["initial_state"]) and torch.equal(g["initial_state"].cpu(), d["grad_final_state"])
    assert (g["weight"] == 0).all() and (g["bias"] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_heads_of_zeros(dtype):
    """A head whose activations are all 0 gives 0 and passes 1 / sqrt(eps) of its gradient on, as the formula says."""
    d = U.conv_batch([30], 64, 4, dtype, 3, norm=32, bias=False, act="none", state=False)
    d["x"][:, :32] = 0
    d["grad_y"] *= 1e-3
    _check_fwd(d, _fwd(d))
    _check_bwd(d, _bwd(d))
    assert (_fwd(d)[0][:, :32] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_extreme_sums(dtype):
    """SiLU far out: 0 on one side, its argument on the other, and slopes of 0 and 1."""
    d = U.conv_batch([16], 8, 2, dtype, 4, bias=False, state=False)
    d["weight"][:, 0], d["weight"][:, 1] = 0.0, 1.0
    d["x"][:] = torch.tensor([-3e4, -200.0, -90.0, -30.0, 30.0, 90.0, 200.0, 3e4]).to(U.DT[dtype])
    y, g = _fwd(d)[0].double().cpu(), _bwd(d)["x"].double().cpu()
    _no_error()
    x = d["x"].double()
    assert (y[:, :3].abs() <= 1e-36).all() and (y[:, 4:] - x[:, 4:]).abs().max() <= 3e4 * U.HALF[dtype]
    assert (g[:, :3].abs() <= 1e-34).all() and torch.allclose(g[:, 5:], d["grad_y"].double()[:, 5:], rtol=1e-6)


def test_nan_stays_in_its_channel():
    d = U.conv_batch([60, 50], 64, 4, "bf16", 5)
    y0, g0 = _fwd(d)[0], _bwd(d)
    d["x"][20, 7] = float("nan")
    y, g = _fwd(d)[0], _bwd(d)
    _no_error()
    bad = torch.zeros((110, 64), dtype=torch.bool)
    bad[20:24, 7] = True
    assert torch.equal(y.isnan().cpu(), bad) and torch.equal(y.cpu()[~bad], y0.cpu()[~bad])
    gx = g["x"].isnan().cpu()
    bad[17:20, 7] = True
    assert torch.equal(gx, bad) and torch.equal(g["x"].cpu()[~bad], g0["x"].cpu()[~bad])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("norm", [0, 64])
def test_views(dtype, norm):
    d = U.conv_batch([90, 2, 108], 128, 4, dtype, 6, norm=norm)
    r, g = _fwd(d), _bwd(d)
    x = U.to(d)
    for pad in (0, 3):
        wide = torch.zeros((200, 256 + pad), dtype=U.DT[dtype], device="cuda")
        v = wide[:, pad + 128:]
        v.copy_(x["x"])
        state = x["initial_state"].clone()
        how = dict(activation="silu", norm_dim=norm, cu_seqlens=x["cu_seqlens"])
        y, last = kda.short_conv_fwd(v, x["weight"], x["bias"], initial_state=state, final_state=state, **how)
        g2 = kda.short_conv_bwd(v, x["weight"], x["bias"], x["grad_y"], initial_state=x["initial_state"], grad_final_state=x["grad_final_state"], **how)
        _no_error()
        assert torch.equal(y, r[0]) and torch.equal(last, r[1]) and last is state
        # the sums over tokens may be grouped otherwise where vectors are narrower, everything else may not differ
        assert torch.equal(g["x"], g2["x"]) and torch.equal(g["initial_state"], g2["initial_state"])
        size = U.conv_grads_ref(d, True)
        for k in ("weight", "bias"):
            U.close(k, g2[k], U.f64(g[k]), size[k], 2 * (4 * _roundings(d) + 200), 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("norm", [0, 32])
def test_views_whose_rows_end_inside_a_copy(dtype, norm):
    """96 or 100 of 104 channels: rows come by copies, whose last channels are others' (and NaN)."""
    D = 96 if norm else 100
    d = U.conv_batch([90, 1, 109], D, 4, dtype, 15, norm=norm)
    r, g = _fwd(d), _bwd(d)
    wide = torch.full((200, 104), float("nan"), dtype=U.DT[dtype], device="cuda")
    wide[:, :D] = d["x"].cuda()
    v = {**d, "x": wide[:, :D]}
    r2, g2 = _fwd(v), _bwd(v)
    _no_error()
    assert torch.equal(r2[0], r[0]) and torch.equal(r2[1], r[1]) and torch.equal(g2["x"], g["x"]) and torch.equal(g2["initial_state"], g["initial_state"])


def test_rows_far_apart():
    d = U.conv_batch([2, 1], 64, 4, "bf16", 16, norm=64)
    r, g = _fwd(d), _bwd(d)
    big = torch.empty((3, 1 << 29), dtype=torch.bfloat16, device="cuda")
    big[:, 64:128] = d["x"].cuda()
    v = {**d, "x": big[:, 64:128]}
    r2, g2 = _fwd(v), _bwd(v)
    _no_error()
    assert torch.equal(r2[0], r[0]) and torch.equal(r2[1], r[1]) and all(torch.equal(g2[k], g[k]) for k in g)


@pytest.mark.parametrize("dtype", DTYPES)
def test_another_eps(dtype):
    """norm_eps: sequences, gradients and steps."""
    eps = 0.3
    d = U.conv_batch([40], 64, 4, dtype, 17, norm=32)
    y, tail = _fwd(d, norm_eps=eps)
    g = _bwd(d, norm_eps=eps)
    state, x = d["initial_state"].cuda(), U.to(d)
    steps = torch.cat([kda.short_conv_step(x["x"][t:t + 1], x["weight"], x["bias"], state, norm_dim=32, norm_eps=eps) for t in range(40)])
    _no_error()
    a = [U.f64(d[k]) for k in ("x", "initial_state", "weight", "bias", "grad_y", "grad_final_state")]
    want, _ = R.conv(a[0], a[1][0], a[2], a[3], "silu", 32, eps)
    U.close("y", y, want, U.conv_sizes(d), _roundings(d), U.HALF[dtype])
    U.close("steps", steps, want, U.conv_sizes(d), _roundings(d), U.HALF[dtype])
    assert torch.equal(state, tail)
    want, size = (R.conv_grads(a[0], a[1][0], a[2], a[3], a[4], a[5][0], "silu", 32, eps, magnitudes=m) for m in (False, True))
    for k, o in (("x", "x"), ("weight", "w"), ("bias", "b")):
        U.close(k, g[k], want[o], size[o] + 0.1 * abs(size[o]).max(), 4 * _roundings(d) + 40, U.HALF[dtype] if k == "x" else U.U32)


def test_output_at_odd_elements():
    d = U.conv_batch([90, 110], 64, 4, "bf16", 7, norm=64)
    want = _fwd(d)[0]
    buf = torch.zeros(200 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    y = _fwd(d, out=buf[1:1 + 200 * 64].view(200, 64))[0]
    _no_error()
    assert torch.equal(y, want) and buf[0] == 0 and (buf[1 + 200 * 64:] == 0).all()


def test_bad_cu_seqlens():
    d = U.conv_batch([64, 100, 36], 64, 4, "bf16", 8)
    good = _fwd(d)[0]
    for bad in ([0, 64, 50, 200], [0, 64, 300, 200], [0, 64, 164, 190], [5, 64, 164, 200], [0, -7, 164, 200]):
        cu = torch.tensor(bad, dtype=torch.int32).cuda()
        out = torch.full_like(good, 7.0)
        _fwd(d, cu_seqlens=cu, out=out)
        torch.cuda.synchronize()
        assert kda.get_device_error() == 7, bad
        if bad[1] == 64 and bad[0] == 0 and bad[2] >= 64:
            assert torch.equal(out[:64], good[:64])
        _bwd(d, cu_seqlens=cu)
        torch.cuda.synchronize()
        assert kda.get_device_error() == 7, bad


def test_same_bits_again_and_graphs():
    d = U.conv_batch([3000, 1, 700], 256, 4, "bf16", 9, norm=128)
    r, g = _fwd(d), _bwd(d)
    x = U.to(d)
    how = dict(norm_dim=128, cu_seqlens=x["cu_seqlens"], initial_state=x["initial_state"])

    def call():
        y, last = kda.short_conv_fwd(x["x"], x["weight"], x["bias"], output_final_state=True, **how)
        return y, last, kda.short_conv_bwd(x["x"], x["weight"], x["bias"], x["grad_y"], grad_final_state=x["grad_final_state"], **how)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = call()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], r[0]) and torch.equal(out[1], r[1]) and all(torch.equal(out[2][k], g[k]) for k in g)
    _no_error()


def test_finite_checks():
    d = U.conv_batch([100, 30], 33, 4, "bf16", 10)
    kda.set_debug_checks(kda.CHECK_FINITE)
    try:
        _fwd(d), _bwd(d)
        assert kda.get_device_error() == 0
        d["x"][128, 32] = float("inf")
        _fwd(d)
        assert kda.get_device_error() == 12
        _bwd(d)
        assert kda.get_device_error() == 12
    finally:
        kda.set_debug_checks(0)


def test_a_sequence_does_not_depend_on_its_neighbours():
    """The same bits alone and behind more than 2^32 elements."""
    D, T0, T1 = 8192, 530000, 100
    d = U.conv_batch([T1], D, 4, "bf16", 11, norm=128, state=False)
    x = U.to(d)
    y1, t1 = kda.short_conv_fwd(x["x"], x["weight"], x["bias"], norm_dim=128, output_final_state=True)
    big = torch.zeros((T0 + T1, D), dtype=torch.bfloat16, device="cuda")
    big[T0:] = x["x"]
    y2, t2 = kda.short_conv_fwd(big, x["weight"], x["bias"], norm_dim=128, cu_seqlens=U.cu([T0, T1]).cuda(), output_final_state=True)
    _no_error()
    assert torch.equal(y2[T0:], y1) and torch.equal(t2[1:], t1)


def test_gradients_behind_32_bits():
    D, T0, lens = 8192, 264000, [100, 2, 70]
    d = U.conv_batch(lens, D, 4, "bf16", 14, norm=128)
    x, m = U.to(d), sum(lens)
    big = {k: torch.zeros((T0 + m, D), dtype=torch.bfloat16, device="cuda") for k in ("x", "grad_y")}
    for k in big:
        big[k][T0:] = x[k]
    hist, tail = (torch.cat((torch.zeros_like(x[k][:1]), x[k])) for k in ("initial_state", "grad_final_state"))
    g = kda.short_conv_bwd(big["x"], x["weight"], x["bias"], big["grad_y"], activation="silu", norm_dim=128, cu_seqlens=U.cu([T0] + lens).cuda(),
                           initial_state=hist, grad_final_state=tail)
    _no_error()
    assert (g["x"][:T0:1000] == 0).all()
    _check_bwd(d, {"x": g["x"][T0:], "weight": g["weight"], "bias": g["bias"], "initial_state": g["initial_state"][1:]})


# ---------------------------------------------------------------- single tokens
def _step(d, pool, idx, **kw):
    x = U.to(d)
    return kda.short_conv_step(x["x"], x["weight"], x["bias"], pool, activation=d["activation"], norm_dim=d["norm_dim"],
                               state_indices=None if idx is None else idx.cuda(), **kw)


def _step_batch(N, D, K, dtype, seed, slots, **kw):
    d = U.conv_batch([1] * N, D, K, dtype, seed, **kw)
    g = torch.Generator().manual_seed(seed)
    pool = torch.randn((slots, K - 1, D), generator=g).to(U.DT[dtype])
    idx = torch.randperm(slots, generator=g)[:N].to(torch.int32)
    pool[idx.long()] = d["initial_state"]
    return d, pool, idx


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,D,K,norm", [(1, 8, 4, 0), (5, 100, 2, 0), (3, 4096, 4, 128), (200, 33, 3, 0), (7, 256, 4, 256), (2, 96, 4, 32), (1, 64, 3, 64)])
def test_step(dtype, N, D, K, norm):
    d, pool, idx = _step_batch(N, D, K, dtype, N + D, N + 3, norm=norm, act="none" if N == 5 else "silu")
    p = pool.cuda()
    y = _step(d, p, idx)
    at = idx.long()
    _check_fwd(d, (y, p[at.cuda()]))
    rest = torch.ones(N + 3, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(p.cpu()[rest], pool[rest])
    q = pool[at].contiguous().cuda()
    assert torch.equal(_step(d, q, None), y) and torch.equal(q, p[at.cuda()])


@pytest.mark.parametrize("dtype", DTYPES)
def test_step_padded_and_bad_rows(dtype):
    d, pool, idx = _step_batch(40, 64, 4, dtype, 1, 60, norm=64)
    want = _step(d, pool.cuda(), idx)
    bad = idx.clone()
    bad[[3, 17]] = -1
    bad[20], bad[30], bad[31] = 60, -5, bad[7]
    used = torch.ones(40, dtype=torch.bool)
    used[[3, 17, 20, 30, 31]] = False
    p, out = pool.cuda(), torch.full((40, 64), 9.0, dtype=U.DT[dtype], device="cuda")
    y = _step(d, p, bad, out=out)
    torch.cuda.synchronize()
    assert kda.get_device_error() == 8 and y is out
    assert torch.equal(y.cpu()[used], want.cpu()[used]) and (y.cpu()[~used] == 9).all()
    untouched = torch.ones(60, dtype=torch.bool)
    untouched[idx.long()[used]] = False
    assert torch.equal(p.cpu()[untouched], pool[untouched])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad", (0, 3))
def test_step_views(dtype, pad):
    d, pool, idx = _step_batch(9, 64, 4, dtype, 14, 12, norm=64)
    p, q = pool.cuda(), pool.cuda()
    y = _step(d, p, idx)
    wide = torch.zeros((9, 128 + pad), dtype=U.DT[dtype], device="cuda")
    wide[:, pad:pad + 64] = d["x"].cuda()
    y2 = _step({**d, "x": wide[:, pad:pad + 64]}, q, idx)
    _no_error()
    assert torch.equal(y2, y) and torch.equal(p, q)


@pytest.mark.parametrize("dtype", DTYPES)
def test_steps_continue_a_prefill(dtype):
    """A prompt in two parts (one shorter than the taps) and then token by token: the bits of one pass."""
    d = U.conv_batch([80], 128, 4, dtype, 12, norm=64)
    x = U.to(d)
    how = dict(norm_dim=64)
    whole, last = kda.short_conv_fwd(x["x"], x["weight"], x["bias"], initial_state=x["initial_state"], output_final_state=True, **how)
    y1, s = kda.short_conv_fwd(x["x"][:68], x["weight"], x["bias"], initial_state=x["initial_state"], output_final_state=True, **how)
    y2, s = kda.short_conv_fwd(x["x"][68:70], x["weight"], x["bias"], initial_state=s, final_state=s, **how)
    rest = [kda.short_conv_step(x["x"][t:t + 1], x["weight"], x["bias"], s, **how) for t in range(70, 80)]
    _no_error()
    assert torch.equal(s, last)
    y, _ = U.conv_ref(d)
    U.close("y", torch.cat([y1, y2] + rest), y, U.conv_sizes(d), _roundings(d), U.HALF[dtype])
    U.close("y", whole, y, U.conv_sizes(d), _roundings(d), U.HALF[dtype])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,K", [(1, 2), (2, 3), (7, 2), (33, 4)])
def test_step_finite_checks(dtype, D, K):
    """Of the rows and slots that the step wrote alone, rows shorter than a vector among them."""
    d, pool, idx = _step_batch(6, D, K, dtype, 13, 9)
    idx[2] = -1
    rest = torch.ones(9, dtype=torch.bool)
    rest[idx[idx >= 0].long()] = False
    pool[rest] = float("nan")
    kda.set_debug_checks(kda.CHECK_FINITE)
    try:
        p, out = pool.cuda(), torch.full((6, D), float("nan"), dtype=U.DT[dtype], device="cuda")
        _step(d, p, idx, out=out)
        assert kda.get_device_error() == 0
        d["x"][5, D - 1] = float("inf")
        _step(d, p, idx, out=out)
        assert kda.get_device_error() == 12
    finally:
        kda.set_debug_checks(0)
