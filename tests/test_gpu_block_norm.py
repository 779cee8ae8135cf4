"""GPU tests of the norms around a block with its gate and residual scale, against the fp64 oracle."""
import ctypes

import pytest
import torch

from linear_attention_kda_gb300 import kda
from oracle import layer_ref as R
from tests import layer_util as U

pytestmark = pytest.mark.gpu
TYPES = (("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"))


def _no_error():
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0


def _fwd(d, **kw):
    x = U.to(d)
    return kda.block_norm_fwd(x["y"], x["residual"], x["gate"], **U.norm_options(x), **kw)


def _bwd(d, **kw):
    x = U.to(d)
    return kda.block_norm_bwd(x["y"], x["residual"], x["gate"], x["grad_residual"], x["grad_normed"], **U.norm_options(x), **kw)


# a mean of squares (a tree of at most 16 in order, then halves: 16 + 9 + 16 roundings, halved by the root), the gate's sigmoid (an
# argument up to 6: 10 u) and a handful of products; a row's mean of signed terms, 41 roundings of its magnitudes
ROUNDINGS = 100


def _check_fwd(d, r):
    _no_error()
    y, res, g, s, post, pre = U.norm_args(d)
    want = R.block_norm(y, res, g, s, post, pre)
    term = abs(want[0] - res) + abs(res)
    U.close("residual", r[0], want[0], term, ROUNDINGS, U.HALF[d["res"]])
    if pre is None:
        assert r[1] is None
    else:
        k = abs(want[1]) / abs(want[0]).clip(1e-300)
        U.close("normed", r[1], want[1], term * k + abs(want[1]), ROUNDINGS, U.HALF[d["dtype"]])


def _check_bwd(d, g, tokens=None):
    _no_error()
    y, res, gt, s, post, pre = U.norm_args(d)
    dr, dn = U.f64(d["grad_residual"]), U.f64(d["grad_normed"])
    want = R.block_norm_grads(y, res, gt, s, post, pre, dr, dn)
    size = R.block_norm_grads(y, res, gt, s, post, pre, dr, dn, magnitudes=True)
    names = {"residual": "r", "y": "y", "gate": "gate", "post_weight": "post", "pre_weight": "pre", "scale": "scale"}
    expect = {"residual", "y"} | ({"gate"} if gt is not None else set()) | {k for k in ("post_weight", "pre_weight") if d[k] is not None} | (
        {"scale"} if isinstance(d["scale"], torch.Tensor) else set())
    assert set(g) == expect
    for k in g:
        par = k in ("post_weight", "pre_weight", "scale")
        half = U.U32 if par else U.HALF[d["res" if k == "residual" else "dtype"]]
        # r' is formed again with its own errors, relative to |r| + |scale p|: rows of 2 and 1, so that r' may be 20 times smaller than either
        # in an element but not in a row; 3 for the row's share
        U.close(k, g[k], want[names[k]], 3 * size[names[k]] + (0 if k == "residual" and pre is None else 0.05 * size[names[k]].max()),
                3 * ROUNDINGS + (d["T"] if par or k == "gate" else 0), half)


CASES = [(t, g, p, v) for t in TYPES for g in ("channel", "token", "none") for p in ((True, True), (True, False), (False, True), (False, False))
         for v in (True, False)]


@pytest.mark.parametrize("types,gate,norms,vec", CASES)
def test_parts(types, gate, norms, vec):
    d = U.norm_batch(37, 264, types[0], 1, res=types[1], gate=gate, post=norms[0], pre=norms[1], vec=vec)
    _check_fwd(d, _fwd(d))
    _check_bwd(d, _bwd(d))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", [1, 2, 3, 8, 31, 64, 100, 256, 257, 264, 512, 520, 1000, 1024, 1032, 2048, 2049, 2056, 4096, 4100, 4104, 7168, 8191, 8192])
def test_widths(types, D):
    d = U.norm_batch(5, D, types[0], D, res=types[1])
    _check_fwd(d, _fwd(d))
    if D > 3:  # with fewer channels the norm leaves hardly any gradient: a difference of equal numbers
        _check_bwd(d, _bwd(d))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T", [1, 2, 3, 151, 153, 700, 5000])
def test_tokens(types, T):
    d = U.norm_batch(T, 128, types[0], T, res=types[1])
    _check_fwd(d, _fwd(d))
    _check_bwd(d, _bwd(d))


def test_empty():
    d = U.norm_batch(0, 64, "bf16", 1)
    r, n = _fwd(d)
    g = _bwd(d)
    _no_error()
    assert r.shape == n.shape == (0, 64) and all((g[k] == 0).all() for k in ("post_weight", "pre_weight", "scale"))


@pytest.mark.parametrize("types", TYPES)
def test_norm_without_weights(types):
    d = U.norm_batch(20, 96, types[0], 2, res=types[1])
    one = torch.ones(96)
    x = U.to({**d, "post_weight": None, "pre_weight": None})
    a = kda.block_norm_fwd(x["y"], x["residual"], x["gate"], scale=x["scale"])
    b = _fwd({**d, "post_weight": one, "pre_weight": one})
    g = kda.block_norm_bwd(x["y"], x["residual"], x["gate"], x["grad_residual"], x["grad_normed"], scale=x["scale"])
    g1 = _bwd({**d, "post_weight": one, "pre_weight": one})
    _no_error()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and set(g) == {"y", "residual", "gate", "scale"}
    assert all(torch.equal(g[k], g1[k]) for k in g)


@pytest.mark.parametrize("types", TYPES)
def test_first_norm(types):
    """In front of the first block: the norm of the residual stream alone."""
    d = U.norm_batch(20, 96, types[0], 3, res=types[1])
    x = U.to(d)
    out = torch.empty((20, 96), dtype=U.DT[types[0]], device="cuda")
    r, n = kda.block_norm_fwd(None, x["residual"], pre_weight=x["pre_weight"], normed=out)
    g = kda.block_norm_bwd(None, x["residual"], None, x["grad_residual"], x["grad_normed"], pre_weight=x["pre_weight"])
    _no_error()
    assert r is x["residual"] and n is out and set(g) == {"residual", "pre_weight"}
    res, pre = U.f64(d["residual"]), U.f64(d["pre_weight"])
    want = R.block_norm(None, res, None, 1.0, None, pre)[1]
    U.close("normed", n, want, abs(want), ROUNDINGS, U.HALF[types[0]])
    a = [R.block_norm_grads(None, res, None, 1.0, None, pre, U.f64(d["grad_residual"]), U.f64(d["grad_normed"]), magnitudes=m) for m in (False, True)]
    U.close("residual", g["residual"], a[0]["r"], a[1]["r"], 3 * ROUNDINGS, U.HALF[types[1]])
    U.close("pre_weight", g["pre_weight"], a[0]["pre"], a[1]["pre"], ROUNDINGS + 20, U.U32)


@pytest.mark.parametrize("types", TYPES)
def test_gradients_of_one_output(types):
    d = U.norm_batch(20, 96, types[0], 4, res=types[1])
    x = U.to(d)
    for miss in ("grad_residual", "grad_normed"):
        e = {**d, miss: torch.zeros_like(d[miss])}
        gr, gn = (None if k == miss else x[k] for k in ("grad_residual", "grad_normed"))
        g = kda.block_norm_bwd(x["y"], x["residual"], x["gate"], gr, gn, **U.norm_options(x))
        _check_bwd(e, g)
    only = _bwd(d, param_grads=False)
    assert set(only) == {"y", "residual", "gate"} and torch.equal(only["y"], _bwd(d)["y"])


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", [96, 101])
def test_in_place(types, D):
    d = U.norm_batch(33, D, types[0], 5, res=types[1])
    want, g = _fwd(d), _bwd(d)
    x = U.to(d)
    r, n = kda.block_norm_fwd(x["y"], x["residual"], x["gate"], residual_out=x["residual"], normed=x["y"], **U.norm_options(x))
    _no_error()
    assert r is x["residual"] and n is x["y"] and torch.equal(r, want[0]) and torch.equal(n, want[1])
    for over in ("y", "grad_normed"):  # by the C call: gradients over y or grad_normed, and over grad_residual_out
        x = U.to(d)
        L = kda.load_library()
        ws = torch.empty(kda.block_norm_bwd_workspace_size(33, D, U.DT[types[0]]), dtype=torch.uint8, device="cuda")
        w = {k: torch.empty(D, device="cuda") for k in ("post_weight", "pre_weight", "scale")}
        gate = torch.empty_like(x["gate"])
        code = {"f32": 0, "bf16": 1}
        p = lambda t: t.data_ptr()  # noqa: E731
        a = kda.BlockNormBwdArgs(T=33, D=D, dtype=code[types[0]], residual_dtype=code[types[1]], gate_kind=1, post_norm=1, pre_norm=1, eps=1e-6,
                                 scale=1.0, scale_vec=p(x["scale"]), y=p(x["y"]), gate=p(x["gate"]), residual=p(x["residual"]),
                                 post_weight=p(x["post_weight"]), pre_weight=p(x["pre_weight"]), grad_residual_out=p(x["grad_residual"]),
                                 grad_normed=p(x["grad_normed"]), grad_y=p(x[over]), grad_gate=p(gate), grad_residual=p(x["grad_residual"]),
                                 grad_post_weight=p(w["post_weight"]), grad_pre_weight=p(w["pre_weight"]), grad_scale=p(w["scale"]))
        assert L.kda_block_norm_bwd(ctypes.byref(a), p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
        _no_error()
        assert torch.equal(x[over], g["y"]) and torch.equal(x["grad_residual"], g["residual"]) and torch.equal(gate, g["gate"])
        assert all(torch.equal(w[k], g[k]) for k in w)


@pytest.mark.parametrize("types", TYPES)
def test_rows_of_zeros_and_large_values(types):
    """y = 0 leaves r and passes dp / sqrt(eps) on; rows of 1e15 (whose squares' sum is far from fp32's end) are as good as others."""
    d = U.norm_batch(12, 64, types[0], 6, res=types[1])
    d["y"][3] = 0
    d["y"][5], d["residual"][5] = 0, 0
    d["y"][7] *= 1e15
    d["grad_residual"] *= 1e-3
    d["grad_normed"] *= 1e-3
    r = _fwd(d)
    _check_fwd(d, r)
    assert torch.equal(r[0][3].cpu(), d["residual"][3]) and (r[1][5] == 0).all()
    g = _bwd(d)
    _no_error()
    y, res, gt, s, post, pre = U.norm_args(d)
    want = R.block_norm_grads(y, res, gt, s, post, pre, U.f64(d["grad_residual"]), U.f64(d["grad_normed"]))
    size = R.block_norm_grads(y, res, gt, s, post, pre, U.f64(d["grad_residual"]), U.f64(d["grad_normed"]), magnitudes=True)
    for k in ("y", "residual"):
        n = "r" if k == "residual" else k
        # by rows: each has a scale of its own
        sz = 3 * size[n] + 0.05 * size[n].max(-1, keepdims=True)
        U.close(k, g[k], want[n], sz, 3 * ROUNDINGS, U.HALF[types[1] if k == "residual" else types[0]])


def test_nan_stays_in_its_row():
    d = U.norm_batch(40, 200, "bf16", 7)
    r0, g0 = _fwd(d), _bwd(d, param_grads=False)
    d["y"][11, 5], d["gate"][20, 100], d["residual"][30, 0] = float("nan"), float("inf"), float("nan")
    d["gate"][21, 100] = -float("inf")
    r, g = _fwd(d), _bwd(d, param_grads=False)
    _no_error()
    bad = torch.zeros(40, dtype=torch.bool)
    bad[[11, 30]] = True
    assert torch.equal(r[1].isnan().any(-1).cpu(), bad) and torch.equal(g["y"].isnan().any(-1).cpu(), bad)
    same = ~bad
    same[[20, 21]] = False
    assert all(torch.equal(a.cpu()[same], b.cpu()[same]) for a, b in zip(r + tuple(g.values()), r0 + tuple(g0.values())))
    assert g["gate"][20, 100] == 0 and g["gate"][21, 100] == 0  # a gate at its end has no slope


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("D", [101, 264, 1024])
def test_gradients_of_infinities_without_a_norm(types, gate, D):
    """Without its norm y's gradient is scale * sigmoid(gate) * dr', whatever y is."""
    d = U.norm_batch(20, D, types[0], 12, res=types[1], gate=gate, post=False, pre=False)
    want = _bwd(d)
    d["y"][3, 5], d["y"][4, 6], d["y"][7, 0] = float("inf"), -float("inf"), float("nan")
    g = _bwd(d)
    _no_error()
    assert torch.equal(g["y"], want["y"]) and torch.equal(g["residual"], want["residual"]) and want["y"].isfinite().all()


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", [101, 264, 1024])
def test_another_eps(types, D):
    d = U.norm_batch(40, D, types[0], 13, res=types[1])
    r, g = _fwd(d, eps=0.3), _bwd(d, eps=0.3)
    _no_error()
    y, res, gate, s, post, pre = U.norm_args(d)
    dr, dn = U.f64(d["grad_residual"]), U.f64(d["grad_normed"])
    want = R.block_norm(y, res, gate, s, post, pre, 0.3)
    U.close("residual", r[0], want[0], abs(want[0] - res) + abs(res), ROUNDINGS, U.HALF[types[1]])
    U.close("normed", r[1], want[1], (abs(want[0] - res) + abs(res)) * abs(want[1]) / abs(want[0]).clip(1e-300) + abs(want[1]), ROUNDINGS, U.HALF[types[0]])
    want, size = (R.block_norm_grads(y, res, gate, s, post, pre, dr, dn, 0.3, magnitudes=m) for m in (False, True))
    for k, o in (("residual", "r"), ("y", "y"), ("gate", "gate"), ("post_weight", "post"), ("pre_weight", "pre"), ("scale", "scale")):
        par = k in ("post_weight", "pre_weight", "scale")
        half = U.U32 if par else U.HALF[types[1] if k == "residual" else types[0]]
        U.close(k, g[k], want[o], 3 * size[o] + 0.05 * size[o].max(), 3 * ROUNDINGS + (40 if par else 0), half)


# ---------------------------------------------------------------- rows above 512 channels, several to a block: copies into places that are taken in turn
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,D", [(3100, 520), (3100, 1024), (1300, 2048), (1300, 4096), (700, 7168), (700, 8192)])
def test_many_wide_rows(types, T, D):
    d = U.norm_batch(T, D, types[0], D, res=types[1])
    _check_fwd(d, _fwd(d))
    _check_bwd(d, _bwd(d))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("gate", ["channel", "token", "none"])
@pytest.mark.parametrize("norms", [(True, True), (True, False), (False, True), (False, False)])
def test_parts_of_many_wide_rows(types, gate, norms):
    d = U.norm_batch(1900, 1024, types[0], 14, res=types[1], gate=gate, post=norms[0], pre=norms[1], vec=norms[0])
    _check_fwd(d, _fwd(d))
    _check_bwd(d, _bwd(d))


@pytest.mark.parametrize("types", TYPES)
def test_one_gradient_of_many_wide_rows(types):
    d = U.norm_batch(1900, 1024, types[0], 15, res=types[1])
    x = U.to(d)
    for miss in ("grad_residual", "grad_normed"):
        gr, gn = (None if k == miss else x[k] for k in ("grad_residual", "grad_normed"))
        _check_bwd({**d, miss: torch.zeros_like(d[miss])}, kda.block_norm_bwd(x["y"], x["residual"], x["gate"], gr, gn, **U.norm_options(x)))


@pytest.mark.parametrize("types", TYPES)
def test_first_norm_of_many_wide_rows(types):
    d = U.norm_batch(1900, 1024, types[0], 16, res=types[1])
    x = U.to(d)
    g = kda.block_norm_bwd(None, x["residual"], None, x["grad_residual"], x["grad_normed"], pre_weight=x["pre_weight"])
    _no_error()
    a = [R.block_norm_grads(None, U.f64(d["residual"]), None, 1.0, None, U.f64(d["pre_weight"]), U.f64(d["grad_residual"]), U.f64(d["grad_normed"]),
                            magnitudes=m) for m in (False, True)]
    U.close("residual", g["residual"], a[0]["r"], a[1]["r"], 3 * ROUNDINGS, U.HALF[types[1]])
    U.close("pre_weight", g["pre_weight"], a[0]["pre"], a[1]["pre"], ROUNDINGS + 1900, U.U32)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("over", ["y", "grad_normed"])
def test_many_wide_rows_in_place(types, over):
    """By the C call: gradients over y or grad_normed, and over grad_residual_out."""
    T, D, code = 1900, 1024, {"f32": 0, "bf16": 1}
    d = U.norm_batch(T, D, types[0], 17, res=types[1])
    want, x = _bwd(d), U.to(d)
    ws = torch.empty(kda.block_norm_bwd_workspace_size(T, D, U.DT[types[0]]), dtype=torch.uint8, device="cuda")
    w, gate = {k: torch.empty(D, device="cuda") for k in ("post_weight", "pre_weight", "scale")}, torch.empty_like(x["gate"])
    p = {k: v.data_ptr() for k, v in x.items() if isinstance(v, torch.Tensor)}
    a = kda.BlockNormBwdArgs(T=T, D=D, dtype=code[types[0]], residual_dtype=code[types[1]], gate_kind=1, post_norm=1, pre_norm=1, eps=1e-6, scale=1.0,
                             scale_vec=p["scale"], y=p["y"], gate=p["gate"], residual=p["residual"], post_weight=p["post_weight"],
                             pre_weight=p["pre_weight"], grad_residual_out=p["grad_residual"], grad_normed=p["grad_normed"], grad_y=p[over],
                             grad_gate=gate.data_ptr(), grad_residual=p["grad_residual"], grad_post_weight=w["post_weight"].data_ptr(),
                             grad_pre_weight=w["pre_weight"].data_ptr(), grad_scale=w["scale"].data_ptr())
    stream = torch.cuda.current_stream().cuda_stream
    assert kda.load_library().kda_block_norm_bwd(ctypes.byref(a), ws.data_ptr(), ws.numel(), stream) == 0
    _no_error()
    assert torch.equal(x[over], want["y"]) and torch.equal(x["grad_residual"], want["residual"]) and torch.equal(gate, want["gate"])
    assert all(torch.equal(w[k], want[k]) for k in w)


def test_gradients_behind_32_bits():
    D, T = 8192, 264000
    d = U.norm_batch(3, D, "bf16", 18, gate="token")
    x = U.to(d)
    big = {k: torch.zeros((T, D) if x[k].dim() == 2 else (T,), dtype=torch.bfloat16, device="cuda")
           for k in ("y", "residual", "gate", "grad_residual", "grad_normed")}
    for k in big:
        big[k][-3:] = x[k]
    g = kda.block_norm_bwd(big["y"], big["residual"], big["gate"], big["grad_residual"], big["grad_normed"], **U.norm_options(x))
    _check_bwd(d, {k: v[-3:] if k in ("y", "residual", "gate") else v for k, v in g.items()})
    assert (g["residual"][:-3:1000] == 0).all() and (g["y"][:-3:1000] == 0).all()


def test_same_bits_again_and_graphs():
    d = U.norm_batch(3000, 1024, "bf16", 8, res="f32")
    r, g = _fwd(d), _bwd(d)
    x = U.to(d)

    def call():
        return kda.block_norm_fwd(x["y"], x["residual"], x["gate"], **U.norm_options(x)) + (
            kda.block_norm_bwd(x["y"], x["residual"], x["gate"], x["grad_residual"], x["grad_normed"], **U.norm_options(x)),)

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


def test_tensors_at_odd_elements():
    d = U.norm_batch(30, 96, "bf16", 9, res="f32")
    want, g = _fwd(d), _bwd(d)
    x = U.to(d)
    for k in ("y", "gate", "grad_normed", "residual", "grad_residual"):
        buf = torch.zeros(30 * 96 + 1, dtype=x[k].dtype, device="cuda")
        buf[1:] = x[k].reshape(-1)
        x[k] = buf[1:].view(30, 96)
    r = kda.block_norm_fwd(x["y"], x["residual"], x["gate"], **U.norm_options(x))
    _check_fwd(d, r)
    _check_bwd(d, kda.block_norm_bwd(x["y"], x["residual"], x["gate"], x["grad_residual"], x["grad_normed"], **U.norm_options(x)))


def test_rows_behind_32_bits():
    D, T = 8192, 530000
    d = U.norm_batch(3, D, "bf16", 10, gate="token")
    x = U.to(d)
    want, g = _fwd(d), _bwd(d, param_grads=False)
    big = {k: torch.zeros((T, D) if x[k].dim() == 2 else (T,), dtype=torch.bfloat16, device="cuda") for k in ("y", "residual", "gate")}
    for k in big:
        big[k][-3:] = x[k]
    r, n = kda.block_norm_fwd(big["y"], big["residual"], big["gate"], **U.norm_options(x))
    _no_error()
    assert torch.equal(r[-3:], want[0]) and torch.equal(n[-3:], want[1]) and (r[:-3:1000] == 0).all()


def test_finite_checks():
    d = U.norm_batch(30, 101, "bf16", 11, res="f32")
    kda.set_debug_checks(kda.CHECK_FINITE)
    try:
        _fwd(d), _bwd(d)
        assert kda.get_device_error() == 0
        d["y"][29, 100] = float("inf")
        _fwd(d)
        assert kda.get_device_error() == 12
        _bwd(d)
        assert kda.get_device_error() == 12
    finally:
        kda.set_debug_checks(0)
