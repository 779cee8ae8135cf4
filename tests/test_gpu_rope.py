"""GPU tests of kda_rope against angles reduced in exact arithmetic."""
import decimal
import math

import pytest
import torch

from linear_attention_kda_gb300 import kda

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
DT = {"f32": (torch.float32, U32), "bf16": (torch.bfloat16, 2.0 ** -8)}
TWO_PI = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def _angles(positions, freqs):
    """positions * freqs modulo 2 pi, the product and the reduction in 60 digits."""
    out = torch.empty((len(positions), len(freqs)), dtype=torch.float64)
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        for i, p in enumerate(positions.tolist()):
            for j, f in enumerate(freqs.tolist()):
                out[i, j] = float((decimal.Decimal(f) * p) % TWO_PI)
    return out


def _want(x, positions, freqs, layout, scale, inverse):
    x, r = x.double(), 2 * len(freqs)
    a = _angles(positions, freqs)
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None] * (-1 if inverse else 1)
    i, j = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    y, m = x.clone(), torch.zeros_like(x)
    y[..., i], y[..., j] = scale * (x[..., i] * c - x[..., j] * s), scale * (x[..., j] * c + x[..., i] * s)
    m[..., i] = m[..., j] = abs(scale) * (x[..., i].abs() + x[..., j].abs())
    return y, m


def _check(got, x, positions, freqs, layout, scale, inverse, dtype):
    want, terms = _want(x.cpu(), positions.cpu(), freqs, layout, scale, inverse)
    r = 2 * len(freqs)
    # sine and cosine: 2^-25 half turns from the fp32 fraction (9.4e-8) and two steps of the function (2.4e-7 at most),
    # 6 U32 together; scale, product and sum: 3 roundings
    bound = 9 * U32 * terms + DT[dtype][1] * want.abs() + 1e-37
    assert ((got.double().cpu() - want).abs() <= bound)[..., :r].all()
    assert torch.equal(got[..., r:].cpu(), x[..., r:].cpu())


def _inputs(T, Hq, Hk, d, dtype, seed, top=1 << 20):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((T, Hq, d), generator=g).to(DT[dtype][0]).cuda()
    k = torch.randn((T, Hk, d), generator=g).to(DT[dtype][0]).cuda()
    return q, k, torch.randint(0, top, (T,), generator=g).to(torch.int32).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hk,d,rot", [(1, 1, 1, 2, 2), (5, 3, 1, 64, 64), (9, 2, 2, 128, 64), (7, 4, 2, 80, 40), (3, 2, 1, 50, 6),
                                           (17, 1, 1, 256, 256), (2, 5, 3, 1024, 32), (33, 8, 2, 128, 128), (4, 2, 2, 96, 90)])
def test_rotation(dtype, layout, T, Hq, Hk, d, rot):
    q, k, pos = _inputs(T, Hq, Hk, d, dtype, T)
    f = kda.rope_frequencies(rot)
    yq, yk = kda.rope(q, k, pos, f, layout=layout, scale=1.25)
    torch.cuda.synchronize()
    _check(yq, q, pos, f, layout, 1.25, False, dtype)
    _check(yk, k, pos, f, layout, 1.25, False, dtype)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_and_negative_positions(layout):
    q, k, _ = _inputs(8, 1, 1, 64, "f32", 3)
    pos = torch.tensor([0, 1, -1, 1 << 23, (1 << 31) - 1, -(1 << 31), 123456789, -987654321], dtype=torch.int32).cuda()
    for f in (kda.rope_frequencies(64), kda.rope_frequencies(64, 5e5, "linear", 32.0), -kda.rope_frequencies(64), 100.0 * kda.rope_frequencies(64)):
        yq, yk = kda.rope(q, k, pos, f, layout=layout)
        torch.cuda.synchronize()
        _check(yq, q, pos, f, layout, 1.0, False, "f32")
        _check(yk, k, pos, f, layout, 1.0, False, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_inverse_is_the_gradient(dtype, layout):
    """The derivative of sum(rope(x) * w) is the inverse rotation of w (against autograd of the formula, fp64)."""
    q, w, pos = _inputs(6, 2, 2, 64, dtype, 4)
    f = kda.rope_frequencies(32)
    got, none = kda.rope(w, None, pos, f, layout=layout, scale=0.5, inverse=True)
    assert none is None
    x = q.double().cpu().requires_grad_()
    y = torch.empty_like(x)
    a = _angles(pos, f)
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    i, j = (slice(0, 16), slice(16, 32)) if layout == "half" else (slice(0, 32, 2), slice(1, 32, 2))
    y = x.clone()
    y[..., i] = 0.5 * (x[..., i] * c - x[..., j] * s)
    y[..., j] = 0.5 * (x[..., j] * c + x[..., i] * s)
    (y * w.double().cpu()).sum().backward()
    _check(got, w, pos, f, layout, 0.5, True, dtype)
    terms = _want(w.cpu(), pos.cpu(), f, layout, 0.5, True)[1]
    assert ((got.double().cpu() - x.grad).abs() <= 9 * U32 * terms + DT[dtype][1] * x.grad.abs() + 1e-37).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [64, 24])
def test_in_place_and_strided(dtype, layout, rot):
    """q and k as slices of one fused projection, rotated where they lie; the values between them stay."""
    T, Hq, Hk, d = 13, 4, 2, 64
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn((T, (Hq + 2 * Hk) * d), generator=g).to(DT[dtype][0]).cuda()
    _, _, pos = _inputs(T, 1, 1, 2, dtype, 6)
    f = kda.rope_frequencies(rot)
    before = qkv.clone()
    q, k = qkv[:, :Hq * d].view(T, Hq, d), qkv[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
    wq, wk = kda.rope(q, k, pos, f, layout=layout)  # to new tensors
    assert torch.equal(qkv, before)
    rq, rk = kda.rope(q, k, pos, f, layout=layout, out_q=q, out_k=k)
    torch.cuda.synchronize()
    assert rq is q and rk is k and torch.equal(q, wq) and torch.equal(k, wk)
    assert torch.equal(qkv[:, (Hq + Hk) * d:], before[:, (Hq + Hk) * d:])
    _check(wq, before[:, :Hq * d].view(T, Hq, d), pos, f, layout, 1.0, False, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_unaligned_views(dtype, layout, shift):
    """Rows that start at odd elements (of an odd stride) take the element-wise form."""
    T, H, d = 5, 2, 32
    buf = torch.randn((T * (H * d + shift) + 8,), generator=torch.Generator().manual_seed(7)).to(DT[dtype][0]).cuda()
    x = buf[shift:shift + T * (H * d + shift)].view(T, H * d + shift)[:, :H * d].view(T, H, d)
    _, _, pos = _inputs(T, 1, 1, 2, dtype, 8)
    f = kda.rope_frequencies(32)
    y, _ = kda.rope(x, None, pos, f, layout=layout)
    torch.cuda.synchronize()
    _check(y, x, pos, f, layout, 1.0, False, dtype)


def test_many_tokens():
    """Whole tensors of a prefill, compared on samples of tokens (first, last, between)."""
    q, k, pos = _inputs(70001, 8, 2, 128, "bf16", 9, 1 << 30)
    f = kda.rope_frequencies(128, 5e5)
    yq, yk = kda.rope(q, k, pos, f)
    torch.cuda.synchronize()
    at = torch.tensor([0, 1, 2, 31, 32, 35000, 69998, 69999, 70000])
    _check(yq[at.cuda()], q[at.cuda()], pos[at.cuda()], f, "half", 1.0, False, "bf16")
    _check(yk[at.cuda()], k[at.cuda()], pos[at.cuda()], f, "half", 1.0, False, "bf16")


def test_captured_and_replayed():
    q, k, pos = _inputs(20, 2, 2, 64, "f32", 10)
    f = kda.rope_frequencies(64)
    kda.rope(q, k, pos, f)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yq, yk = kda.rope(q, k, pos, f.clone())  # the frequencies are read during the call only
    q2, k2, pos2 = _inputs(20, 2, 2, 64, "f32", 11)
    for x, y in ((q, q2), (k, k2), (pos, pos2)):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    _check(yq, q2, pos2, f, "half", 1.0, False, "f32")
    _check(yk, k2, pos2, f, "half", 1.0, False, "f32")


def test_rotated_products_depend_on_the_distance_alone():
    """q rotated at m and k at n give the product of q and k turned by m - n, also far out."""
    q, k, _ = _inputs(1, 1, 1, 64, "f32", 12)
    f = kda.rope_frequencies(64)
    q, k = q.expand(4, 1, 64).contiguous(), k.expand(4, 1, 64).contiguous()
    m = torch.tensor([5, 1005, 1000005, 2000000005], dtype=torch.int32).cuda()
    yq, _ = kda.rope(q, None, m, f)
    _, yk = kda.rope(None, k, m - 3, f)
    s = (yq.double() * yk.double()).sum(-1).flatten()
    # each rotated value is off by 9 U32 of its pair: the product of two rows by 2 * 9 * U32 * 2 |q| |k|
    assert float((s - s[0]).abs().max()) <= 2 * 36 * U32 * float(q[0].norm() * k[0].norm())
    assert math.isfinite(float(s[0]))
