"""Host-side checks (no GPU) of the gated recurrence, short convolution and block norm calls: struct layouts, refusals."""
import ctypes
import os
import subprocess

import pytest
import torch

from linear_attention_kda_gb300 import build as kbuild, kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 32  # far apart, 16-byte aligned addresses that nothing dereferences
BF16, F32 = kda.KDA_BF16, kda.KDA_F32
STRUCTS = {"kda_scan_args": kda.ScanArgs, "kda_scan_bwd_args": kda.ScanBwdArgs, "kda_scan_step_args": kda.ScanStepArgs,
           "kda_short_conv_args": kda.ShortConvArgs, "kda_short_conv_bwd_args": kda.ShortConvBwdArgs,
           "kda_short_conv_step_args": kda.ShortConvStepArgs, "kda_block_norm_args": kda.BlockNormArgs,
           "kda_block_norm_bwd_args": kda.BlockNormBwdArgs}
FUNCTION = {s: c[:-5] + ("_fwd" if c in ("kda_scan_args", "kda_short_conv_args", "kda_block_norm_args") else "") for c, s in STRUCTS.items()}
WITH_WORKSPACE = (kda.ScanArgs, kda.ScanBwdArgs, kda.ShortConvBwdArgs, kda.BlockNormBwdArgs)


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


@pytest.fixture
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("valid arguments with made-up addresses must not reach a GPU")


def test_struct_layouts(tmp_path):
    rows = "".join(f'printf("{c} sizeof %zu\\n", sizeof({c}));\n' + "".join(
        f'printf("{c} {f} %zu\\n", offsetof({c}, {f}));\n' for f, _ in s._fields_) for c, s in STRUCTS.items())
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "kda.h"\nint main(void) {\n' + rows + "return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        c, f, v = line.split()
        s = STRUCTS[c]
        assert int(v) == (ctypes.sizeof(s) if f == "sizeof" else getattr(s, f).offset), (c, f)


def _make(struct, defaults, **kw):
    """Arguments with an address of their own for every pointer that neither names; `at(name)` finds it."""
    a = {f: (i + 1) * FAKE for i, (f, t) in enumerate(struct._fields_) if t is ctypes.c_void_p}
    return struct(**{**a, **defaults, **kw})


def at(struct, name):
    return (1 + [f for f, _ in struct._fields_].index(name)) * FAKE


def _scan(**kw):
    return _make(kda.ScanArgs, dict(T=128, N=2, D=64, dtype=BF16, gate_kind=1, input_scale=0, g_min=-5.0), **kw)


def _scan_bwd(**kw):
    return _make(kda.ScanBwdArgs, dict(T=128, N=2, D=64, dtype=BF16, gate_kind=1, input_scale=0, g_min=-5.0), **kw)


def _scan_step(**kw):
    return _make(kda.ScanStepArgs, dict(N=4, D=64, dtype=BF16, gate_kind=1, input_scale=0, g_min=-5.0, num_slots=9), **kw)


def _conv(**kw):
    return _make(kda.ShortConvArgs, dict(T=128, N=2, D=256, K=4, dtype=BF16, activation=1, norm_dim=128, norm_eps=1e-6), **kw)


def _conv_bwd(**kw):
    return _make(kda.ShortConvBwdArgs, dict(T=128, N=2, D=256, K=4, dtype=BF16, activation=1, norm_dim=128, norm_eps=1e-6), **kw)


def _conv_step(**kw):
    return _make(kda.ShortConvStepArgs, dict(N=4, D=256, K=4, dtype=BF16, activation=1, norm_dim=128, norm_eps=1e-6, num_slots=9), **kw)


def _norm(**kw):
    return _make(kda.BlockNormArgs, dict(T=8, D=256, dtype=BF16, residual_dtype=BF16, gate_kind=1, post_norm=1, pre_norm=1, eps=1e-6,
                                         scale=1.0), **kw)


def _norm_bwd(**kw):
    return _make(kda.BlockNormBwdArgs, dict(T=8, D=256, dtype=BF16, residual_dtype=BF16, gate_kind=1, post_norm=1, pre_norm=1, eps=1e-6,
                                            scale=1.0), **kw)


def _call(lib, a, ws=FAKE << 8, ws_bytes=1 << 50):
    f = getattr(lib, FUNCTION[type(a)])
    return f(ctypes.byref(a), ws, ws_bytes, None) if isinstance(a, WITH_WORKSPACE) else f(ctypes.byref(a), None)


NAN = float("nan")
SCAN = [(dict(D=0), 1), (dict(D=(1 << 20) + 1), 2), (dict(dtype=4), 3), (dict(gate_kind=4), 1), (dict(gate_kind=-1), 1), (dict(input_scale=3), 1),
        (dict(gate_kind=0, g_min=0.0), 1), (dict(gate_kind=0, g_min=NAN), 1), (dict(gate_kind=3), 1), (dict(x=None), 1), (dict(z=None), 1),
        (dict(x=FAKE + 1), 4), (dict(z=FAKE * 90 + 1), 4), (dict(A_log=FAKE * 91 + 2), 4), (dict(x_stride=63), 1), (dict(z_stride=-64), 1),
        (dict(i_stride=(1 << 30) + 1), 1)]
CONV = [(dict(D=0), 1), (dict(D=257), 1), (dict(K=1), 2), (dict(K=5), 2), (dict(norm_dim=48), 2), (dict(norm_dim=512), 2), (dict(activation=2), 1),
        (dict(norm_eps=0.0), 1), (dict(norm_eps=NAN), 1), (dict(weight=None), 1), (dict(x=None), 1), (dict(dtype=2), 3), (dict(x=FAKE * 90 + 1), 4),
        (dict(weight=FAKE * 90 + 2), 4), (dict(x_stride=255), 1), (dict(D=(1 << 20) + 128), 2)]
NORM = [(dict(T=-1), 1), (dict(D=0), 1), (dict(D=8193), 2), (dict(T=1 << 31), 2), (dict(dtype=3), 3), (dict(dtype=F32, residual_dtype=BF16), 3),
        (dict(residual_dtype=7), 3), (dict(gate_kind=3), 1), (dict(gate_kind=0), 1), (dict(gate=None), 1), (dict(post_norm=2), 1), (dict(post_norm=0), 1),
        (dict(pre_norm=0), 1), (dict(eps=0.0), 1), (dict(eps=NAN), 1), (dict(scale=NAN), 1), (dict(residual=None), 1), (dict(y=None), 1),
        (dict(y=FAKE * 90 + 1), 4), (dict(residual=FAKE * 91 + 1), 4), (dict(scale_vec=FAKE * 92 + 2), 4), (dict(post_weight=FAKE * 93 + 1), 4)]


@pytest.mark.parametrize("make", [_scan, _scan_bwd, _scan_step])
@pytest.mark.parametrize("kw,code", SCAN)
def test_scan_rejects(lib, make, kw, code):
    assert _call(lib, make(**kw)) == code


@pytest.mark.parametrize("make", [_conv, _conv_bwd, _conv_step])
@pytest.mark.parametrize("kw,code", CONV)
def test_conv_rejects(lib, make, kw, code):
    assert _call(lib, make(**kw)) == code


@pytest.mark.parametrize("make", [_norm, _norm_bwd])
@pytest.mark.parametrize("kw,code", NORM)
def test_norm_rejects(lib, make, kw, code):
    assert _call(lib, make(**kw)) == code


@pytest.mark.parametrize("make", [_scan, _scan_bwd, _conv, _conv_bwd])
@pytest.mark.parametrize("kw,code", [(dict(T=-1), 1), (dict(N=0), 1), (dict(T=1 << 31), 2), (dict(T=129, cu_seqlens=None), 1), (dict(cu_seqlens=FAKE * 90 + 2), 4),
                                     (dict(T=(1 << 31) - 2, D=1 << 20), 2)])
def test_packed_calls_reject(lib, make, kw, code):
    assert _call(lib, make(**kw)) == code


@pytest.mark.parametrize("make", [_scan_step, _conv_step])
@pytest.mark.parametrize("kw,code", [(dict(N=-1), 1), (dict(num_slots=-1), 1), (dict(state_indices=None, num_slots=3), 1), (dict(state=None), 1),
                                     (dict(num_slots=1 << 31), 2), (dict(state_indices=FAKE * 90 + 2), 4), (dict(state=FAKE * 90 + 1), 4)])
def test_steps_reject(lib, make, kw, code):
    assert _call(lib, make(**kw)) == code


A, B, C = kda.ScanArgs, kda.ScanBwdArgs, kda.ScanStepArgs
V, W, X = kda.ShortConvArgs, kda.ShortConvBwdArgs, kda.ShortConvStepArgs
P, Q = kda.BlockNormArgs, kda.BlockNormBwdArgs


@pytest.mark.parametrize("a", [
    _scan(h=at(A, "x")), _scan(h=at(A, "z") + 64), _scan(h=at(A, "input_gate")), _scan(final_state=at(A, "initial_state") + 16),
    _scan(final_state=at(A, "h")), _scan(checkpoints=at(A, "h") + 256), _scan(checkpoints=at(A, "initial_state")), _scan(h=at(A, "cu_seqlens")),
    _scan(h=at(A, "A_log")), _scan(x_stride=4096, h=at(A, "x") + 128), _scan(h=None),
    _scan_bwd(grad_x=at(B, "x")), _scan_bwd(grad_z=at(B, "grad_h")), _scan_bwd(grad_x=at(B, "grad_z") + 128), _scan_bwd(grad_input_gate=None),
    _scan_bwd(input_gate=None), _scan_bwd(grad_A_log=at(B, "A_log")), _scan_bwd(grad_initial_state=at(B, "grad_final_state")), _scan_bwd(checkpoints=None),
    _scan_bwd(grad_h=None), _scan_bwd(grad_x=at(B, "checkpoints")), _scan_bwd(gate_kind=3, A_log=None, dt_bias=None, grad_A_log=None),
    _scan_step(h=at(C, "x")), _scan_step(state=at(C, "h") + 64), _scan_step(h=None), _scan_step(state=at(C, "z")),
    _conv(y=at(V, "x")), _conv(final_state=at(V, "initial_state") + 32), _conv(y=at(V, "final_state")), _conv(y=at(V, "weight")), _conv(y=None),
    _conv_bwd(grad_x=at(W, "grad_y")), _conv_bwd(grad_x=at(W, "x")), _conv_bwd(grad_weight=at(W, "weight")), _conv_bwd(grad_bias=at(W, "grad_weight") + 64),
    _conv_bwd(grad_initial_state=at(W, "grad_final_state")), _conv_bwd(grad_y=None), _conv_bwd(grad_x=None),
    _conv_step(y=at(X, "x")), _conv_step(y=at(X, "state")), _conv_step(state=at(X, "x") + 32), _conv_step(y=None),
    _norm(residual_out=at(P, "residual") + 64), _norm(normed=at(P, "gate")), _norm(normed=at(P, "residual_out")), _norm(residual_out=at(P, "y")),
    _norm(residual_out=None), _norm(normed=None), _norm(normed=at(P, "y") + 32), _norm(y=None, residual_out=None, gate=None, gate_kind=0),
    _norm(y=None, residual_out=None, gate=None, gate_kind=0, post_norm=0, post_weight=None),
    _norm_bwd(grad_y=at(Q, "gate")), _norm_bwd(grad_residual=at(Q, "residual")), _norm_bwd(grad_gate=at(Q, "gate")), _norm_bwd(grad_y=at(Q, "grad_residual")),
    _norm_bwd(grad_y=None), _norm_bwd(grad_gate=None), _norm_bwd(grad_residual=None), _norm_bwd(grad_scale=at(Q, "scale_vec")),
    _norm_bwd(pre_norm=0, pre_weight=None), _norm_bwd(pre_norm=0, pre_weight=None, grad_normed=None), _norm_bwd(grad_y=at(Q, "y") + 16),
])
def test_overlaps_and_missing_tensors_are_refused(lib, a):
    assert _call(lib, a) == 1


@pytest.mark.parametrize("a", [
    _scan(), _scan(final_state=at(A, "initial_state")), _scan(input_gate=None), _scan(A_log=None, dt_bias=None, gate_kind=3), _scan(gate_kind=0),
    _scan(gate_kind=2, input_scale=2), _scan(cu_seqlens=None), _scan(initial_state=None, final_state=None, checkpoints=None), _scan(T=0, x=None, z=None, h=None),
    _scan(x_stride=192, z_stride=192, i_stride=192, z=at(A, "x") + 128, input_gate=at(A, "x") + 256), _scan(D=65, x=FAKE + 2, dtype=BF16),
    _scan_bwd(), _scan_bwd(input_gate=None, grad_input_gate=None), _scan_bwd(grad_A_log=None, grad_dt_bias=None, grad_initial_state=None, grad_final_state=None),
    _scan_bwd(gate_kind=3, A_log=None, dt_bias=None, grad_A_log=None, grad_dt_bias=None), _scan_step(), _scan_step(state_indices=None), _scan_step(num_slots=0),
    _conv(), _conv(norm_dim=0, D=7), _conv(final_state=at(V, "initial_state")), _conv(bias=None, initial_state=None, final_state=None), _conv(x_stride=768),
    _conv(T=0, x=None, y=None), _conv_bwd(), _conv_bwd(grad_weight=None, grad_bias=None, grad_initial_state=None), _conv_step(), _conv_step(K=2, norm_dim=0),
    _norm(), _norm(residual_out=at(P, "residual"), normed=at(P, "y")), _norm(residual_dtype=F32), _norm(gate_kind=0, gate=None), _norm(gate_kind=2),
    _norm(y=None, residual_out=None, gate=None, gate_kind=0, post_norm=0, post_weight=None, scale_vec=None), _norm(pre_norm=0, pre_weight=None, normed=None),
    _norm(D=8191, dtype=BF16, y=FAKE * 90 + 2), _norm_bwd(), _norm_bwd(grad_residual=at(Q, "grad_residual_out"), grad_y=at(Q, "y")),
    _norm_bwd(grad_y=at(Q, "grad_normed")), _norm_bwd(grad_residual_out=None, grad_normed=None),
])
def test_valid_calls_stop_at_the_device_check(lib, no_gpu, a):
    assert _call(lib, a) == 9


@pytest.mark.parametrize("make", [_scan, _scan_bwd, _conv, _conv_bwd])
def test_tokens_whose_tiles_end_behind_32_bits_are_refused(lib, make):
    for kw in (dict(T=(1 << 31) - 4095, N=1), dict(T=1 << 33, N=1), dict(T=64, N=1 << 31), dict(T=(1 << 31) - 4096, N=1, D=1 << 14)):
        assert _call(lib, make(**kw)) == 2, kw


def test_empty_calls(lib):
    assert _call(lib, _scan_step(N=0)) == 0
    assert _call(lib, _conv_step(N=0)) == 0
    assert _call(lib, _norm(T=0)) == 0


@pytest.mark.parametrize("make", [_scan, _scan_bwd, _conv_bwd, _norm_bwd])
def test_workspaces(lib, make):
    a = make()
    name = FUNCTION[type(a)] + "_workspace_size"
    sizes = [a.T, a.N, a.D] if hasattr(a, "N") else [a.T, a.D]
    if hasattr(a, "K"):
        sizes.append(a.K)
    need = getattr(lib, name)(*sizes, BF16)
    sizes[-2 if hasattr(a, "K") else -1] = 0
    assert getattr(lib, name)(*sizes, BF16) == 0
    if need:
        assert _call(lib, make(), ws_bytes=need - 1) == 5
        assert _call(lib, make(), ws=None) == 5
        assert _call(lib, make(), ws=(FAKE << 8) + 16) == 4


@pytest.mark.parametrize("a", [
    _scan_step(D=1 << 20, N=1, num_slots=(1 << 31) - 1, state=FAKE - 4096),
    _conv_step(D=1 << 20, N=1, num_slots=(1 << 31) - 1, state=FAKE - 4096),
])
def test_pools_that_no_address_reaches_are_refused(lib, a):
    assert _call(lib, a) == 2


def test_binding_refuses_before_the_library():
    x, w, p = torch.zeros((8, 64)), torch.zeros((64, 4)), torch.zeros(64)
    i32 = dict(dtype=torch.int32)
    for call, err in [
        (lambda: kda.scan_fwd(x, x), ValueError),                                      # on the CPU
        (lambda: kda.scan_fwd(x, x[:4]), ValueError),
        (lambda: kda.scan_fwd(x, x.bfloat16()), TypeError),
        (lambda: kda.scan_fwd(x.half(), x.half()), TypeError),
        (lambda: kda.scan_fwd(x, x, gate="odd"), ValueError),
        (lambda: kda.scan_fwd(x, x, input_scale="odd"), ValueError),
        (lambda: kda.scan_fwd(x[0], x[0]), ValueError),
        (lambda: kda.scan_bwd(x, x, None, x[:, :2], x), ValueError),
        (lambda: kda.scan_step(x, x, None, torch.zeros((8, 4, 64))), ValueError),
        (lambda: kda.short_conv_fwd(x, w[:32]), ValueError),
        (lambda: kda.short_conv_fwd(x, w, activation="odd"), ValueError),
        (lambda: kda.short_conv_bwd(x, w, None, x[:2]), ValueError),
        (lambda: kda.short_conv_step(x, w, None, torch.zeros((8, 64))), ValueError),
        (lambda: kda.block_norm_fwd(x, x), ValueError),
        (lambda: kda.block_norm_fwd(None, x, pre_norm=False), ValueError),
        (lambda: kda.block_norm_fwd(None, x, post_weight=p), ValueError),
        (lambda: kda.block_norm_fwd(None, x, scale=p), ValueError),
        (lambda: kda.block_norm_bwd(x, x, None, x, x, pre_norm=False), ValueError),
    ]:
        with pytest.raises(err):
            call()
    meta = lambda *s, **k: torch.empty(s, device="meta", **k)  # noqa: E731
    with pytest.raises(ValueError):
        kda.scan_fwd(meta(8, 64), meta(8, 64), cu_seqlens=meta(1, **i32))


def test_norm_without_a_block_looks_at_the_type_of_what_it_writes(lib, no_gpu, monkeypatch):
    """In front of the first block the type of normed (or of its gradient) says what the call computes in: types that there are, and
    none that the residual stream may not stand beside."""
    x, half = torch.zeros((8, 64)), torch.zeros((8, 64), dtype=torch.float16)
    for call in (lambda: kda.block_norm_fwd(None, x, normed=half), lambda: kda.block_norm_bwd(None, x, None, None, half),
                 lambda: kda.block_norm_fwd(None, half), lambda: kda.block_norm_fwd(None, x, normed=x.to(torch.int32))):
        with pytest.raises(TypeError):
            call()
    monkeypatch.setattr(kda, "_require", lambda *a: None)  # (that the tensors are on the CPU; the library refuses or stops at its device check)
    monkeypatch.setattr(kda, "_run", lambda where, device, fn, packed, *more: kda._check(fn(packed, *more, None), where))
    for call in (lambda r, n: kda.block_norm_fwd(None, r, normed=n), lambda r, n: kda.block_norm_bwd(None, r, None, None, n)):
        with pytest.raises(kda.KDAError) as e:
            call(x.bfloat16(), x)
        assert e.value.code == 3
    for r, n in ((x, x.clone()), (x, x.bfloat16()), (x.bfloat16(), x.bfloat16())):
        with pytest.raises(kda.KDAError) as e:
            kda.block_norm_fwd(None, r, normed=n)
        assert e.value.code == 9
