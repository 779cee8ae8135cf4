"""Host-side checks (no GPU) of the linear-attention, state-copy and rotary calls: struct layouts, refusals."""
import ctypes
import os
import subprocess

import pytest
import torch

from linear_attention_kda_gb300 import build as kbuild, kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 32  # far apart, 16-byte aligned addresses that nothing dereferences
GAP = 1 << 32
STRUCTS = {"kda_linear_args": kda.LinearArgs, "kda_linear_bwd_args": kda.LinearBwdArgs, "kda_linear_step_args": kda.LinearStepArgs,
           "kda_state_copy_args": kda.StateCopyArgs, "kda_rope_args": kda.RopeArgs}


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


def _addresses(names):
    return {n: FAKE + i * GAP for i, n in enumerate(names)}


def _fwd(**kw):
    a = dict(T=128, N=1, H=4, Hq=4, Hk=4, Hv=4, dk=128, dv=128, dtype=kda.KDA_BF16, g_per_token=1, scale=1.0, cu_seqlens=None,
             **_addresses(["q", "k", "v", "g", "o", "initial_state", "final_state"]))
    return kda.LinearArgs(**{**a, **kw})


def _bwd(**kw):
    a = dict(T=128, N=1, H=4, Hq=4, Hk=4, Hv=4, dk=128, dv=128, dtype=kda.KDA_BF16, g_per_token=1, scale=1.0, cu_seqlens=None,
             **_addresses(["q", "k", "v", "g", "grad_o", "initial_state", "grad_final_state", "grad_q", "grad_k", "grad_v", "grad_g",
                           "grad_initial_state"]))
    return kda.LinearBwdArgs(**{**a, **kw})


def _step(**kw):
    a = dict(N=4, H=4, Hq=4, Hk=4, Hv=4, dk=128, dv=128, dtype=kda.KDA_BF16, g_per_token=1, scale=1.0, num_slots=9,
             **_addresses(["q", "k", "v", "g", "o", "state", "state_indices"]))
    return kda.LinearStepArgs(**{**a, **kw})


def _copy(**kw):
    a = dict(slot_bytes=4096, src_slots=8, dst_slots=8, P=3, src_pool=FAKE, dst_pool=FAKE, src=2 * FAKE, dst=3 * FAKE)
    return kda.StateCopyArgs(**{**a, **kw})


_FREQS = (ctypes.c_double * 128)(*([0.5] * 128))


def _rope(**kw):
    a = dict(T=8, Hq=4, Hk=2, d=128, rot=128, dtype=kda.KDA_BF16, layout=0, inverse=0, scale=1.0, freqs=ctypes.addressof(_FREQS),
             q_stride=0, k_stride=0, q_out_stride=0, k_out_stride=0, **_addresses(["positions", "q", "k", "q_out", "k_out"]))
    return kda.RopeArgs(**{**a, **kw})


def _call(lib, a, ws=FAKE << 8, ws_bytes=1 << 50):
    p = ctypes.byref(a)
    if isinstance(a, kda.LinearArgs):
        return lib.kda_linear_chunk_fwd(p, ws, ws_bytes, None)
    if isinstance(a, kda.LinearBwdArgs):
        return lib.kda_linear_chunk_bwd(p, ws, ws_bytes, None)
    return {kda.LinearStepArgs: lib.kda_linear_recurrent_step, kda.StateCopyArgs: lib.kda_state_copy, kda.RopeArgs: lib.kda_rope}[type(a)](p, None)


# refusals that the three linear calls share
COMMON = [(dict(H=0), 1), (dict(Hq=3), 1), (dict(Hk=8), 1), (dict(Hv=0), 1), (dict(Hq=2, Hk=2, Hv=2), 1), (dict(dk=96), 2), (dict(dv=32), 2),
          (dict(dtype=7), 3), (dict(scale=float("nan")), 1), (dict(g_per_token=2), 1), (dict(q=None), 1), (dict(v=None), 1),
          (dict(q=FAKE + 2), 4), (dict(v=FAKE * 3 + 8), 4), (dict(g=FAKE * 4 + 2), 4), (dict(H=70000, Hq=70000, Hk=70000, Hv=70000), 2)]


@pytest.mark.parametrize("make", [_fwd, _bwd, _step])
@pytest.mark.parametrize("kw,code", COMMON)
def test_linear_rejects(lib, make, kw, code):
    assert _call(lib, make(**kw)) == code


@pytest.mark.parametrize("a,code", [
    (_fwd(T=-1), 1), (_fwd(N=0), 1), (_fwd(T=130, N=4), 1), (_fwd(T=1 << 31), 2), (_fwd(o=None), 1), (_fwd(o=FAKE), 1),
    (_fwd(o=FAKE + 1024), 1), (_fwd(final_state=FAKE * 6 + 16), 1), (_fwd(final_state=FAKE * 5), 1), (_fwd(cu_seqlens=FAKE * 5), 1),
    (_fwd(cu_seqlens=FAKE * 9 + 2), 4), (_fwd(initial_state=FAKE * 6 + 8), 4), (_fwd(T=(1 << 31) - 64, H=4096, Hq=4096, Hk=4096, Hv=4096), 2),
    (_bwd(N=0), 1), (_bwd(grad_o=None), 1), (_bwd(grad_k=None), 1), (_bwd(grad_q=FAKE * 9), 1), (_bwd(grad_v=FAKE * 3), 1), (_bwd(g=None), 1),
    (_bwd(grad_g=FAKE * 11 + 2), 4), (_bwd(grad_initial_state=FAKE * 6), 1), (_bwd(T=130, N=4), 1),
    (_step(N=-1), 1), (_step(num_slots=-1), 1), (_step(state_indices=None, num_slots=3), 1), (_step(o=FAKE), 1), (_step(state=FAKE + 2048), 1),
    (_step(state=None), 1), (_step(state=FAKE * 6 + 4), 4), (_step(o=FAKE * 6), 1), (_step(num_slots=1 << 31), 2),
    (_copy(P=-1), 1), (_copy(slot_bytes=24), 2), (_copy(src=None), 1), (_copy(dst_pool=None), 1), (_copy(src_pool=None), 1),
    (_copy(src_slots=4), 1), (_copy(dst_pool=FAKE + 4096), 1), (_copy(dst_pool=FAKE * 5 + 8), 4), (_copy(src=FAKE + 64), 1), (_copy(dst=2 * FAKE + 2), 4),
    (_copy(src_slots=1 << 31), 2),
    (_rope(T=-1), 1), (_rope(Hq=0, Hk=0), 1), (_rope(rot=0), 2), (_rope(rot=63), 2), (_rope(rot=130), 2), (_rope(d=2048), 2), (_rope(d=1), 2),
    (_rope(d=512, rot=258), 2), (_rope(Hq=1025), 2), (_rope(dtype=5), 3), (_rope(layout=2), 1), (_rope(inverse=3), 1), (_rope(scale=float("inf")), 1), (_rope(freqs=None), 1),
    (_rope(positions=None), 1), (_rope(q=None), 1), (_rope(k_out=None), 1), (_rope(q_stride=500), 1), (_rope(q=FAKE * 2 + 1), 4), (_rope(positions=FAKE + 2), 4),
    (_rope(q_out=FAKE * 2 + 256), 1), (_rope(q_out=FAKE * 2, q_out_stride=1024), 1), (_rope(k_out=FAKE * 2), 1), (_rope(k_out=FAKE * 4), 1), (_rope(q_out=FAKE), 1),
])
def test_rejects(lib, a, code):
    assert _call(lib, a) == code


def test_rope_refuses_frequencies_that_are_no_numbers(lib):
    for bad in (float("nan"), float("inf"), -1.0001e6):
        f = (ctypes.c_double * 64)(*([0.5] * 63 + [bad]))
        assert _call(lib, _rope(freqs=ctypes.addressof(f))) == 1


@pytest.mark.parametrize("a", [
    _fwd(), _fwd(g=None), _fwd(final_state=FAKE * 6), _fwd(initial_state=None, final_state=None), _fwd(Hq=2, Hk=1), _fwd(T=0, q=None, k=None, v=None, o=None),
    _bwd(), _bwd(g=None, grad_g=None), _bwd(grad_initial_state=None, initial_state=None, grad_final_state=None), _step(), _step(num_slots=0), _step(g=None),
    _step(state_indices=None), _copy(), _copy(dst_pool=FAKE * 5, dst_slots=3), _rope(), _rope(Hk=0, k=None, k_out=None), _rope(q_out=2 * FAKE, k_out=3 * FAKE),
    # slices of one fused projection of 4 + 2 + 2 heads, in place
    _rope(q=FAKE, k=FAKE + 4 * 256, q_out=FAKE, k_out=FAKE + 4 * 256, q_stride=1024, k_stride=1024, q_out_stride=1024, k_out_stride=1024, positions=9 * FAKE),
])
def test_valid_calls_stop_at_the_device_check(lib, no_gpu, a):
    assert _call(lib, a) == 9


def test_fused_slices_that_meet_are_refused(lib):
    # k's rows begin inside q's
    a = dict(q=FAKE, q_out=FAKE, q_stride=1024, k_stride=1024, q_out_stride=1024, k_out_stride=1024, positions=9 * FAKE)
    assert _call(lib, _rope(k=FAKE + 3 * 256, k_out=FAKE + 3 * 256, **a)) == 1
    # a row's end meets the next row's beginning
    assert _call(lib, _rope(k=FAKE + 7 * 256, k_out=FAKE + 7 * 256, **a)) == 1


def test_empty_calls(lib):
    assert _call(lib, _step(N=0)) == 0
    assert _call(lib, _copy(P=0)) == 0
    assert _call(lib, _copy(slot_bytes=0)) == 0
    assert _call(lib, _rope(T=0)) == 0


def test_workspaces(lib):
    for dt in (torch.float32, torch.bfloat16):
        f = kda.linear_chunk_fwd_workspace_size(1000, 3, 8, 128, 128, dt)
        b = kda.linear_chunk_bwd_workspace_size(1000, 3, 8, 128, 128, dt)
        assert f >= 0 and b > 0
        assert kda.linear_chunk_fwd_workspace_size(1000, 0, 8, 128, 128, dt) == 0
        assert kda.linear_chunk_bwd_workspace_size(1000, 3, 8, 96, 128, dt) == 0
        assert kda.linear_chunk_bwd_workspace_size(1000, 3, 8, 128, 128, dt, Hq=2) >= b
    need = kda.linear_chunk_fwd_workspace_size(128, 1, 4, 128, 128, torch.bfloat16)
    if need:
        assert _call(lib, _fwd(), ws_bytes=need - 1) == 5
    need = kda.linear_chunk_bwd_workspace_size(128, 1, 4, 128, 128, torch.bfloat16)
    assert _call(lib, _bwd(), ws_bytes=need - 1) == 5
    assert _call(lib, _bwd(), ws=None) == 5
    assert _call(lib, _bwd(), ws=(FAKE << 8) + 16) == 4


def test_binding_refuses_before_the_library():
    q, v, g = torch.zeros((8, 4, 64)), torch.zeros((8, 4, 64)), torch.zeros((8, 4))
    for call, err in [
        (lambda: kda.linear_chunk_fwd(q, q, v, g), ValueError),                                  # on the CPU
        (lambda: kda.linear_chunk_fwd(q, q[:4], v, g), ValueError),                              # lengths differ
        (lambda: kda.linear_chunk_fwd(q, q.bfloat16(), v, g), TypeError),
        (lambda: kda.linear_chunk_fwd(q.half(), q.half(), v.half(), g), TypeError),
        (lambda: kda.linear_chunk_fwd(q, q, v, g.double()), TypeError),
        (lambda: kda.linear_chunk_fwd(q, q, v, g[:, :2]), ValueError),
        (lambda: kda.linear_chunk_fwd(q.transpose(0, 1), q, v, g), ValueError),
        (lambda: kda.linear_chunk_fwd(q, q, v, g, initial_state=torch.zeros((2, 4, 64, 64))), ValueError),
        (lambda: kda.linear_chunk_bwd(q, q, v, g, v[:, :2]), ValueError),
        (lambda: kda.linear_recurrent_step(q, q, v, g, torch.zeros((9, 4, 64, 32))), ValueError),
        (lambda: kda.linear_recurrent_step(q, q, v, g, torch.zeros((9, 4, 64))), ValueError),
        (lambda: kda.state_copy(torch.zeros((4, 8)), torch.zeros(2, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)), TypeError),
        (lambda: kda.state_copy(torch.zeros((4, 8)), torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)), ValueError),
        (lambda: kda.rope(None, None, g, g), ValueError),
        (lambda: kda.rope(q, q, torch.zeros(8, dtype=torch.int32), torch.ones(8)), ValueError),  # fp32 frequencies
        (lambda: kda.rope(q, q, torch.zeros(8, dtype=torch.int32), torch.ones(8, dtype=torch.float64), layout="odd"), ValueError),
    ]:
        with pytest.raises(err):
            call()


def test_rope_frequencies():
    f = kda.rope_frequencies(8)
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    assert torch.equal(kda.rope_frequencies(8, scaling="linear", factor=4.0), f / 4)
    n = kda.rope_frequencies(8, scaling="ntk", factor=4.0)
    assert n[0] == 1.0 and abs(float(n[-1] / (f[-1] / 4)) - 1) < 1e-12
    # 1 turns 1024 / 2 pi = 163 times over 1024 positions, 1e-3 a sixth of a time: the ends are kept and divided by 4
    y = kda.rope_frequencies(8, scaling="yarn", factor=4.0, original_length=1024)
    assert y[0] == f[0] and y[-1] == f[-1] / 4 and (y <= f).all() and (y >= f / 4).all()
    assert kda.rope_attention_scale(1.0) == 1.0 and abs(kda.rope_attention_scale(10.0) - 1.2302585092994046) < 1e-15
    for bad in (lambda: kda.rope_frequencies(7), lambda: kda.rope_frequencies(8, scaling="odd"), lambda: kda.rope_frequencies(8, scaling="yarn", factor=2.0)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("a", [
    # a pool of 2^64 bytes begins a slot before the other one and would end where it began
    _copy(slot_bytes=1 << 40, src_slots=1 << 24, dst_slots=1 << 24, dst_pool=FAKE + 4096),
    _copy(slot_bytes=1 << 40, src_slots=1, dst_slots=1 << 23, dst_pool=FAKE - 4096),
    _step(H=65535, Hq=65535, Hk=65535, Hv=65535, N=1, num_slots=(1 << 31) - 1, state=FAKE - 4096, g_per_token=0),
])
def test_pools_that_no_address_reaches_are_refused(lib, a):
    assert _call(lib, a) == 2
