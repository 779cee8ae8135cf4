"""Thin ctypes binding of libkda (include/kda.h).

Argument marshalling only: every step of KDA runs inside libkda's CUDA
kernels.  PyTorch supplies device memory (outputs and the prefill workspace
are allocated here with torch) and the current stream.  If libkda is not
built or cannot be loaded, every call raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkda.so")

KDA_F32, KDA_BF16 = 0, 1
# gate of the log-decay (kda_gate_kind_t): Eq. 5 bounded below by g_min, or the unbounded softplus gate
GATE_KINDS = {"lower_bound": 0, "softplus": 1}
_STATUS = {
    0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_UNSUPPORTED_SHAPE",
    3: "KDA_ERR_UNSUPPORTED_DTYPE", 4: "KDA_ERR_MISALIGNED", 5: "KDA_ERR_WORKSPACE",
    6: "KDA_ERR_CUDA", 7: "KDA_ERR_BAD_SEQLENS", 8: "KDA_ERR_BAD_STATE_INDEX",
    9: "KDA_ERR_NO_DEVICE", 10: "KDA_ERR_DEVICE_TIMEOUT", 11: "KDA_ERR_BAD_TOKEN_COUNT",
    12: "KDA_ERR_NUMERIC",
}
EXPORTED = ["kda_gate", "kda_chunk_fwd", "kda_chunk_fwd_workspace_size", "kda_recurrent_step",
            "kda_status_string", "kda_get_device_error", "kda_abi_version",
            "kda_set_profile_events", "kda_chunk_fwd_kernel_count", "kda_chunk_fwd_static_ws",
            "kda_last_cuda_error", "kda_chunk_fwd_schedule", "kda_output_gate", "kda_recurrent_replay",
            "kda_chunk_fwd_workspace_size_gate", "kda_chunk_bwd", "kda_chunk_bwd_workspace_size",
            "kda_selftest_bounded_wait", "kda_set_debug_checks", "kda_set_chunk_schedule",
            "kda_chunk_bwd_workspace_size_min", "kda_linear_chunk_fwd", "kda_linear_chunk_fwd_workspace_size",
            "kda_linear_chunk_bwd", "kda_linear_chunk_bwd_workspace_size", "kda_linear_recurrent_step",
            "kda_state_copy", "kda_rope"]
STATIC_WORKSPACE_BYTES = 64 << 20

_vp = ctypes.c_void_p
_i64, _i32, _f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class GateArgs(ctypes.Structure):
    _fields_ = [("T", _i64), ("N", _i64), ("H", _i32), ("dk", _i32), ("dtype", ctypes.c_int),
                ("z", _vp), ("dt_bias", _vp), ("A_log", _vp), ("g_min", _f32),
                ("chunk_size", _i32), ("cu_seqlens", _vp), ("out", _vp), ("gate_kind", _i32)]


class ChunkArgs(ctypes.Structure):
    _fields_ = [("T", _i64), ("N", _i64), ("H", _i32), ("dk", _i32), ("dv", _i32),
                ("dtype", ctypes.c_int), ("q", _vp), ("k", _vp), ("z", _vp), ("v", _vp),
                ("beta", _vp), ("dt_bias", _vp), ("A_log", _vp), ("g_min", _f32), ("scale", _f32),
                ("cu_seqlens", _vp), ("cu_seqlens_host", _vp), ("initial_state", _vp),
                ("final_state", _vp), ("o", _vp), ("chunk_size", _i32),
                ("out_gate", _vp), ("out_norm_weight", _vp), ("out_norm_eps", _f32), ("gate_kind", _i32)]


class ReplayArgs(ctypes.Structure):
    _fields_ = [("N", _i64), ("H", _i32), ("dk", _i32), ("dv", _i32), ("dtype", ctypes.c_int), ("R", _i32),
                ("rq", _vp), ("rk", _vp), ("rz", _vp), ("rv", _vp), ("rbeta", _vp), ("n_replay", _vp),
                ("M", _i32), ("q", _vp), ("k", _vp), ("z", _vp), ("v", _vp), ("beta", _vp), ("n_commit", _vp),
                ("dt_bias", _vp), ("A_log", _vp), ("g_min", _f32), ("scale", _f32), ("state", _vp),
                ("state_indices", _vp), ("num_slots", _i64), ("o", _vp), ("gate_kind", _i32)]


class ChunkBwdArgs(ctypes.Structure):
    _fields_ = [("T", _i64), ("N", _i64), ("H", _i32), ("dk", _i32), ("dv", _i32), ("dtype", ctypes.c_int),
                ("q", _vp), ("k", _vp), ("z", _vp), ("v", _vp), ("beta", _vp), ("dt_bias", _vp), ("A_log", _vp),
                ("g_min", _f32), ("scale", _f32), ("cu_seqlens", _vp), ("initial_state", _vp), ("grad_o", _vp),
                ("grad_final_state", _vp), ("grad_q", _vp), ("grad_k", _vp), ("grad_z", _vp), ("grad_v", _vp),
                ("grad_beta", _vp), ("grad_dt_bias", _vp), ("grad_A_log", _vp), ("grad_initial_state", _vp),
                ("chunk_size", _i32), ("gate_kind", _i32)]


class OutputGateArgs(ctypes.Structure):
    _fields_ = [("T", _i64), ("H", _i32), ("dv", _i32), ("dtype", ctypes.c_int), ("o", _vp), ("g", _vp),
                ("norm_weight", _vp), ("eps", _f32), ("y", _vp)]


class StepArgs(ctypes.Structure):
    _fields_ = [("N", _i64), ("H", _i32), ("dk", _i32), ("dv", _i32), ("dtype", ctypes.c_int),
                ("q", _vp), ("k", _vp), ("z", _vp), ("v", _vp), ("beta", _vp),
                ("dt_bias", _vp), ("A_log", _vp), ("g_min", _f32), ("scale", _f32),
                ("state", _vp), ("state_indices", _vp), ("num_slots", _i64), ("o", _vp), ("gate_kind", _i32)]


class LinearArgs(ctypes.Structure):
    _fields_ = [("T", _i64), ("N", _i64), ("H", _i32), ("Hq", _i32), ("Hk", _i32), ("Hv", _i32), ("dk", _i32),
                ("dv", _i32), ("dtype", ctypes.c_int), ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp),
                ("g_per_token", _i32), ("scale", _f32), ("cu_seqlens", _vp), ("initial_state", _vp),
                ("final_state", _vp), ("o", _vp)]


class LinearBwdArgs(ctypes.Structure):
    _fields_ = [("T", _i64), ("N", _i64), ("H", _i32), ("Hq", _i32), ("Hk", _i32), ("Hv", _i32), ("dk", _i32),
                ("dv", _i32), ("dtype", ctypes.c_int), ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp),
                ("g_per_token", _i32), ("scale", _f32), ("cu_seqlens", _vp), ("initial_state", _vp), ("grad_o", _vp),
                ("grad_final_state", _vp), ("grad_q", _vp), ("grad_k", _vp), ("grad_v", _vp), ("grad_g", _vp),
                ("grad_initial_state", _vp)]


class LinearStepArgs(ctypes.Structure):
    _fields_ = [("N", _i64), ("H", _i32), ("Hq", _i32), ("Hk", _i32), ("Hv", _i32), ("dk", _i32), ("dv", _i32),
                ("dtype", ctypes.c_int), ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp), ("g_per_token", _i32),
                ("scale", _f32), ("state", _vp), ("state_indices", _vp), ("num_slots", _i64), ("o", _vp)]


class StateCopyArgs(ctypes.Structure):
    _fields_ = [("src_pool", _vp), ("dst_pool", _vp), ("slot_bytes", _i64), ("src_slots", _i64), ("dst_slots", _i64),
                ("P", _i64), ("src", _vp), ("dst", _vp)]


class RopeArgs(ctypes.Structure):
    _fields_ = [("T", _i64), ("Hq", _i32), ("Hk", _i32), ("d", _i32), ("rot", _i32), ("dtype", ctypes.c_int),
                ("layout", _i32), ("inverse", _i32), ("scale", _f32), ("positions", _vp), ("freqs", _vp), ("q", _vp),
                ("k", _vp), ("q_out", _vp), ("k_out", _vp), ("q_stride", _i64), ("k_stride", _i64),
                ("q_out_stride", _i64), ("k_out_stride", _i64)]


class KDAError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = int(code)
        super().__init__(f"{where}: {_STATUS.get(int(code), code)}")


_lock = threading.Lock()
_lib = None


def load_library(path: Optional[str] = None):
    """Loads libkda.so (raises if missing: build it with linear_attention_kda_gb300.build)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"libkda is not built ({p} missing); run "
                               "`python -m linear_attention_kda_gb300.build`")
        L = ctypes.CDLL(p)
        L.kda_gate.argtypes = [ctypes.POINTER(GateArgs), _vp]
        L.kda_gate.restype = ctypes.c_int
        L.kda_chunk_fwd.argtypes = [ctypes.POINTER(ChunkArgs), _vp, ctypes.c_size_t, _vp]
        L.kda_chunk_fwd.restype = ctypes.c_int
        L.kda_chunk_fwd_workspace_size.argtypes = [_i64, _i64, _i32, _i32, _i32, ctypes.c_int, _i32, _vp]
        L.kda_chunk_fwd_workspace_size.restype = ctypes.c_size_t
        L.kda_chunk_fwd_workspace_size_gate.argtypes = [_i64, _i64, _i32, _i32, _i32, ctypes.c_int, _i32, _vp, _i32]
        L.kda_chunk_fwd_workspace_size_gate.restype = ctypes.c_size_t
        L.kda_chunk_bwd_workspace_size.argtypes = [_i64, _i64, _i32, _i32, _i32, _i32]
        L.kda_chunk_bwd_workspace_size.restype = ctypes.c_size_t
        L.kda_chunk_bwd_workspace_size_min.argtypes = [_i64, _i64, _i32, _i32, _i32, _i32]
        L.kda_chunk_bwd_workspace_size_min.restype = ctypes.c_size_t
        L.kda_chunk_bwd.argtypes = [ctypes.POINTER(ChunkBwdArgs), _vp, ctypes.c_size_t, _vp]
        L.kda_chunk_bwd.restype = ctypes.c_int
        L.kda_selftest_bounded_wait.argtypes = [_vp, _vp]
        L.kda_selftest_bounded_wait.restype = ctypes.c_int
        L.kda_recurrent_step.argtypes = [ctypes.POINTER(StepArgs), _vp]
        L.kda_recurrent_step.restype = ctypes.c_int
        L.kda_status_string.argtypes = [ctypes.c_int]
        L.kda_status_string.restype = ctypes.c_char_p
        L.kda_get_device_error.argtypes = [_vp]
        L.kda_get_device_error.restype = ctypes.c_int
        L.kda_abi_version.restype = ctypes.c_int
        L.kda_set_profile_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), _i32]
        L.kda_set_profile_events.restype = ctypes.c_int
        L.kda_chunk_fwd_kernel_count.argtypes = [ctypes.POINTER(ChunkArgs)]
        L.kda_chunk_fwd_kernel_count.restype = _i32
        L.kda_chunk_fwd_schedule.argtypes = [ctypes.POINTER(ChunkArgs), ctypes.POINTER(_i64)]
        L.kda_chunk_fwd_schedule.restype = ctypes.c_int
        L.kda_chunk_fwd_static_ws.argtypes = [ctypes.POINTER(ChunkArgs), _vp]
        L.kda_chunk_fwd_static_ws.restype = ctypes.c_int
        L.kda_set_debug_checks.argtypes = [_i32]
        L.kda_set_debug_checks.restype = ctypes.c_int
        L.kda_set_chunk_schedule.argtypes = [_i32]
        L.kda_set_chunk_schedule.restype = ctypes.c_int
        L.kda_recurrent_replay.argtypes = [ctypes.POINTER(ReplayArgs), _vp]
        L.kda_recurrent_replay.restype = ctypes.c_int
        L.kda_output_gate.argtypes = [ctypes.POINTER(OutputGateArgs), _vp]
        L.kda_output_gate.restype = ctypes.c_int
        # (arguments as packed bytes or by reference to their ctypes structures)
        for name in ("kda_linear_chunk_fwd", "kda_linear_chunk_bwd"):
            getattr(L, name).argtypes = [_vp, _vp, ctypes.c_size_t, _vp]
            getattr(L, name).restype = ctypes.c_int
        for name in ("kda_linear_recurrent_step", "kda_state_copy", "kda_rope"):
            getattr(L, name).argtypes = [_vp, _vp]
            getattr(L, name).restype = ctypes.c_int
        L.kda_linear_chunk_fwd_workspace_size.argtypes = [_i64, _i64, _i32, _i32, _i32, ctypes.c_int]
        L.kda_linear_chunk_fwd_workspace_size.restype = ctypes.c_size_t
        L.kda_linear_chunk_bwd_workspace_size.argtypes = [_i64, _i64] + [_i32] * 6 + [ctypes.c_int]
        L.kda_linear_chunk_bwd_workspace_size.restype = ctypes.c_size_t
        L.kda_last_cuda_error.argtypes = []
        L.kda_last_cuda_error.restype = _i32
        _lib = L
        return L


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _gate_kind(gate: str) -> int:
    if gate not in GATE_KINDS:
        raise ValueError(f"gate must be one of {sorted(GATE_KINDS)}")
    return GATE_KINDS[gate]


def _stream(t: torch.Tensor):
    return torch.cuda.current_stream(t.device).cuda_stream


def _check(code: int, where: str):
    if code != 0:
        if code == 6 and _lib is not None:  # KDA_ERR_CUDA
            where = f"{where} (cudaError_t {int(_lib.kda_last_cuda_error())})"
        raise KDAError(code, where)


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def gate(z: torch.Tensor, dt_bias=None, A_log=None, g_min: float = -5.0, chunk_size: int = 0,
         cu_seqlens: Optional[torch.Tensor] = None, n_seq: int = 1, out=None,
         gate: str = "lower_bound") -> torch.Tensor:
    """kda_gate: g = g_min * sigmoid(exp(A_log) (z + dt_bias)) (Eq. 5), or with gate="softplus"
    g = -exp(A_log) * softplus(z + dt_bias); or its chunk-local cumsum."""
    L = load_library()
    T, H, dk = z.shape
    _contig(z, dt_bias, A_log, cu_seqlens)
    if out is None:
        out = torch.empty((T, H, dk), dtype=torch.float32, device=z.device)
    a = GateArgs(T=T, N=(cu_seqlens.numel() - 1) if cu_seqlens is not None else n_seq, H=H, dk=dk,
                 dtype=_dtype_code(z), z=_ptr(z), dt_bias=_ptr(dt_bias), A_log=_ptr(A_log),
                 g_min=g_min, chunk_size=chunk_size, cu_seqlens=_ptr(cu_seqlens), out=_ptr(out),
                 gate_kind=_gate_kind(gate))
    _check(L.kda_gate(ctypes.byref(a), _stream(z)), "kda_gate")
    return out


# below this g_min the bounded gate's bf16 d = 128 prefill runs on the fp32 path (kda.h)
TC_MIN_G_MIN = -5.5


def chunk_fwd_workspace_size(T, N, H, dk, dv, dtype: torch.dtype, chunk_size=64, cu_seqlens_host=None,
                             gate: str = "lower_bound", g_min: float = -5.0):
    """kda_chunk_fwd_workspace_size_gate for the path the call takes (the fp32 path's size, that of the
    softplus gate, for a bounded gate with g_min below TC_MIN_G_MIN)."""
    L = load_library()
    if gate == "lower_bound" and not g_min >= TC_MIN_G_MIN:
        gate = "softplus"
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    hp = None
    if cu_seqlens_host is not None:
        hp = cu_seqlens_host.data_ptr()
    return int(L.kda_chunk_fwd_workspace_size_gate(T, N, H, dk, dv, code, chunk_size, hp, _gate_kind(gate)))


def chunk_fwd(q, k, v, z, beta, dt_bias=None, A_log=None, *, g_min: float = -5.0, scale: float = 1.0,
              cu_seqlens: Optional[torch.Tensor] = None, cu_seqlens_host: Optional[torch.Tensor] = None,
              n_seq: int = 1, initial_state: Optional[torch.Tensor] = None,
              output_final_state: bool = False, final_state: Optional[torch.Tensor] = None,
              chunk_size: int = 64, workspace: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, out_gate: Optional[torch.Tensor] = None,
              out_norm_weight: Optional[torch.Tensor] = None, out_norm_eps: float = 1e-6,
              gate: str = "lower_bound"):
    """kda_chunk_fwd: chunkwise KDA prefill (Eq. 1 evaluated as Eq. 3-4).  Returns (o, final_state).
    gate="softplus" selects the unbounded gate (run on the fp32 CUDA-core path).

    With out_gate ([T, H, dv], the gate pre-activation W_g x), o holds the output epilogue of Eq. 6,
    Sigmoid(out_gate) * RMSNorm(o~) (per-head RMSNorm with weight out_norm_weight [H, dv], eps)."""
    L = load_library()
    T, H, dk = q.shape
    dv = v.shape[2]
    _contig(q, k, v, z, beta, dt_bias, A_log, cu_seqlens, initial_state, out_gate, out_norm_weight)
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else n_seq
    if cu_seqlens_host is not None:
        cu_seqlens_host = cu_seqlens_host.to(dtype=torch.int32, device="cpu").contiguous()
    o = out if out is not None else torch.empty((T, H, dv), dtype=q.dtype, device=q.device)
    fs = final_state
    if fs is None and output_final_state:
        fs = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    need = chunk_fwd_workspace_size(T, N, H, dk, dv, q.dtype, chunk_size, cu_seqlens_host, gate, g_min)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=q.device)
    a = ChunkArgs(T=T, N=N, H=H, dk=dk, dv=dv, dtype=_dtype_code(q), q=_ptr(q), k=_ptr(k), z=_ptr(z),
                  v=_ptr(v), beta=_ptr(beta), dt_bias=_ptr(dt_bias), A_log=_ptr(A_log), g_min=g_min,
                  scale=scale, cu_seqlens=_ptr(cu_seqlens),
                  cu_seqlens_host=None if cu_seqlens_host is None else cu_seqlens_host.data_ptr(),
                  initial_state=_ptr(initial_state), final_state=_ptr(fs), o=_ptr(o),
                  chunk_size=chunk_size, out_gate=_ptr(out_gate), out_norm_weight=_ptr(out_norm_weight),
                  out_norm_eps=out_norm_eps, gate_kind=_gate_kind(gate))
    _check(L.kda_chunk_fwd(ctypes.byref(a), _ptr(workspace), workspace.numel(), _stream(q)),
           "kda_chunk_fwd")
    return o, fs


def chunk_bwd(q, k, v, z, beta, dt_bias, A_log, grad_o, *, g_min: float = -5.0, scale: float = 1.0,
              cu_seqlens: Optional[torch.Tensor] = None, n_seq: int = 1,
              initial_state: Optional[torch.Tensor] = None, grad_final_state: Optional[torch.Tensor] = None,
              gate: str = "lower_bound", param_grads: bool = True, state_grad: bool = True,
              workspace: Optional[torch.Tensor] = None) -> dict:
    """kda_chunk_bwd: gradients of the chunked prefill given grad_o (and grad_final_state).

    Returns a dict with q, k, v, z, beta (dtype of q) and, when asked, dt_bias, A_log (fp32) and
    initial_state (fp32 [N, H, dk, dv])."""
    L = load_library()
    T, H, dk = q.shape
    dv = v.shape[2]
    _contig(q, k, v, z, beta, dt_bias, A_log, grad_o, cu_seqlens, initial_state, grad_final_state)
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else n_seq
    g = {n: torch.empty_like(x) for n, x in (("q", q), ("k", k), ("v", v), ("z", z), ("beta", beta))}
    if param_grads:
        g["dt_bias"] = torch.zeros((H, dk), dtype=torch.float32, device=q.device)
        g["A_log"] = torch.zeros((H,), dtype=torch.float32, device=q.device)
    if state_grad:
        g["initial_state"] = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    if workspace is None:  # a given workspace is used as it is (a smaller one segments a long sequence)
        need = int(L.kda_chunk_bwd_workspace_size(T, N, H, dk, dv, 64))
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=q.device)
    a = ChunkBwdArgs(T=T, N=N, H=H, dk=dk, dv=dv, dtype=_dtype_code(q), q=_ptr(q), k=_ptr(k), z=_ptr(z), v=_ptr(v),
                     beta=_ptr(beta), dt_bias=_ptr(dt_bias), A_log=_ptr(A_log), g_min=g_min, scale=scale,
                     cu_seqlens=_ptr(cu_seqlens), initial_state=_ptr(initial_state), grad_o=_ptr(grad_o),
                     grad_final_state=_ptr(grad_final_state), grad_q=_ptr(g["q"]), grad_k=_ptr(g["k"]),
                     grad_z=_ptr(g["z"]), grad_v=_ptr(g["v"]), grad_beta=_ptr(g["beta"]),
                     grad_dt_bias=_ptr(g.get("dt_bias")), grad_A_log=_ptr(g.get("A_log")),
                     grad_initial_state=_ptr(g.get("initial_state")), chunk_size=64, gate_kind=_gate_kind(gate))
    _check(L.kda_chunk_bwd(ctypes.byref(a), _ptr(workspace), workspace.numel(), _stream(q)), "kda_chunk_bwd")
    return g


def chunk_bwd_workspace_size(T, N, H, dk=128, dv=128, minimum: bool = False) -> int:
    """kda_chunk_bwd_workspace_size (one pass), or with minimum=True kda_chunk_bwd_workspace_size_min
    (the smallest workspace kda_chunk_bwd accepts: segments of one long sequence)."""
    L = load_library()
    f = L.kda_chunk_bwd_workspace_size_min if minimum else L.kda_chunk_bwd_workspace_size
    return int(f(T, N, H, dk, dv, 64))


def output_gate(o, g, norm_weight=None, eps: float = 1e-6, *, out: Optional[torch.Tensor] = None):
    """kda_output_gate: Sigmoid(g) * RMSNorm(o) per (token, head) (Eq. 6 without projections).
    o, g: [T, H, dv]; norm_weight: [H, dv] fp32 or None; out may be o (in place)."""
    L = load_library()
    T, H, dv = o.shape
    _contig(o, g, norm_weight)
    y = out if out is not None else torch.empty_like(o)
    a = OutputGateArgs(T=T, H=H, dv=dv, dtype=_dtype_code(o), o=_ptr(o), g=_ptr(g),
                       norm_weight=_ptr(norm_weight), eps=eps, y=_ptr(y))
    _check(L.kda_output_gate(ctypes.byref(a), _stream(o)), "kda_output_gate")
    return y


def recurrent_step(q, k, v, z, beta, dt_bias, A_log, state, *, g_min: float = -5.0, scale: float = 1.0,
                   state_indices: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   gate: str = "lower_bound"):
    """kda_recurrent_step: one decode token per sequence; `state` is updated in place.  Returns o."""
    L = load_library()
    N, H, dk = q.shape
    dv = v.shape[2]
    _contig(q, k, v, z, beta, dt_bias, A_log, state, state_indices)
    o = out if out is not None else torch.empty((N, H, dv), dtype=q.dtype, device=q.device)
    a = StepArgs(N=N, H=H, dk=dk, dv=dv, dtype=_dtype_code(q), q=_ptr(q), k=_ptr(k), z=_ptr(z),
                 v=_ptr(v), beta=_ptr(beta), dt_bias=_ptr(dt_bias), A_log=_ptr(A_log), g_min=g_min,
                 scale=scale, state=_ptr(state), state_indices=_ptr(state_indices),
                 num_slots=state.shape[0], o=_ptr(o), gate_kind=_gate_kind(gate))
    _check(L.kda_recurrent_step(ctypes.byref(a), _stream(q)), "kda_recurrent_step")
    return o


def recurrent_replay(cached, n_replay, new, n_commit, dt_bias, A_log, state, *, g_min: float = -5.0,
                     scale: float = 1.0, state_indices: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, gate: str = "lower_bound"):
    """kda_recurrent_replay: speculative decoding with replay (section 5.4).

    cached: (q, k, z, v, beta) of the cached draft window, [N, R, H, d] / [N, R, H] (or None: R = 0);
    new: (q, k, z, v, beta) of the new tokens, [N, M, H, d] / [N, M, H]; n_replay, n_commit: int32 [N]
    on the device.  Replays the accepted cached tokens, runs the new ones (outputs returned,
    [N, M, H, dv]) and writes back the state after the first n_commit new tokens, in place."""
    L = load_library()
    q, k, z, v, beta = new
    N, M, H, dk = q.shape
    dv = v.shape[3]
    if cached is None:
        rq = rk = rz = rv = rb = None
        R = 0
    else:
        rq, rk, rz, rv, rb = cached
        R = rq.shape[1]
    _contig(q, k, z, v, beta, rq, rk, rz, rv, rb, n_replay, n_commit, dt_bias, A_log, state, state_indices)
    o = out if out is not None else torch.empty((N, M, H, dv), dtype=q.dtype, device=q.device)
    a = ReplayArgs(N=N, H=H, dk=dk, dv=dv, dtype=_dtype_code(q), R=R, rq=_ptr(rq), rk=_ptr(rk), rz=_ptr(rz),
                   rv=_ptr(rv), rbeta=_ptr(rb), n_replay=_ptr(n_replay), M=M, q=_ptr(q), k=_ptr(k), z=_ptr(z),
                   v=_ptr(v), beta=_ptr(beta), n_commit=_ptr(n_commit), dt_bias=_ptr(dt_bias),
                   A_log=_ptr(A_log), g_min=g_min, scale=scale, state=_ptr(state),
                   state_indices=_ptr(state_indices), num_slots=state.shape[0], o=_ptr(o),
                   gate_kind=_gate_kind(gate))
    _check(L.kda_recurrent_replay(ctypes.byref(a), _stream(q)), "kda_recurrent_replay")
    return o


# ---------------------------------------------------------------- linear attention with a decay per head
# A decode step's kernel takes 4 us, so what a call does on the host counts: quick checks (a second,
# descriptive look only where something is wrong), arguments packed by struct (a third of a ctypes.Structure's
# time, same layout), the current device and stream asked for once.
_LINEAR = struct.Struct("@qq7iPPPPifPPPP")
_LINEAR_BWD = struct.Struct("@qq7iPPPPif" + "P" * 9)
_LINEAR_STEP = struct.Struct("@q7iPPPPifPPqP")
_STATE_COPY = struct.Struct("@PPqqqqPP")
_ROPE = struct.Struct("@qiiiiiiifPPPPPPqqqq")
assert [x.size for x in (_LINEAR, _LINEAR_BWD, _LINEAR_STEP, _STATE_COPY, _ROPE)] == [
    ctypes.sizeof(x) for x in (LinearArgs, LinearBwdArgs, LinearStepArgs, StateCopyArgs, RopeArgs)]


def _require(where: str, device: int, spec):
    """Says what is wrong with a call's (name, tensor, shape, dtype): shape, dtype, dense layout, one CUDA device (None
    passes)."""
    for name, t, shape, dtype in spec:
        if t is None:
            continue
        if t.shape != shape:
            raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        if t.dtype is not dtype:
            raise TypeError(f"{where}: {name} is {t.dtype}, not {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be contiguous")
        if t.get_device() != device:
            raise ValueError(f"{where}: {name} is not on the device of the others")
    if device < 0:
        raise ValueError(f"{where}: tensors must be on a CUDA device")


def _off(t, shape, dtype, device) -> bool:
    return t.shape != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous()


def _run(where: str, device: int, fn, packed: bytes, *more):
    """Calls fn(args, *more, stream) with `device` current, on its current stream."""
    if torch.cuda.current_device() != device:
        with torch.cuda.device(device):
            code = fn(packed, *more, _raw_stream(device))
    else:
        code = fn(packed, *more, _raw_stream(device))
    if code:
        _check(code, where)


def _raw_stream(device: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device)  # torch.cuda.current_stream without its Python object


def _p(t):
    return 0 if t is None else t.data_ptr()


def _linear_heads(where, q, k, v, g):
    """(rows, H, Hq, Hk, Hv, dk, dv, g per token, dtype code) of a linear-attention call."""
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError(f"{where}: q, k and v have three dimensions (rows, heads, channels)")
    T, Hq, dk = q.shape
    Hk = k.shape[1]
    _, Hv, dv = v.shape
    if g is not None and g.dim() not in (1, 2):
        raise ValueError(f"{where}: g has shape [rows, heads] or [heads]")
    return T, max(Hq, Hk, Hv), Hq, Hk, Hv, dk, dv, int(g is not None and g.dim() == 2), _dtype_code(q)


def _n_sequences(where, cu_seqlens, n_seq):
    if cu_seqlens is None:
        return n_seq
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError(f"{where}: cu_seqlens has shape [sequences + 1]")
    return cu_seqlens.numel() - 1


def _workspace(where, workspace, need, device):
    """(address, bytes, tensor that holds it)"""
    if workspace is None:
        if need == 0:
            return 0, 0, None
        workspace = torch.empty((need,), dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"{where}: the workspace must be contiguous and on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def linear_chunk_fwd_workspace_size(T, N, H, dk, dv, dtype: torch.dtype) -> int:
    """kda_linear_chunk_fwd_workspace_size (bytes; 0 on invalid sizes, and where none is needed)."""
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(load_library().kda_linear_chunk_fwd_workspace_size(T, N, H, dk, dv, code))


def linear_chunk_bwd_workspace_size(T, N, H, dk, dv, dtype: torch.dtype, Hq=None, Hk=None, Hv=None) -> int:
    """kda_linear_chunk_bwd_workspace_size (bytes; 0 on invalid sizes)."""
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(load_library().kda_linear_chunk_bwd_workspace_size(T, N, H, Hq or H, Hk or H, Hv or H, dk, dv, code))


def linear_chunk_fwd(q, k, v, g=None, *, scale: float = 1.0, cu_seqlens: Optional[torch.Tensor] = None,
                     n_seq: int = 1, initial_state: Optional[torch.Tensor] = None, output_final_state: bool = False,
                     final_state: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None):
    """kda_linear_chunk_fwd: linear attention with a decay per head over whole sequences,
    S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.  Returns (o, final_state).

    q [T, Hq, dk], k [T, Hk, dk], v [T, Hv, dv] (fp32 or bf16; H = the largest head count, a multiple of the
    others); g: log-decay, at most 0, fp32 [T, H] or [H], or None (no decay); states fp32 [N, H, dk, dv]."""
    where, L, f32 = "linear_chunk_fwd", _lib or load_library(), torch.float32
    T, H, Hq, Hk, Hv, dk, dv, per_token, code = _linear_heads(where, q, k, v, g)
    N, dt, dev = _n_sequences(where, cu_seqlens, n_seq), q.dtype, q.get_device()
    state, gshape = (N, H, dk, dv), (T, H) if per_token else (H,)
    if (dev < 0 or not q.is_contiguous() or _off(k, (T, Hk, dk), dt, dev) or _off(v, (T, Hv, dv), dt, dev)
            or (g is not None and _off(g, gshape, f32, dev)) or (cu_seqlens is not None and _off(cu_seqlens, (N + 1,), torch.int32, dev))
            or (initial_state is not None and _off(initial_state, state, f32, dev))
            or (final_state is not None and _off(final_state, state, f32, dev)) or (out is not None and _off(out, (T, H, dv), dt, dev))):
        _require(where, dev, (("q", q, (T, Hq, dk), dt), ("k", k, (T, Hk, dk), dt), ("v", v, (T, Hv, dv), dt),
                              ("g", g, gshape, f32), ("cu_seqlens", cu_seqlens, (N + 1,), torch.int32),
                              ("initial_state", initial_state, state, f32), ("final_state", final_state, state, f32),
                              ("out", out, (T, H, dv), dt)))
    if out is None:
        out = torch.empty_like(v) if Hv == H else torch.empty((T, H, dv), dtype=dt, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty(state, dtype=f32, device=q.device)
    ws, ws_bytes, _keep = _workspace(where, workspace, L.kda_linear_chunk_fwd_workspace_size(T, N, H, dk, dv, code), q.device)
    _run("kda_linear_chunk_fwd", dev, L.kda_linear_chunk_fwd,
         _LINEAR.pack(T, N, H, Hq, Hk, Hv, dk, dv, code, _p(q), _p(k), _p(v), _p(g), per_token, scale, _p(cu_seqlens),
                      _p(initial_state), _p(final_state), _p(out)), ws, ws_bytes)
    return out, final_state


def linear_chunk_bwd(q, k, v, g, grad_o, *, scale: float = 1.0, cu_seqlens: Optional[torch.Tensor] = None,
                     n_seq: int = 1, initial_state: Optional[torch.Tensor] = None,
                     grad_final_state: Optional[torch.Tensor] = None, decay_grad: bool = True,
                     state_grad: bool = True, workspace: Optional[torch.Tensor] = None) -> dict:
    """kda_linear_chunk_bwd: gradients of linear_chunk_fwd given grad_o (and grad_final_state).

    Returns a dict with q, k, v (shapes and dtype of the inputs) and, when asked, g (fp32, the shape of g; not
    without g) and initial_state (fp32 [N, H, dk, dv])."""
    where, L, f32 = "linear_chunk_bwd", _lib or load_library(), torch.float32
    T, H, Hq, Hk, Hv, dk, dv, per_token, code = _linear_heads(where, q, k, v, g)
    N, dt, dev = _n_sequences(where, cu_seqlens, n_seq), q.dtype, q.get_device()
    state, gshape = (N, H, dk, dv), (T, H) if per_token else (H,)
    if (dev < 0 or not q.is_contiguous() or _off(k, (T, Hk, dk), dt, dev) or _off(v, (T, Hv, dv), dt, dev)
            or _off(grad_o, (T, H, dv), dt, dev) or (g is not None and _off(g, gshape, f32, dev))
            or (cu_seqlens is not None and _off(cu_seqlens, (N + 1,), torch.int32, dev))
            or (initial_state is not None and _off(initial_state, state, f32, dev))
            or (grad_final_state is not None and _off(grad_final_state, state, f32, dev))):
        _require(where, dev, (("q", q, (T, Hq, dk), dt), ("k", k, (T, Hk, dk), dt), ("v", v, (T, Hv, dv), dt),
                              ("g", g, gshape, f32), ("grad_o", grad_o, (T, H, dv), dt),
                              ("cu_seqlens", cu_seqlens, (N + 1,), torch.int32), ("initial_state", initial_state, state, f32),
                              ("grad_final_state", grad_final_state, state, f32)))
    grads = {"q": torch.empty_like(q), "k": torch.empty_like(k), "v": torch.empty_like(v)}
    if decay_grad and g is not None:
        grads["g"] = torch.empty_like(g)
    if state_grad:
        grads["initial_state"] = torch.empty(state, dtype=f32, device=q.device)
    need = L.kda_linear_chunk_bwd_workspace_size(T, N, H, Hq, Hk, Hv, dk, dv, code)
    ws, ws_bytes, _keep = _workspace(where, workspace, need, q.device)
    _run("kda_linear_chunk_bwd", dev, L.kda_linear_chunk_bwd,
         _LINEAR_BWD.pack(T, N, H, Hq, Hk, Hv, dk, dv, code, _p(q), _p(k), _p(v), _p(g), per_token, scale, _p(cu_seqlens),
                          _p(initial_state), _p(grad_o), _p(grad_final_state), _p(grads["q"]), _p(grads["k"]), _p(grads["v"]),
                          _p(grads.get("g")), _p(grads.get("initial_state"))), ws, ws_bytes)
    return grads


def linear_recurrent_step(q, k, v, g, state, *, scale: float = 1.0, state_indices: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None):
    """kda_linear_recurrent_step: one decode token per sequence of linear attention with a decay per head; `state`
    [slots, H, dk, dv] is updated in place.  Shapes as linear_chunk_fwd with N rows; state_indices int32 [N] (-1: an
    unused row of a padded batch, left alone with its row of the output).  Returns o [N, H, dv]."""
    where, L = "linear_recurrent_step", _lib or load_library()
    N, H, Hq, Hk, Hv, dk, dv, per_token, code = _linear_heads(where, q, k, v, g)
    if state.dim() != 4:
        raise ValueError(f"{where}: state has shape [slots, heads, dk, dv]")
    slots, dt, dev = state.shape[0], q.dtype, q.get_device()
    f32, gshape = torch.float32, (N, H) if per_token else (H,)
    if (dev < 0 or not q.is_contiguous() or _off(k, (N, Hk, dk), dt, dev) or _off(v, (N, Hv, dv), dt, dev)
            or _off(state, (slots, H, dk, dv), f32, dev) or (g is not None and _off(g, gshape, f32, dev))
            or (state_indices is not None and _off(state_indices, (N,), torch.int32, dev))
            or (out is not None and _off(out, (N, H, dv), dt, dev))):
        _require(where, dev, (("q", q, (N, Hq, dk), dt), ("k", k, (N, Hk, dk), dt), ("v", v, (N, Hv, dv), dt), ("g", g, gshape, f32),
                              ("state", state, (slots, H, dk, dv), f32), ("state_indices", state_indices, (N,), torch.int32),
                              ("out", out, (N, H, dv), dt)))
    if N > 0 and slots < (1 if state_indices is not None else N):
        raise ValueError(f"{where}: {slots} state slots for {N} sequences")
    if out is None:
        out = torch.empty_like(v) if Hv == H else torch.empty((N, H, dv), dtype=dt, device=q.device)
    _run("kda_linear_recurrent_step", dev, L.kda_linear_recurrent_step,
         _LINEAR_STEP.pack(N, H, Hq, Hk, Hv, dk, dv, code, _p(q), _p(k), _p(v), _p(g), per_token, scale, _p(state),
                           _p(state_indices), slots, _p(out)))
    return out


# ---------------------------------------------------------------- upkeep of state pools
def state_copy(pool: torch.Tensor, src: torch.Tensor, dst: torch.Tensor, *, out_pool: Optional[torch.Tensor] = None):
    """kda_state_copy: slot dst[p] becomes a copy of slot src[p], for p = 0, 1, ... in this order; src[p] = -1 clears
    the slot, dst[p] = -1 skips the pair.  pool, out_pool: [slots, ...] of any dtype (a slot's bytes a multiple of
    16); out_pool, by default the pool itself, is changed in place and returned.  src, dst: int32 [P]."""
    where, L = "state_copy", _lib or load_library()
    to = pool if out_pool is None else out_pool
    if pool.dim() < 2 or src.dim() != 1 or to.dim() != pool.dim():
        raise ValueError(f"{where}: the pools have shape [slots, ...] and src one dimension")
    dt, dev, P = pool.dtype, pool.get_device(), src.shape
    if (dev < 0 or not pool.is_contiguous() or _off(src, P, torch.int32, dev) or _off(dst, P, torch.int32, dev)
            or (to is not pool and _off(to, to.shape[:1] + pool.shape[1:], dt, dev))):
        _require(where, dev, (("pool", pool, pool.shape, dt), ("out_pool", to, to.shape[:1] + pool.shape[1:], dt),
                              ("src", src, P, torch.int32), ("dst", dst, P, torch.int32)))
    n, m = pool.shape[0], to.shape[0]
    slot = (pool.numel() // n if n else to.numel() // m if m else 0) * pool.element_size()
    _run("kda_state_copy", dev, L.kda_state_copy, _STATE_COPY.pack(_p(pool), _p(to), slot, n, m, P[0], _p(src), _p(dst)))
    return to


# ---------------------------------------------------------------- rotary positions
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}


def rope_frequencies(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0, *,
                     original_length: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0) -> torch.Tensor:
    """Frequencies of kda.rope, radians per position: float64 [rot / 2] on the host, base^(-2 i / rot).

    scaling for contexts `factor` times as long: None; "linear" (positions interpolated: every frequency divided by
    factor); "ntk" (the base raised so that the slowest frequency alone is divided by factor); "yarn" (pairs that turn
    less than beta_slow times over original_length positions as "linear", those that turn more than beta_fast times as
    they are, a ramp over the pairs' index between them; rope_attention_scale(factor) is the matching scale)."""
    if rot < 2 or rot % 2 or not base > 1 or not factor > 0:
        raise ValueError("rope_frequencies: rot is even and at least 2, base above 1, factor above 0")
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        if rot == 2:
            raise ValueError("rope_frequencies: ntk scaling needs rot > 2")
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling is None or scaling == "ntk":
        return f
    if scaling == "linear":
        return f / factor
    if scaling != "yarn":
        raise ValueError('rope_frequencies: scaling is None, "linear", "ntk" or "yarn"')
    if original_length < 1 or not beta_fast > beta_slow > 0:
        raise ValueError("rope_frequencies: yarn needs original_length and beta_fast > beta_slow > 0")

    def pair(turns):  # index of the pair that turns this often over the original length
        return rot * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot - 1)
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
    return f * (1.0 - ramp) + f / factor * ramp


def rope_attention_scale(factor: float) -> float:
    """The scale that goes with "yarn" frequencies, 0.1 ln(factor) + 1 (1 up to factor 1)."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0


def rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: torch.Tensor, freqs: torch.Tensor, *,
         layout: str = "half", scale: float = 1.0, inverse: bool = False, out_q: Optional[torch.Tensor] = None,
         out_k: Optional[torch.Tensor] = None):
    """kda_rope: rotary positions on q [T, Hq, d] and k [T, Hk, d] (either may be None).  Returns (q, k) rotated.

    positions: int32 [T] on the device; freqs: float64 [rot / 2] on the host (rope_frequencies), rotating the first
    rot channels of every head.  layout "half" pairs channel i with i + rot / 2, "interleaved" 2 i with 2 i + 1.
    inverse=True turns back, which is also the gradient: rope(grad_q, grad_k, ..., inverse=True).  out_q = q rotates in
    place; q and k may be views with a token stride (heads and channels dense), as slices of a fused projection are."""
    where, L = "rope", _lib or load_library()
    first = q if q is not None else k
    if first is None:
        raise ValueError(f"{where}: q or k is needed")
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"{where}: layout must be one of {sorted(ROPE_LAYOUTS)}")
    if first.dim() != 3:
        raise ValueError(f"{where}: q and k have three dimensions (tokens, heads, channels)")
    T, _, d = first.shape
    dt, dev = first.dtype, first.get_device()
    code = _dtype_code(first)
    if freqs.is_cuda or freqs.dtype is not torch.float64 or freqs.dim() != 1:
        raise ValueError(f"{where}: freqs is a float64 vector on the host")
    if not freqs.is_contiguous():
        freqs = freqs.contiguous()
    plain = out_q is None and out_k is None and (q is None or q.is_contiguous()) and (k is None or k.is_contiguous())
    Hq, Hk = 0 if q is None else q.shape[1], 0 if k is None else k.shape[1]
    if (dev < 0 or _off(positions, (T,), torch.int32, dev) or (plain and k is not None and _off(k, (T, Hk, d), dt, dev))):
        _require(where, dev, (("positions", positions, (T,), torch.int32), ("q", q if plain else None, (T, Hq, d), dt),
                              ("k", k if plain else None, (T, Hk, d), dt)))
    if plain:
        yq, yk = None if q is None else torch.empty_like(q), None if k is None else torch.empty_like(k)
        _run("kda_rope", dev, L.kda_rope,
             _ROPE.pack(T, Hq, Hk, d, 2 * freqs.numel(), code, ROPE_LAYOUTS[layout], int(inverse), scale, positions.data_ptr(),
                        freqs.data_ptr(), _p(q), _p(k), _p(yq), _p(yk), 0, 0, 0, 0))
        return yq, yk

    def rows(name, x, y):  # (heads, input, its token stride, output, its token stride); 0 heads: absent
        if x is None:
            return 0, None, 0, None, 0
        if x.dim() != 3 or x.shape[0] != T or x.shape[2] != d:
            raise ValueError(f"{where}: {name} has shape {tuple(x.shape)}")
        H = x.shape[1]
        dense = x.is_contiguous()
        if y is None:
            y = torch.empty_like(x) if dense else torch.empty((T, H, d), dtype=dt, device=x.device)
        strides = []
        for t in (x, y):
            if t.shape != x.shape:
                raise ValueError(f"{where}: out_{name} has shape {tuple(t.shape)}, not {tuple(x.shape)}")
            if t.dtype is not dt:
                raise TypeError(f"{where}: {name} or its output is {t.dtype}, not {dt}")
            if t.get_device() != dev:
                raise ValueError(f"{where}: {name} or its output is not on the device of the others")
            if t.is_contiguous():
                strides.append(0)
                continue
            st, sh, sd = t.stride()
            if T > 0 and H > 0 and (sd != 1 or (H > 1 and sh != d) or (T > 1 and st < H * d)):
                raise ValueError(f"{where}: {name}'s heads and channels must be dense, its tokens at most strided")
            strides.append(st if T > 1 else 0)
        return H, x, strides[0], y, strides[1]

    Hq, q, sq, yq, oq = rows("q", q, out_q)
    Hk, k, sk, yk, ok = rows("k", k, out_k)
    _run("kda_rope", dev, L.kda_rope,
         _ROPE.pack(T, Hq, Hk, d, 2 * freqs.numel(), code, ROPE_LAYOUTS[layout], int(inverse), scale, positions.data_ptr(),
                    freqs.data_ptr(), _p(q), _p(k), _p(yq), _p(yk), sq, sk, oq, ok))
    return yq, yk


def selftest_bounded_wait(device=None) -> tuple:
    """kda_selftest_bounded_wait: a wait nothing completes must give up on its own.  Returns
    (device error code read afterwards, seconds waited)."""
    L = load_library()
    t = torch.zeros((1,), dtype=torch.int64, device=device or "cuda")
    _check(L.kda_selftest_bounded_wait(_vp(t.data_ptr()), torch.cuda.current_stream(t.device).cuda_stream),
           "kda_selftest_bounded_wait")
    code = get_device_error(t.device)
    return code, int(t.item()) / 1e9


def get_device_error(device=None) -> int:
    """Waits for the current stream and returns (and clears) the device error code (0 = none)."""
    L = load_library()
    return int(L.kda_get_device_error(torch.cuda.current_stream(device).cuda_stream))


CHECK_FINITE = 1
SCHEDULES = {"auto": 0, "separate": 1, "fused": 2, "team": 3}


def set_chunk_schedule(mode: str) -> None:
    """kda_set_chunk_schedule: "auto" (the library's latency model), or force "separate", "fused" or
    "team" where the problem is eligible for it (process-wide; every schedule computes the same result)."""
    _check(load_library().kda_set_chunk_schedule(SCHEDULES[mode]), "kda_set_chunk_schedule")



def set_debug_checks(flags: int) -> None:
    """kda_set_debug_checks: with CHECK_FINITE, every entry point scans what it wrote and sets
    KDA_ERR_NUMERIC (read with get_device_error) on a NaN or an infinity; 0 turns the checks off."""
    _check(load_library().kda_set_debug_checks(int(flags)), "kda_set_debug_checks")


def status_string(code: int) -> str:
    return load_library().kda_status_string(int(code)).decode()


def set_profile_events(events) -> None:
    """Per-kernel timing: pass torch.cuda.Event objects (already recorded once), or [] to stop."""
    L = load_library()
    if not events:
        _check(L.kda_set_profile_events(None, 0), "kda_set_profile_events")
        return
    arr = (ctypes.c_void_p * len(events))(*[int(e.cuda_event) for e in events])
    _check(L.kda_set_profile_events(arr, len(events)), "kda_set_profile_events")


def chunk_fwd_kernel_count(T=0, N=1, H=1, dk=128, dv=128, dtype=torch.bfloat16, cu_seqlens_host=None,
                           gate: str = "lower_bound", out_gate: bool = False, g_min: float = -5.0) -> int:
    """Kernels kda_chunk_fwd launches for these sizes (the split-sequence state pass adds two; with
    out_gate, a separate epilogue pass adds one where the output pass does not apply it)."""
    cu = None
    if cu_seqlens_host is not None:
        cu = cu_seqlens_host.to(dtype=torch.int32, device="cpu").contiguous()
    a = ChunkArgs(T=T, N=N, H=H, dk=dk, dv=dv, dtype=KDA_BF16 if dtype == torch.bfloat16 else KDA_F32,
                  cu_seqlens_host=None if cu is None else cu.data_ptr(), chunk_size=64,
                  gate_kind=_gate_kind(gate), out_gate=16 if out_gate else None, g_min=g_min)
    return int(load_library().kda_chunk_fwd_kernel_count(ctypes.byref(a)))


def chunk_fwd_schedule(T=0, N=1, H=1, dk=128, dv=128, dtype=torch.bfloat16, cu_seqlens_host=None,
                       gate: str = "lower_bound", g_min: float = -5.0) -> dict:
    """The schedule kda_chunk_fwd picks for these sizes (see kda_chunk_fwd_schedule in kda.h)."""
    cu = None
    if cu_seqlens_host is not None:
        cu = cu_seqlens_host.to(dtype=torch.int32, device="cpu").contiguous()
    a = ChunkArgs(T=T, N=N, H=H, dk=dk, dv=dv, dtype=KDA_BF16 if dtype == torch.bfloat16 else KDA_F32,
                  cu_seqlens_host=None if cu is None else cu.data_ptr(), chunk_size=64,
                  gate_kind=_gate_kind(gate), g_min=g_min)
    out = (_i64 * 4)()
    _check(load_library().kda_chunk_fwd_schedule(ctypes.byref(a), out), "kda_chunk_fwd_schedule")
    return {"fused": out[0] == 1, "team": out[0] == 2, "own_chunks": int(out[1]) if out[0] == 1 else 0,
            "team_producers": int(out[1]) if out[0] == 2 else 0, "seg_len": int(out[2]), "kernels": int(out[3])}


def chunk_fwd_static_ws(q, k, v, z, beta, dt_bias=None, A_log=None, *, g_min: float = -5.0,
                        scale: float = 1.0, cu_seqlens: Optional[torch.Tensor] = None,
                        cu_seqlens_host: Optional[torch.Tensor] = None, n_seq: int = 1,
                        initial_state: Optional[torch.Tensor] = None,
                        final_state: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                        gate: str = "lower_bound"):
    """kda_chunk_fwd_static_ws: prefill using the library's own fixed scratch buffer.

    For callers that must not allocate device scratch: outputs (`out`,
    `final_state`) are caller-provided tensors here (allocated by this helper only
    when omitted); the library uses its internal buffer of STATIC_WORKSPACE_BYTES
    and rejects larger problems (KDA_ERR_WORKSPACE).  Calls on one device share
    that buffer, so they must not overlap in time.
    """
    L = load_library()
    T, H, dk = q.shape
    dv = v.shape[2]
    _contig(q, k, v, z, beta, dt_bias, A_log, cu_seqlens, initial_state)
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else n_seq
    if cu_seqlens_host is not None:
        cu_seqlens_host = cu_seqlens_host.to(dtype=torch.int32, device="cpu").contiguous()
    o = out if out is not None else torch.empty((T, H, dv), dtype=q.dtype, device=q.device)
    a = ChunkArgs(T=T, N=N, H=H, dk=dk, dv=dv, dtype=_dtype_code(q), q=_ptr(q), k=_ptr(k), z=_ptr(z),
                  v=_ptr(v), beta=_ptr(beta), dt_bias=_ptr(dt_bias), A_log=_ptr(A_log), g_min=g_min,
                  scale=scale, cu_seqlens=_ptr(cu_seqlens),
                  cu_seqlens_host=None if cu_seqlens_host is None else cu_seqlens_host.data_ptr(),
                  initial_state=_ptr(initial_state), final_state=_ptr(final_state), o=_ptr(o),
                  chunk_size=64, gate_kind=_gate_kind(gate))
    _check(L.kda_chunk_fwd_static_ws(ctypes.byref(a), _stream(q)), "kda_chunk_fwd_static_ws")
    return o, final_state
