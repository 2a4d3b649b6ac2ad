"""Thin Python binding of libkda (``include/kda.h``), through ctypes.

Argument marshalling only: shape/dtype checks, pointer extraction, default
output allocation through PyTorch, and the caller's current CUDA stream.  Every
step of the operator runs in the CUDA kernels behind the C ABI; when the library
is missing or fails to load, every call raises.
"""

from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple, Optional

import torch

from . import build as _build

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE, KDA_ERR_CUDA, KDA_ERR_DEVICE = range(6)
KDA_ERR_TOO_LARGE = 6
KDA_NOALLOC_MAX_SEQS = 16384
KDA_DTYPE_F32, KDA_DTYPE_BF16 = 0, 1
KDA_DEVERR_CU_SEQLENS, KDA_DEVERR_STATE_IDX = 0x1, 0x2
KDA_DEVERR_PAGES, KDA_DEVERR_EXHAUSTED, KDA_DEVERR_PARENT = 0x20, 0x40, 0x80
KDA_DEVERR_TOKEN = 0x100
KDA_BEAM_MAX_K, KDA_MAX_POOLS, KDA_FORK_MAX_ROWS = 32, 8, 8192
KDA_ROTARY_HALF, KDA_ROTARY_INTERLEAVED = 0, 1
KDA_LOGPROBS_MAX_TOP = 32

class PrefillOptions(ctypes.Structure):
    """kda_prefill_options (include/kda.h)."""
    _fields_ = [("snapshot_every", ctypes.c_int32), ("snapshots", ctypes.c_void_p),
                ("snapshot_offsets", ctypes.c_void_p), ("alpha_mode", ctypes.c_int32),
                ("single_kernel", ctypes.c_int32)]


class DecodeOptions(ctypes.Structure):
    """kda_decode_options (include/kda.h)."""
    _fields_ = [("alpha_mode", ctypes.c_int32), ("state_dtype", ctypes.c_int32)]


class Pool(ctypes.Structure):
    """kda_pool (include/kda.h); _POOL packs the same fields."""
    _fields_ = [("data", ctypes.c_void_p), ("layer_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
                ("slot_bytes", ctypes.c_int64), ("layers", ctypes.c_int32), ("slots", ctypes.c_int32)]


KDA_ALPHA_PER_CHANNEL, KDA_ALPHA_PER_HEAD, KDA_ALPHA_NONE = 0, 1, 2


# Every function include/kda.h declares, with its ctypes signature.
_vp, _i32, _i64, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
SIGNATURES = {
    "kda_prefill_workspace_size": (_sz, [_i32, _i64, _i32, _i32, _i32, ctypes.c_int]),
    "kda_prefill_launch_count": (_i64, [_i32, _i64, _i32, _i32, _i32, ctypes.c_int, _sz]),
    "kda_prefill": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32, ctypes.c_int,
                                   _f32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "kda_prefill_ex": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32, ctypes.c_int,
                                      _f32, _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "kda_decode_step": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                       ctypes.c_int, _f32, _vp]),
    "kda_prefill_backward_workspace_size": (_sz, [_i32, _i64, _i32, _i32, _i32, ctypes.c_int]),
    "kda_prefill_backward": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32,
                                            ctypes.c_int, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                            _vp, _sz, _vp]),
    "kda_decode_step_ex": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                          ctypes.c_int, _f32, _vp, _vp]),
    "kda_decode_step_bf16_state": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32,
                                                  _i32, ctypes.c_int, _f32, _vp]),
    "kda_prefill_noalloc": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32,
                                           ctypes.c_int, _f32, _vp, _vp, _vp, _vp]),
    "kda_prefill_host_buffer_size": (_sz, [_i32, _i64, _i32, _i32, _i32, ctypes.c_int]),
    "kda_prefill_host": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32, ctypes.c_int,
                                        _f32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "kda_attention_decode_workspace_size": (_sz, [_i32, _i32, _i32, _i32, ctypes.c_int]),
    "kda_attention_decode": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                            _i32, _i64, _i64, ctypes.c_int, _f32, _i32, _i32, _vp, _vp, _vp, _sz,
                                            _vp]),
    "kda_beam_select_workspace_size": (_sz, [_i32, _i32, _i32, ctypes.c_int]),
    "kda_beam_select": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i32, _i32, _i32, _i32, ctypes.c_int, _vp, _vp, _vp, _vp,
                                       _vp, _sz, _vp]),
    "kda_copy_pages": (ctypes.c_int, [_vp, _i32, _vp, _vp, _i32, _vp]),
    "kda_state_fork": (ctypes.c_int, [_vp, _i32, _vp, _vp, _i32, _vp, _vp]),
    "kda_cache_fork_workspace_size": (_sz, [_i32, _i32, _i32, _i32]),
    "kda_cache_fork": (ctypes.c_int, [_vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp,
                                      _vp, _i32, _vp, _sz, _vp]),
    "kda_cache_compact_workspace_size": (_sz, [_i32]),
    "kda_cache_compact": (ctypes.c_int, [_vp, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _sz, _vp]),
    "kda_rotary": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i64, _i64, ctypes.c_int, _i32, _f32,
                                  _i32, _vp, _i64, _vp, _i64, _vp]),
    "kda_cache_append": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                        _i64, _i64, _i64, _i32, _i32, _i32, _i64, _i64, ctypes.c_int, _i32, _f32, _vp,
                                        _i64, _vp]),
    "kda_attention_prefill_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, ctypes.c_int]),
    "kda_attention_prefill": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                             _i32, _i64, _i64, ctypes.c_int, _f32, _i32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "kda_token_logprobs": (ctypes.c_int, [_vp, _i64, _vp, _i32, _i32, ctypes.c_int, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "kda_token_logprobs_backward": (ctypes.c_int, [_vp, _i64, _vp, _vp, _vp, _vp, _vp, _i32, _i32, ctypes.c_int, _vp,
                                                   _i64, _vp]),
    "kda_get_device_error": (ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_uint32)]),
    "kda_status_string": (ctypes.c_char_p, [ctypes.c_int]),
}


class KdaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {kda_status_string(code)} ({code})")
        self.code = code


_LIB = None


def lib_path() -> str:
    """The in-tree libkda, or the library named by the KDA_LIBRARY environment variable."""
    return os.environ.get("KDA_LIBRARY") or _build.LIB


def load():
    """Load libkda (built in-tree by ``build.build()``); raises if it is missing."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libkda is not built ({path} missing); run kda_gated_delta_03_gb300.build.build()")
        L = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _LIB = L
    return _LIB


def kda_status_string(code: int) -> str:
    return load().kda_status_string(int(code)).decode()


def _dt(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return KDA_DTYPE_BF16
    if t == torch.float32:
        return KDA_DTYPE_F32
    raise TypeError(f"unsupported q/k/v dtype {t}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(name, t, dtype, shape, device):
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def kda_prefill_workspace_size(num_seqs: int, total_tokens: int, H: int, d_k: int, d_v: int,
                               dtype: torch.dtype = torch.bfloat16) -> int:
    return int(load().kda_prefill_workspace_size(num_seqs, total_tokens, H, d_k, d_v, _dt(dtype)))


def kda_prefill_launch_count(num_seqs: int, total_tokens: int, H: int, d_k: int, d_v: int,
                             dtype: torch.dtype = torch.bfloat16, workspace_bytes: int = None) -> int:
    """Kernel launches of one kda_prefill call (with the recommended workspace when none is given)."""
    if workspace_bytes is None:
        workspace_bytes = kda_prefill_workspace_size(num_seqs, total_tokens, H, d_k, d_v, dtype)
    return int(load().kda_prefill_launch_count(num_seqs, total_tokens, H, d_k, d_v, _dt(dtype), workspace_bytes))


def _alpha_shape(mode, lead, dk):
    return {KDA_ALPHA_PER_CHANNEL: (*lead, dk), KDA_ALPHA_PER_HEAD: tuple(lead)}.get(mode)


def kda_prefill(q, k, v, beta, alpha, cu_seqlens, state_in=None, *, scale: float = 1.0, state_out=None,
                o=None, workspace=None, stream=None, snapshot_every: int = 0, snapshots=None, snapshot_offsets=None,
                alpha_mode: int = KDA_ALPHA_PER_CHANNEL, single_kernel: bool = False):
    """Chunkwise prefill over packed sequences; returns (o, state_out).

    q, k [T, H, d_k], v [T, H, d_v] (bf16 or f32); beta [T, H] f32; alpha [T, H, d_k] f32;
    cu_seqlens [N + 1] int32 (device); state_in [N, H, d_k, d_v] f32 or None.
    With snapshot_every > 0 (a multiple of 64): snapshots [S, H, d_k, d_v] f32 and snapshot_offsets
    [N + 1] int32 (device) receive the state of sequence n after each multiple of snapshot_every tokens
    (kda_prefill_ex).  alpha_mode: KDA_ALPHA_PER_CHANNEL (alpha [T, H, d_k]), KDA_ALPHA_PER_HEAD (Gated
    DeltaNet, alpha [T, H]) or KDA_ALPHA_NONE (DeltaNet, alpha may be None).  single_kernel: run one bf16
    d=128 sequence on the single-kernel path instead of the two-phase path (whose fp16 operands end at
    65,504; KDA_DEVERR_RANGE reports values beyond).
    """
    L = load()
    T, H, dk = q.shape
    dv = v.shape[2]
    dev = q.device
    N = cu_seqlens.shape[0] - 1
    _check("q", q, q.dtype, (T, H, dk), dev)
    _check("k", k, q.dtype, (T, H, dk), dev)
    _check("v", v, q.dtype, (T, H, dv), dev)
    _check("beta", beta, torch.float32, (T, H), dev)
    if alpha_mode != KDA_ALPHA_NONE or alpha is not None:
        _check("alpha", alpha, torch.float32, _alpha_shape(alpha_mode, (T, H), dk), dev)
    _check("cu_seqlens", cu_seqlens, torch.int32, (N + 1,), dev)
    if state_in is not None:
        _check("state_in", state_in, torch.float32, (N, H, dk, dv), dev)
    if state_out is None:
        state_out = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    _check("state_out", state_out, torch.float32, (N, H, dk, dv), dev)
    if o is None:
        o = torch.empty((T, H, dv), dtype=q.dtype, device=dev)
    _check("o", o, q.dtype, (T, H, dv), dev)
    need = int(L.kda_prefill_workspace_size(N, T, H, dk, dv, _dt(q.dtype)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(cu_seqlens), N, T, H, dk, dv, _dt(q.dtype),
            float(scale), _ptr(state_in), _ptr(state_out), _ptr(o), _ptr(workspace), wbytes, _stream(stream))
    if snapshot_every or alpha_mode != KDA_ALPHA_PER_CHANNEL or single_kernel:
        if snapshot_every:
            S = snapshots.shape[0]
            _check("snapshots", snapshots, torch.float32, (S, H, dk, dv), dev)
            _check("snapshot_offsets", snapshot_offsets, torch.int32, (N + 1,), dev)
        opts = PrefillOptions(int(snapshot_every), _ptr(snapshots), _ptr(snapshot_offsets), int(alpha_mode),
                              int(bool(single_kernel)))
        rc = L.kda_prefill_ex(*args, ctypes.byref(opts))
        name = "kda_prefill_ex"
    else:
        rc = L.kda_prefill(*args)
        name = "kda_prefill"
    if rc != KDA_OK:
        raise KdaError(name, rc)
    return o, state_out


def kda_prefill_noalloc(q, k, v, beta, alpha, cu_seqlens, state_in=None, *, scale: float = 1.0, state_out=None,
                        o=None, stream=None):
    """kda_prefill for callers that cannot allocate device memory: no workspace argument; the library
    uses a fixed static device array (at most KDA_NOALLOC_MAX_SEQS sequences) and allocates nothing.

    Pass preallocated `state_out` and `o` to keep the whole call allocation-free; when they are None,
    this wrapper allocates them through PyTorch.  Returns (o, state_out).
    """
    L = load()
    T, H, dk = q.shape
    dv = v.shape[2]
    dev = q.device
    N = cu_seqlens.shape[0] - 1
    _check("q", q, q.dtype, (T, H, dk), dev)
    _check("k", k, q.dtype, (T, H, dk), dev)
    _check("v", v, q.dtype, (T, H, dv), dev)
    _check("beta", beta, torch.float32, (T, H), dev)
    _check("alpha", alpha, torch.float32, (T, H, dk), dev)
    _check("cu_seqlens", cu_seqlens, torch.int32, (N + 1,), dev)
    if state_in is not None:
        _check("state_in", state_in, torch.float32, (N, H, dk, dv), dev)
    if state_out is None:
        state_out = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    _check("state_out", state_out, torch.float32, (N, H, dk, dv), dev)
    if o is None:
        o = torch.empty((T, H, dv), dtype=q.dtype, device=dev)
    _check("o", o, q.dtype, (T, H, dv), dev)
    rc = L.kda_prefill_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(cu_seqlens), N, T, H, dk,
                               dv, _dt(q.dtype), float(scale), _ptr(state_in), _ptr(state_out), _ptr(o),
                               _stream(stream))
    if rc != KDA_OK:
        raise KdaError("kda_prefill_noalloc", rc)
    return o, state_out


def kda_prefill_host(q, k, v, beta, alpha, cu_seqlens, state_in=None, *, scale: float = 1.0, state_out=None,
                     o=None, device_buffer=None, stream=None):
    """kda_prefill with every tensor in host memory (CPU tensors; pin them for the copies to overlap with
    the compute).  The library streams the inputs to the device and the outputs back, segment by segment,
    through `device_buffer` (a uint8 CUDA tensor of kda_prefill_host_buffer_size bytes, allocated here when
    None).  Asynchronous on `stream`: synchronise it before reading the returned (o, state_out)."""
    L = load()
    T, H, dk = q.shape
    dv = v.shape[2]
    cpu = torch.device("cpu")
    N = cu_seqlens.shape[0] - 1
    _check("q", q, q.dtype, (T, H, dk), cpu)
    _check("k", k, q.dtype, (T, H, dk), cpu)
    _check("v", v, q.dtype, (T, H, dv), cpu)
    _check("beta", beta, torch.float32, (T, H), cpu)
    _check("alpha", alpha, torch.float32, (T, H, dk), cpu)
    _check("cu_seqlens", cu_seqlens, torch.int32, (N + 1,), cpu)
    if state_in is not None:
        _check("state_in", state_in, torch.float32, (N, H, dk, dv), cpu)
    pin = q.is_pinned()
    if state_out is None:
        state_out = torch.empty((N, H, dk, dv), dtype=torch.float32, pin_memory=pin)
    _check("state_out", state_out, torch.float32, (N, H, dk, dv), cpu)
    if o is None:
        o = torch.empty((T, H, dv), dtype=q.dtype, pin_memory=pin)
    _check("o", o, q.dtype, (T, H, dv), cpu)
    need = int(L.kda_prefill_host_buffer_size(N, T, H, dk, dv, _dt(q.dtype)))
    if device_buffer is None:
        device_buffer = torch.empty(max(need, 1), dtype=torch.uint8, device=torch.device("cuda",
                                                                                           torch.cuda.current_device()))
    rc = L.kda_prefill_host(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(cu_seqlens), N, T, H, dk, dv,
                            _dt(q.dtype), float(scale), _ptr(state_in), _ptr(state_out), _ptr(o), _ptr(device_buffer),
                            device_buffer.numel() * device_buffer.element_size(), _stream(stream))
    if rc != KDA_OK:
        raise KdaError("kda_prefill_host", rc)
    return o, state_out


def kda_decode_step(q, k, v, beta, alpha, state, state_idx=None, *, scale: float = 1.0, o=None, stream=None,
                    alpha_mode: int = KDA_ALPHA_PER_CHANNEL):
    """One fused decode step; updates `state` ([P, H, d_k, d_v] f32, or bf16 for the bf16-stored state) in
    place and returns o [B, H, d_v]."""
    L = load()
    B, H, dk = q.shape
    dv = v.shape[2]
    dev = q.device
    P = state.shape[0]
    _check("q", q, q.dtype, (B, H, dk), dev)
    _check("k", k, q.dtype, (B, H, dk), dev)
    _check("v", v, q.dtype, (B, H, dv), dev)
    _check("beta", beta, torch.float32, (B, H), dev)
    if alpha_mode != KDA_ALPHA_NONE or alpha is not None:
        _check("alpha", alpha, torch.float32, _alpha_shape(alpha_mode, (B, H), dk), dev)
    bf16_state = state.dtype == torch.bfloat16
    _check("state", state, torch.bfloat16 if bf16_state else torch.float32, (P, H, dk, dv), dev)
    if state_idx is not None:
        _check("state_idx", state_idx, torch.int32, (B,), dev)
    if o is None:
        o = torch.empty((B, H, dv), dtype=q.dtype, device=dev)
    _check("o", o, q.dtype, (B, H, dv), dev)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(state), _ptr(state_idx), P, _ptr(o), B, H,
            dk, dv, _dt(q.dtype), float(scale), _stream(stream))
    if alpha_mode != KDA_ALPHA_PER_CHANNEL:
        name = "kda_decode_step_ex"
        rc = L.kda_decode_step_ex(*args, ctypes.byref(DecodeOptions(int(alpha_mode), int(bf16_state))))
    else:
        name = "kda_decode_step_bf16_state" if bf16_state else "kda_decode_step"
        rc = getattr(L, name)(*args)
    if rc != KDA_OK:
        raise KdaError(name, rc)
    return o


def kda_prefill_backward(q, k, v, beta, alpha, cu_seqlens, grad_o, state_in=None, grad_state_out=None, *,
                         scale: float = 1.0, want_state_grad: bool = True, workspace=None, stream=None):
    """Backward pass of kda_prefill (per-channel alpha).  Returns (grad_q, grad_k, grad_v, grad_beta,
    grad_alpha, grad_state_in or None) for the loss sum(o * grad_o) + sum(state_out * grad_state_out)."""
    L = load()
    T, H, dk = q.shape
    dv = v.shape[2]
    dev = q.device
    N = cu_seqlens.shape[0] - 1
    for name, t, dt_, shape in (("q", q, q.dtype, (T, H, dk)), ("k", k, q.dtype, (T, H, dk)),
                                ("v", v, q.dtype, (T, H, dv)), ("beta", beta, torch.float32, (T, H)),
                                ("alpha", alpha, torch.float32, (T, H, dk)),
                                ("cu_seqlens", cu_seqlens, torch.int32, (N + 1,)),
                                ("grad_o", grad_o, q.dtype, (T, H, dv))):
        _check(name, t, dt_, shape, dev)
    for name, t in (("state_in", state_in), ("grad_state_out", grad_state_out)):
        if t is not None:
            _check(name, t, torch.float32, (N, H, dk, dv), dev)
    gq, gk, gv = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    gb = torch.empty((T, H), dtype=torch.float32, device=dev)
    ga = torch.empty((T, H, dk), dtype=torch.float32, device=dev)
    gs = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev) if want_state_grad else None
    need = int(L.kda_prefill_backward_workspace_size(N, T, H, dk, dv, _dt(q.dtype)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    wbytes = workspace.numel() * workspace.element_size()
    rc = L.kda_prefill_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(cu_seqlens), N, T, H, dk,
                                dv, _dt(q.dtype), float(scale), _ptr(state_in), _ptr(grad_o), _ptr(grad_state_out),
                                _ptr(gq), _ptr(gk), _ptr(gv), _ptr(gb), _ptr(ga), _ptr(gs), _ptr(workspace), wbytes,
                                _stream(stream))
    if rc != KDA_OK:
        raise KdaError("kda_prefill_backward", rc)
    return gq, gk, gv, gb, ga, gs


# ---- decoding a hybrid stack: one call of these takes microseconds, so the checks here stay light ----
_POOL = struct.Struct("@Pqqqii")
_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8
_DTYPES = {torch.float32: KDA_DTYPE_F32, torch.bfloat16: KDA_DTYPE_BF16}
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _check_at(name, t, dtype, shape, dev):
    """_check with the device as its index."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, expected CUDA device {dev}")


def _cuda_index(name, t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _raw_stream(stream, dev):
    return _current_raw_stream(dev) if stream is None else stream.cuda_stream


def _in_stream(stream, call, *args, **kwargs):
    """The call with `stream` as the current one, so that what it allocates itself belongs to that stream: a block of
    another stream's may still be in use there, or be handed out again before this stream is done with it."""
    with torch.cuda.stream(stream):
        return call(*args, **kwargs)


def _too_large(name, *values):
    """Raises for numbers that do not fit the C ABI's 32 bits, of which ctypes would pass the lower ones.  (Callers look at all
    of them at once: or'ed together they are within 31 bits if each is, and the library refuses negative ones.)"""
    raise ValueError(f"{name}: one of the sizes and numbers {values} does not fit 32 bits")


def _workspace(workspace, dev):
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on CUDA device {dev}")
    return workspace.numel() * workspace.element_size()


def _new_workspace(need, dev):
    return torch.empty(max(need, 1), dtype=_U8, device=torch.device("cuda", dev))


def _pools(pools, dev):
    """kda_pool records of tensors [layers, slots, ...] whose slots are contiguous: (bytes, how many)."""
    if isinstance(pools, torch.Tensor):
        pools = (pools,)
    packed = []
    for t in pools:
        shape, stride, e = t.shape, t.stride(), t.element_size()
        if len(shape) < 3:
            raise ValueError(f"pool: shape {tuple(shape)}, expected [layers, slots, ...]")
        if t.get_device() != dev:
            raise ValueError(f"pool is on {t.device}, expected CUDA device {dev}")
        layers, slots = shape[0], shape[1]
        n = 1
        for size in shape[2:]:
            n *= size
        if not t.is_contiguous():
            m = 1
            for size, step in zip(reversed(shape[2:]), reversed(stride[2:])):
                if size != 1 and step != m:
                    raise ValueError("pool: a slot must be contiguous")
                m *= size
        packed.append(_POOL.pack(t.data_ptr(), stride[0] * e if layers > 1 else 0, stride[1] * e if slots > 1 else 0,
                                 n * e, layers, slots))
    return b"".join(packed), len(packed)


def _page_stride(name, t, shape, dtype, dev):
    """Elements from page to page of a pool [P, H_kv, page_size, d] whose pages are contiguous."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected CUDA device {dev}")
    if not t.is_contiguous() and shape[0] and not t[0].is_contiguous():
        raise ValueError(f"{name}: a page must be contiguous")
    return t.stride(0)


def kda_attention_decode_workspace_size(B: int, H_q: int, H_kv: int, d: int,
                                        dtype: torch.dtype = torch.bfloat16) -> int:
    return int(load().kda_attention_decode_workspace_size(B, H_q, H_kv, d, _dt(dtype)))


def kda_attention_decode(q, k_pages, v_pages, block_table, seq_lens, *, scale: float = 1.0, window: int = 0,
                         sinks: int = 0, k_new=None, v_new=None, o=None, lse=None, workspace=None, stream=None):
    """Attention of one new token per sequence over a paged key-value cache; returns o [B, H_q, d].

    q [B, H_q, d] (bf16 or f32); k_pages, v_pages [P, H_kv, page_size, d] of q's dtype (a view whose pages are
    contiguous will do, e.g. one half of a [P, 2, H_kv, page_size, d] pool); block_table [B, M] int32 page
    numbers, seq_lens [B] int32 with the new token.  k_new, v_new [B, H_kv, d]: the new token's key and value,
    stored at position seq_lens - 1 by this call.  window > 0: only the last `window` tokens and the first
    `sinks` are visible.  lse [B, H_q] f32, if given, receives the log of the softmax's sum.
    """
    if stream is not None and (o is None or workspace is None):
        return _in_stream(stream, kda_attention_decode, q, k_pages, v_pages, block_table, seq_lens, scale=scale,
                          window=window, sinks=sinks, k_new=k_new, v_new=v_new, o=o, lse=lse, workspace=workspace)
    L = _LIB or load()
    B, Hq, d = q.shape
    shape = P, Hkv, ps, _ = k_pages.shape
    dt, dev = q.dtype, _cuda_index("q", q)
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}")
    if d != shape[3]:
        raise ValueError(f"k_pages: shape {tuple(shape)}, expected a last dimension of {d}")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    ks = _page_stride("k_pages", k_pages, shape, dt, dev)
    vs = _page_stride("v_pages", v_pages, shape, dt, dev)
    M = block_table.shape[1]
    if (B | Hq | Hkv | P | M | ps | window | sinks) >> 31 not in (0, -1):
        _too_large("kda_attention_decode", B, Hq, Hkv, P, M, ps, window, sinks)
    _check_at("block_table", block_table, _I32, (B, M), dev)
    _check_at("seq_lens", seq_lens, _I32, (B,), dev)
    kn = vn = out_lse = None
    if k_new is not None or v_new is not None:
        if k_new is None or v_new is None:
            raise ValueError("k_new and v_new go together")
        _check_at("k_new", k_new, dt, (B, Hkv, d), dev)
        _check_at("v_new", v_new, dt, (B, Hkv, d), dev)
        kn, vn = k_new.data_ptr(), v_new.data_ptr()
    if o is None:
        o = torch.empty_like(q)
    else:
        _check_at("o", o, dt, (B, Hq, d), dev)
    if lse is not None:
        _check_at("lse", lse, _F32, (B, Hq), dev)
        out_lse = lse.data_ptr()
    if workspace is None:
        workspace = _new_workspace(L.kda_attention_decode_workspace_size(B, Hq, Hkv, d, code), dev)
    wbytes = _workspace(workspace, dev)
    rc = L.kda_attention_decode(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                                seq_lens.data_ptr(), kn, vn, B, Hq, Hkv, d, P, ps, M, ks, vs, code, scale, window,
                                sinks, o.data_ptr(), out_lse, workspace.data_ptr(), wbytes, _raw_stream(stream, dev))
    if rc != KDA_OK:
        raise KdaError("kda_attention_decode", rc)
    return o


def kda_beam_select_workspace_size(N: int, K: int, V: int, dtype: torch.dtype = torch.bfloat16) -> int:
    return int(load().kda_beam_select_workspace_size(N, K, V, _dt(dtype)))


def kda_beam_select(logits, beam_scores, *, finished=None, eos_token: int = -1, scores_out=None, parent=None,
                    token=None, finished_out=None, workspace=None, stream=None):
    """A beam search's selection; returns (scores, parent, token, finished or None), each [N, K], best first.

    logits [N * K, V] (bf16 or f32; rows may lie further apart than V), beam_scores [N, K] f32.  A beam's
    continuation v scores beam_scores + log_softmax(logits)[v]; the K best of a group's K * V, the lowest
    place first among equal ones.  parent holds row numbers n * K + b, as kda_state_fork and kda_cache_fork take
    them.  finished [N, K] uint8: such a beam goes on with eos_token alone, at its unchanged score.
    """
    if stream is not None and (workspace is None or scores_out is None or parent is None or token is None or finished_out is None):
        return _in_stream(stream, kda_beam_select, logits, beam_scores, finished=finished, eos_token=eos_token,
                          scores_out=scores_out, parent=parent, token=token, finished_out=finished_out,
                          workspace=workspace)
    L = _LIB or load()
    N, K = beam_scores.shape
    V = logits.shape[1]
    dev = _cuda_index("logits", logits)
    if logits.shape != (N * K, V):
        raise ValueError(f"logits: shape {tuple(logits.shape)}, expected {(N * K, V)}")
    step, inner = logits.stride()
    if inner != 1 and V > 1 or step < V and N * K > 1:
        raise ValueError("logits: a row must be contiguous")
    _check_at("beam_scores", beam_scores, _F32, (N, K), dev)
    if finished is not None:
        _check_at("finished", finished, _U8, (N, K), dev)
    if scores_out is None:
        scores_out = torch.empty_like(beam_scores)
    else:
        _check_at("scores_out", scores_out, _F32, (N, K), dev)
    if parent is None:
        parent = torch.empty((N, K), dtype=torch.int32, device=logits.device)
    else:
        _check_at("parent", parent, _I32, (N, K), dev)
    if token is None:
        token = torch.empty((N, K), dtype=torch.int32, device=logits.device)
    else:
        _check_at("token", token, _I32, (N, K), dev)
    if finished_out is None:
        if finished is not None:
            finished_out = torch.empty_like(finished)
    else:
        _check_at("finished_out", finished_out, _U8, (N, K), dev)
    code = _DTYPES.get(logits.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {logits.dtype}")
    if workspace is None:
        workspace = _new_workspace(L.kda_beam_select_workspace_size(N, K, V, code), dev)
    wbytes = _workspace(workspace, dev)
    rc = L.kda_beam_select(logits.data_ptr(), max(step, V), beam_scores.data_ptr(),
                           None if finished is None else finished.data_ptr(), eos_token, N, K, V, code,
                           scores_out.data_ptr(), parent.data_ptr(), token.data_ptr(),
                           None if finished_out is None else finished_out.data_ptr(), workspace.data_ptr(), wbytes,
                           _raw_stream(stream, dev))
    if rc != KDA_OK:
        raise KdaError("kda_beam_select", rc)
    return scores_out, parent, token, finished_out


def kda_copy_pages(pools, src, dst, *, stream=None):
    """Copies slot src[i] to slot dst[i] on every layer of every pool.  pools: tensors [layers, slots, ...]
    (any dtype, contiguous slots); src, dst [n] int32 (src None: src[i] = i); negative entries are skipped."""
    dev = _cuda_index("dst", dst)
    n = dst.shape[0]
    _check_at("dst", dst, _I32, (n,), dev)
    if src is not None:
        _check_at("src", src, _I32, (n,), dev)
    arr, count = _pools(pools, dev)
    rc = (_LIB or load()).kda_copy_pages(arr, count, None if src is None else src.data_ptr(), dst.data_ptr(), n,
                               _raw_stream(stream, dev))
    if rc != KDA_OK:
        raise KdaError("kda_copy_pages", rc)


def kda_state_fork(pools, state_idx, parent, *, state_idx_out=None, stream=None):
    """Gives each row i of a decode batch the state of row parent[i] (-1: a row that starts anew); returns the
    new state_idx [B], a permutation of the old one.  pools: one tensor or several [layers, slots, ...] of
    states (kda_decode_step's pool is pool[layer]).  Copies only states that two rows continue."""
    if stream is not None and (state_idx_out is None or not parent.is_contiguous()):
        return _in_stream(stream, kda_state_fork, pools, state_idx, parent, state_idx_out=state_idx_out)
    dev = _cuda_index("state_idx", state_idx)
    parent = parent.reshape(-1) if parent.dim() != 1 else parent
    B = state_idx.shape[0]
    _check_at("state_idx", state_idx, _I32, (B,), dev)
    _check_at("parent", parent, _I32, (B,), dev)
    if state_idx_out is None:
        state_idx_out = torch.empty_like(state_idx)
    else:
        _check_at("state_idx_out", state_idx_out, _I32, (B,), dev)
    arr, count = _pools(pools, dev)
    rc = (_LIB or load()).kda_state_fork(arr, count, state_idx.data_ptr(), parent.data_ptr(), B, state_idx_out.data_ptr(),
                               _raw_stream(stream, dev))
    if rc != KDA_OK:
        raise KdaError("kda_state_fork", rc)
    return state_idx_out


def kda_cache_fork_workspace_size(rows_in: int, rows_out: int, max_pages: int, num_pages: int) -> int:
    return int(load().kda_cache_fork_workspace_size(rows_in, rows_out, max_pages, num_pages))


def kda_cache_fork(block_table, seq_lens, parent, ref_count, page_size: int, *, grow=None, pools=(),
                   block_table_out=None, seq_lens_out=None, ref_count_out=None, copy_src=None, copy_dst=None,
                   workspace=None, stream=None):
    """Replaces the rows of a block table: row i continues old row parent[i] (-1: an empty row) and gets room
    for grow[i] more tokens.  Returns (block_table, seq_lens, ref_count) of the new rows.

    block_table [R, M], seq_lens [R], parent [R'], grow [R'] or None, ref_count [P], all int32.  Whole pages
    are shared and counted, a partly filled last page stays with one row and is copied for the others (on every
    layer of `pools`, tensors [layers, P, ...]), and pages come from the free ones, the lowest first.
    ref_count is updated in place unless ref_count_out is given.  copy_src, copy_dst [R'] receive the pages
    copied, for pools that are not passed here.
    """
    if stream is not None and (block_table_out is None or seq_lens_out is None or workspace is None or not parent.is_contiguous()):
        return _in_stream(stream, kda_cache_fork, block_table, seq_lens, parent, ref_count, page_size, grow=grow,
                          pools=pools, block_table_out=block_table_out, seq_lens_out=seq_lens_out,
                          ref_count_out=ref_count_out, copy_src=copy_src, copy_dst=copy_dst, workspace=workspace)
    L = _LIB or load()
    dev = _cuda_index("block_table", block_table)
    parent = parent.reshape(-1) if parent.dim() != 1 else parent
    R, M = block_table.shape
    P, R2 = ref_count.shape[0], parent.shape[0]
    _check_at("block_table", block_table, _I32, (R, M), dev)
    _check_at("seq_lens", seq_lens, _I32, (R,), dev)
    _check_at("parent", parent, _I32, (R2,), dev)
    _check_at("ref_count", ref_count, _I32, (P,), dev)
    if grow is not None:
        _check_at("grow", grow, _I32, (R2,), dev)
    if block_table_out is None:
        block_table_out = torch.empty((R2, M), dtype=torch.int32, device=block_table.device)
    else:
        _check_at("block_table_out", block_table_out, _I32, (R2, M), dev)
    if seq_lens_out is None:
        seq_lens_out = torch.empty(R2, dtype=torch.int32, device=block_table.device)
    else:
        _check_at("seq_lens_out", seq_lens_out, _I32, (R2,), dev)
    if ref_count_out is None:
        ref_count_out = ref_count
    else:
        _check_at("ref_count_out", ref_count_out, _I32, (P,), dev)
    cs = cd = None
    if copy_src is not None or copy_dst is not None:
        _check_at("copy_src", copy_src, _I32, (R2,), dev)
        _check_at("copy_dst", copy_dst, _I32, (R2,), dev)
        cs, cd = copy_src.data_ptr(), copy_dst.data_ptr()
    arr, count = _pools(pools, dev)
    if workspace is None:
        workspace = _new_workspace(L.kda_cache_fork_workspace_size(R, R2, M, P), dev)
    wbytes = _workspace(workspace, dev)
    rc = L.kda_cache_fork(block_table.data_ptr(), seq_lens.data_ptr(), R, parent.data_ptr(),
                          None if grow is None else grow.data_ptr(), R2, M, page_size, ref_count.data_ptr(), P,
                          block_table_out.data_ptr(), seq_lens_out.data_ptr(), ref_count_out.data_ptr(), cs, cd, arr,
                          count, workspace.data_ptr(), wbytes, _raw_stream(stream, dev))
    if rc != KDA_OK:
        raise KdaError("kda_cache_fork", rc)
    return block_table_out, seq_lens_out, ref_count_out


def kda_cache_compact_workspace_size(num_pages: int) -> int:
    return int(load().kda_cache_compact_workspace_size(num_pages))


def kda_cache_compact(block_table, ref_count, *, pools=(), block_table_out=None, ref_count_out=None, page_map=None,
                      workspace=None, stream=None):
    """Moves the live pages (ref_count > 0) together at the low end of the pools; returns (block_table,
    ref_count, page_map) with the new numbers.  block_table and ref_count are updated in place unless outputs are
    given; page_map [P] int32 holds each page's new number, -1 for a free one."""
    if stream is not None and (page_map is None or workspace is None):
        return _in_stream(stream, kda_cache_compact, block_table, ref_count, pools=pools,
                          block_table_out=block_table_out, ref_count_out=ref_count_out, page_map=page_map,
                          workspace=workspace)
    L = _LIB or load()
    dev = _cuda_index("block_table", block_table)
    R, M = block_table.shape
    P = ref_count.shape[0]
    _check_at("block_table", block_table, _I32, (R, M), dev)
    _check_at("ref_count", ref_count, _I32, (P,), dev)
    if block_table_out is None:
        block_table_out = block_table
    else:
        _check_at("block_table_out", block_table_out, _I32, (R, M), dev)
    if ref_count_out is None:
        ref_count_out = ref_count
    else:
        _check_at("ref_count_out", ref_count_out, _I32, (P,), dev)
    if page_map is None:
        page_map = torch.empty_like(ref_count)
    else:
        _check_at("page_map", page_map, _I32, (P,), dev)
    arr, count = _pools(pools, dev)
    if workspace is None:
        workspace = _new_workspace(L.kda_cache_compact_workspace_size(P), dev)
    wbytes = _workspace(workspace, dev)
    rc = L.kda_cache_compact(block_table.data_ptr(), R, M, ref_count.data_ptr(), P, block_table_out.data_ptr(),
                             ref_count_out.data_ptr(), page_map.data_ptr(), arr, count, workspace.data_ptr(), wbytes,
                             _raw_stream(stream, dev))
    if rc != KDA_OK:
        raise KdaError("kda_cache_compact", rc)
    return block_table_out, ref_count_out, page_map


# ---- a prompt's way through the full-attention layers, and the scores of its tokens ----
_F64 = torch.float64
_LAYOUTS = {"half": KDA_ROTARY_HALF, "interleaved": KDA_ROTARY_INTERLEAVED}
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _elsewhere(dev, stream):
    """Whether a call has to change the current device or stream before it allocates and launches."""
    return stream is not None or dev != _current_device()


def _there(dev, stream, call, *args, **kwargs):
    """The call on its tensors' device and with `stream` as the current one (see _in_stream)."""
    if stream is not None and stream.device_index != dev:                     # (it would run on some other stream)
        raise ValueError(f"stream is on CUDA device {stream.device_index}, the tensors on {dev}")
    with torch.cuda.device(dev):
        if stream is None:
            return call(*args, **kwargs)
        return _in_stream(stream, call, *args, **kwargs)


def _heads(name, t, T, d, dtype, dev):
    """A tensor [T, H, d] whose tokens are contiguous, as a slice of a fused projection is: (H, elements a token)."""
    shape = t.shape
    if len(shape) == 3 and shape[0] == T and shape[2] == d and t.dtype is dtype and t.get_device() == dev:
        H, (step, head, inner) = shape[1], t.stride()
        if inner == 1 and head == d and step >= H * d:
            return H, step
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.dim() != 3 or t.shape[0] != T or t.shape[2] != d:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(T, 'heads', d)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected CUDA device {dev}")
    H = t.shape[1]
    step, head, inner = t.stride()
    if inner != 1 and d > 1 or head != d and H > 1 or step < H * d and T > 1:
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return H, max(step, H * d)


def _out_stride(name, t, shape, dtype, dev):
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    return _heads(name, t, shape[0], shape[2], dtype, dev)[1]


def _frequencies(inv_freq, dev):
    if inv_freq is None:
        return 0, None
    shape = inv_freq.shape
    if len(shape) != 1:
        raise ValueError(f"inv_freq: shape {tuple(shape)}, expected [rotary_dim / 2]")
    _check_at("inv_freq", inv_freq, _F64, shape, dev)
    n = shape[0]
    return 2 * n, inv_freq.data_ptr() if n else None


def _layout(layout):
    code = _LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"layout {layout!r}, expected 'half' or 'interleaved'")
    return code


def kda_rotary(q, k, positions, inv_freq, *, layout: str = "half", rotary_scale: float = 1.0, inverse: bool = False,
               q_out=None, k_out=None, stream=None):
    """Rotary positions of queries and keys; returns (q_out, k_out).

    q [T, H_q, d], k [T, H_kv, d] or None (bf16 or f32; slices of a fused projection will do), positions [T] int32,
    inv_freq [rotary_dim / 2] f64: radians a position, for the pairs (x_i, x_{i + rotary_dim / 2}) (layout "half")
    or (x_2i, x_{2i + 1}) ("interleaved") of every head; the rest of a head is copied.  rotary_scale multiplies
    the rotated part (stretched contexts).  inverse=True turns back with the same scale: the gradient of q, k from
    those of the outputs.  q_out, k_out may be q and k.
    """
    dev = _cuda_index("q", q)
    if _elsewhere(dev, stream):
        return _there(dev, stream, kda_rotary, q, k, positions, inv_freq, layout=layout, rotary_scale=rotary_scale,
                      inverse=inverse, q_out=q_out, k_out=k_out)
    if q.dim() != 3:
        raise ValueError(f"q: shape {tuple(q.shape)}, expected [T, H_q, d]")
    shape = q.shape
    T, d, dt = shape[0], shape[2], q.dtype
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}")
    Hq, qs = _heads("q", q, T, d, dt, dev)
    _check_at("positions", positions, _I32, (T,), dev)
    rot, freq = _frequencies(inv_freq, dev)
    if q_out is None:
        q_out = q.new_empty(shape)
        qos = Hq * d
    else:
        qos = _out_stride("q_out", q_out, shape, dt, dev)
    Hkv = ks = kos = 0
    if k is not None:
        Hkv, ks = _heads("k", k, T, d, dt, dev)
        if k_out is None:
            k_out = k.new_empty(k.shape)
            kos = Hkv * d
        else:
            kos = _out_stride("k_out", k_out, k.shape, dt, dev)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if (T | Hq | Hkv | d) >> 31:
        _too_large("kda_rotary", T, Hq, Hkv, d)
    rc = (_LIB or load()).kda_rotary(q.data_ptr(), None if k is None else k.data_ptr(), positions.data_ptr(), freq, T, Hq,
                                     Hkv, d, rot, qs, ks, code, _layout(layout), rotary_scale, int(inverse),
                                     q_out.data_ptr(), qos, None if k is None else k_out.data_ptr(), kos,
                                     _current_raw_stream(dev))
    if rc != KDA_OK:
        raise KdaError("kda_rotary", rc)
    return q_out, k_out


def kda_cache_append(k, v, k_pages, v_pages, block_table, seq_lens, cu_seqlens, *, q=None, inv_freq=None,
                     layout: str = "half", rotary_scale: float = 1.0, q_out=None, stream=None):
    """Stores a packed batch's new keys and values in their pages; returns q_out (None without q).

    k, v [T, H_kv, d] (bf16 or f32; slices of a fused projection will do): the tokens cu_seqlens[b] .. cu_seqlens[b + 1]
    - 1 go to positions seq_lens[b] - n_b .. seq_lens[b] - 1 of row b of block_table [B, M] (pools as for
    kda_attention_decode; seq_lens with the new tokens, as kda_cache_fork returns it).  With inv_freq (see kda_rotary)
    keys, and queries q [T, H_q, d], are rotated by those positions; q_out may be q.
    """
    dev = _cuda_index("k", k)
    if _elsewhere(dev, stream):
        return _there(dev, stream, kda_cache_append, k, v, k_pages, v_pages, block_table, seq_lens, cu_seqlens, q=q,
                      inv_freq=inv_freq, layout=layout, rotary_scale=rotary_scale, q_out=q_out)
    if k.dim() != 3:
        raise ValueError(f"k: shape {tuple(k.shape)}, expected [T, H_kv, d]")
    T, d, dt = k.shape[0], k.shape[2], k.dtype
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}")
    Hkv, ks = _heads("k", k, T, d, dt, dev)
    if v.shape != k.shape:
        raise ValueError(f"v: shape {tuple(v.shape)}, expected {tuple(k.shape)}")
    vs = _heads("v", v, T, d, dt, dev)[1]
    if k_pages.dim() != 4:
        raise ValueError(f"k_pages: shape {tuple(k_pages.shape)}, expected [P, H_kv, page_size, d]")
    P, _, ps, _ = k_pages.shape
    shape = (P, Hkv, ps, d)
    kps = _page_stride("k_pages", k_pages, shape, dt, dev)
    vps = _page_stride("v_pages", v_pages, shape, dt, dev)
    B, M = block_table.shape
    _check_at("block_table", block_table, _I32, (B, M), dev)
    _check_at("seq_lens", seq_lens, _I32, (B,), dev)
    _check_at("cu_seqlens", cu_seqlens, _I32, (B + 1,), dev)
    rot, freq = _frequencies(inv_freq, dev)
    Hq = qs = qos = 0
    if q is not None:
        Hq, qs = _heads("q", q, T, d, dt, dev)
        if q_out is None:
            q_out = q.new_empty(q.shape)
            qos = Hq * d
        else:
            qos = _out_stride("q_out", q_out, q.shape, dt, dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if (T | B | Hq | Hkv | P | M | ps) >> 31:
        _too_large("kda_cache_append", T, B, Hq, Hkv, P, M, ps)
    rc = (_LIB or load()).kda_cache_append(
        None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
        block_table.data_ptr(), seq_lens.data_ptr(), cu_seqlens.data_ptr(), freq, B, T, Hq, Hkv, d, rot, qs, ks, vs, P, ps,
        M, kps, vps, code, _layout(layout), rotary_scale, None if q is None else q_out.data_ptr(), qos,
        _current_raw_stream(dev))
    if rc != KDA_OK:
        raise KdaError("kda_cache_append", rc)
    return q_out


def kda_attention_prefill_workspace_size(B: int, T: int, H_q: int, H_kv: int, d: int,
                                         dtype: torch.dtype = torch.bfloat16) -> int:
    return int(load().kda_attention_prefill_workspace_size(B, T, H_q, H_kv, d, _dt(dtype)))


def kda_attention_prefill(q, k_pages, v_pages, block_table, seq_lens, cu_seqlens, *, scale: float = 1.0, window: int = 0,
                          sinks: int = 0, o=None, lse=None, workspace=None, stream=None):
    """Attention of a packed batch's new tokens over a paged cache that holds them already; returns o [T, H_q, d].

    q [T, H_q, d] (bf16 or f32), tokens cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of row b at positions seq_lens[b] - n_b ..
    seq_lens[b] - 1: whole prompts, chunks behind what the cache holds, single tokens.  Each sees the tokens up to
    itself; with window > 0 only the last `window` of them and the first `sinks`.  Pools and table as for
    kda_attention_decode.  lse [T, H_q] f32, if given, receives the log of the softmax's sum.  Tokens behind
    cu_seqlens[B] are left as they were.
    """
    dev = _cuda_index("q", q)
    if _elsewhere(dev, stream):
        return _there(dev, stream, kda_attention_prefill, q, k_pages, v_pages, block_table, seq_lens, cu_seqlens,
                      scale=scale, window=window, sinks=sinks, o=o, lse=lse, workspace=workspace)
    L = _LIB or load()
    if q.dim() != 3:
        raise ValueError(f"q: shape {tuple(q.shape)}, expected [T, H_q, d]")
    if k_pages.dim() != 4:
        raise ValueError(f"k_pages: shape {tuple(k_pages.shape)}, expected [P, H_kv, page_size, d]")
    T, Hq, d = q.shape
    shape = P, Hkv, ps, _ = k_pages.shape
    dt = q.dtype
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}")
    if d != shape[3]:
        raise ValueError(f"k_pages: shape {tuple(shape)}, expected a last dimension of {d}")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    ks = _page_stride("k_pages", k_pages, shape, dt, dev)
    vs = _page_stride("v_pages", v_pages, shape, dt, dev)
    B, M = block_table.shape
    if (T | B | Hq | Hkv | P | M | ps | window | sinks) >> 31 not in (0, -1):
        _too_large("kda_attention_prefill", T, B, Hq, Hkv, P, M, ps, window, sinks)
    _check_at("block_table", block_table, _I32, (B, M), dev)
    _check_at("seq_lens", seq_lens, _I32, (B,), dev)
    _check_at("cu_seqlens", cu_seqlens, _I32, (B + 1,), dev)
    out_lse = None
    if o is None:
        o = torch.empty_like(q)
    else:
        _check_at("o", o, dt, (T, Hq, d), dev)
    if lse is not None:
        _check_at("lse", lse, _F32, (T, Hq), dev)
        out_lse = lse.data_ptr()
    if workspace is None:
        workspace = _new_workspace(L.kda_attention_prefill_workspace_size(B, T, Hq, Hkv, d, code), dev)
    wbytes = _workspace(workspace, dev)
    rc = L.kda_attention_prefill(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                                 seq_lens.data_ptr(), cu_seqlens.data_ptr(), B, T, Hq, Hkv, d, P, ps, M, ks, vs, code,
                                 scale, window, sinks, o.data_ptr(), out_lse, workspace.data_ptr(), wbytes,
                                 _current_raw_stream(dev))
    if rc != KDA_OK:
        raise KdaError("kda_attention_prefill", rc)
    return o


class TokenLogprobs(NamedTuple):
    """What kda_token_logprobs returns."""
    logp: torch.Tensor                        # [T] f32
    lse: torch.Tensor                         # [T] f32
    entropy: Optional[torch.Tensor]           # [T] f32, or None
    top_logp: torch.Tensor                    # [T, top] f32
    top_token: torch.Tensor                   # [T, top] int32


def _rows(name, t, dev):
    """A matrix [T, V] with contiguous rows: (T, V, elements a row)."""
    if len(t.shape) != 2:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [T, V]")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected CUDA device {dev}")
    T, V = t.shape
    step, inner = t.stride()
    if inner != 1 and V > 1 or step < V and T > 1:
        raise ValueError(f"{name}: a row must be contiguous")
    return T, V, max(step, V)


def kda_token_logprobs(logits, tokens, *, top: int = 0, entropy: bool = False, stream=None) -> TokenLogprobs:
    """Log probabilities of given tokens under rows of logits; returns a TokenLogprobs.

    logits [T, V] (bf16 or f32; rows may lie further apart than V), tokens [T] int32, -1: none, which gives 0.  lse is the
    log of a row's sum, entropy (if asked for) that of its distribution, top_logp and top_token its `top` likeliest words
    (at most 32), best first, the lowest word first among equal logits.
    """
    dev = _cuda_index("logits", logits)
    if _elsewhere(dev, stream):
        return _there(dev, stream, kda_token_logprobs, logits, tokens, top=top, entropy=entropy)
    T, V, step = _rows("logits", logits, dev)
    code = _DTYPES.get(logits.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {logits.dtype}")
    if (T | V | top) >> 31 not in (0, -1):
        _too_large("kda_token_logprobs", T, V, top)
    _check_at("tokens", tokens, _I32, (T,), dev)
    k, on = max(top, 0), logits.device
    logp, lse = torch.empty((T,), dtype=_F32, device=on), torch.empty((T,), dtype=_F32, device=on)
    H = torch.empty((T,), dtype=_F32, device=on) if entropy else None
    best, word = torch.empty((T, k), dtype=_F32, device=on), torch.empty((T, k), dtype=_I32, device=on)
    rc = (_LIB or load()).kda_token_logprobs(logits.data_ptr(), step, tokens.data_ptr(), T, V, code, top, logp.data_ptr(),
                                             lse.data_ptr(), H.data_ptr() if entropy else None,
                                             best.data_ptr() if top else None, word.data_ptr() if top else None,
                                             _current_raw_stream(dev))
    if rc != KDA_OK:
        raise KdaError("kda_token_logprobs", rc)
    return TokenLogprobs(logp, lse, H, best, word)


def kda_token_logprobs_backward(logits, tokens, lse, grad_logp, *, entropy=None, grad_entropy=None, grad=None,
                                stream=None):
    """The gradient of kda_token_logprobs with regard to the logits; returns grad [T, V] of the logits' type.

    lse [T] f32 as kda_token_logprobs gave it, grad_logp [T] f32; entropy and grad_entropy [T] f32 go together.  grad may
    be logits (in their place).
    """
    dev = _cuda_index("logits", logits)
    if _elsewhere(dev, stream):
        return _there(dev, stream, kda_token_logprobs_backward, logits, tokens, lse, grad_logp, entropy=entropy,
                      grad_entropy=grad_entropy, grad=grad)
    T, V, step = _rows("logits", logits, dev)
    code = _DTYPES.get(logits.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {logits.dtype}")
    if (T | V) >> 31:
        _too_large("kda_token_logprobs_backward", T, V)
    _check_at("tokens", tokens, _I32, (T,), dev)
    _check_at("lse", lse, _F32, (T,), dev)
    _check_at("grad_logp", grad_logp, _F32, (T,), dev)
    if (entropy is None) != (grad_entropy is None):
        raise ValueError("entropy and grad_entropy go together")
    if entropy is not None:
        _check_at("entropy", entropy, _F32, (T,), dev)
        _check_at("grad_entropy", grad_entropy, _F32, (T,), dev)
    if grad is None:
        grad = torch.empty((T, V), dtype=logits.dtype, device=logits.device)
    if grad.dtype is not logits.dtype:
        raise TypeError(f"grad: dtype {grad.dtype}, expected {logits.dtype}")
    if grad.shape != logits.shape:
        raise ValueError(f"grad: shape {tuple(grad.shape)}, expected {tuple(logits.shape)}")
    gstep = _rows("grad", grad, dev)[2]
    rc = (_LIB or load()).kda_token_logprobs_backward(
        logits.data_ptr(), step, tokens.data_ptr(), lse.data_ptr(), None if entropy is None else entropy.data_ptr(),
        grad_logp.data_ptr(), None if entropy is None else grad_entropy.data_ptr(), T, V, code, grad.data_ptr(), gstep,
        _current_raw_stream(dev))
    if rc != KDA_OK:
        raise KdaError("kda_token_logprobs_backward", rc)
    return grad


def kda_get_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error bits."""
    bits = ctypes.c_uint32(0)
    rc = load().kda_get_device_error(_stream(stream), ctypes.byref(bits))
    if rc not in (KDA_OK, KDA_ERR_DEVICE):
        raise KdaError("kda_get_device_error", rc)
    return int(bits.value)
