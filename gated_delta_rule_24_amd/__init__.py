"""Gated delta rule layer core on MI355X (gfx950): a thin Python binding.

Everything numeric runs in the HIP kernels of libgdn.so, reached through its
C ABI (include/gdn.h).  This module only marshals torch tensors (device
memory and the current HIP stream) into that ABI: it checks devices, dtypes
and contiguity, allocates outputs and the workspace, and raises GdnError on a
non-OK status.  There is no CPU fallback: if libgdn.so is missing or cannot
be loaded, every call raises.

    o, S = chunk_fwd(q, k, v, log_alpha, beta, init_state=None, cu_seqlens=None)
    o    = decode_step(state, q, k, v, log_alpha, beta)      # state updated in place

Next to the gated delta rule, with the same conventions: the elementwise gated
linear recurrence, layer norm, and moves of resident states.

    h, s = scan_fwd(x, log_alpha, init_state=None, cu_seqlens=None)
    dx, dlog_alpha, d_init = scan_bwd(log_alpha, h, d_h, init_state=None, d_final=None, cu_seqlens=None)
    h    = scan_step(state, x, log_alpha)                    # state updated in place
    y, mean, rstd = layernorm_fwd(x, weight=None, bias=None)
    dx, dweight, dbias = layernorm_bwd(dy, x, mean, rstd, weight=None)
    state_move(state, src, dst)                              # state updated in place

And the other token mixer of hybrid stacks, attention with a sliding window and
sinks, with its resident ring cache in the inputs' type or in 8 bits.

    o, lse = swa_fwd(q, k, v, window, sinks=0, cu_seqlens=None, cu_seqlens_k=None)
    dq, dk, dv = swa_bwd(d_o, q, k, v, o, lse, window, sinks=0, cu_seqlens=None, cu_seqlens_k=None)
    o    = swa_step(cache, q, k, v, lengths, sinks=0, scales=None, slots=None)   # cache updated in place
    cache_write(cache, k, v, lengths=None, sinks=0, scales=None, slots=None, cu_seqlens=None)
    k, v = cache_read(cache, lengths, sinks=0, scales=None, slots=None, cu_seqlens=None)
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

__all__ = ["GdnError", "chunk_fwd", "chunk_fwd_noalloc", "decode_step", "chunk_bwd", "chunk_fwd_workspace_size",
           "chunk_bwd_workspace_size", "chunk_fwd_check", "scan_fwd", "scan_bwd", "scan_step", "scan_workspace_size",
           "layernorm_fwd", "layernorm_bwd", "layernorm_bwd_workspace_size", "state_move", "state_move_check",
           "swa_fwd", "swa_bwd", "swa_step", "swa_fwd_workspace_size", "swa_bwd_workspace_size", "cache_write",
           "cache_read", "cache_check", "load", "lib_path", "profile", "CHUNK"]

HERE = os.path.dirname(os.path.abspath(__file__))
CHUNK = 64

GDN_FP32, GDN_BF16, GDN_FP16, GDN_E4M3 = 0, 1, 2, 3
GDN_QK_L2NORM = 1
NOALLOC_SCRATCH_BYTES = 64 << 20   # GDN_NOALLOC_SCRATCH_BYTES in gdn.h
_DT = {torch.float32: GDN_FP32, torch.bfloat16: GDN_BF16, torch.float16: GDN_FP16}
_STATUS = {0: "GDN_OK", 1: "GDN_ERR_NULL", 2: "GDN_ERR_SHAPE", 3: "GDN_ERR_DTYPE", 4: "GDN_ERR_ALIGN",
           5: "GDN_ERR_UNSUPPORTED", 6: "GDN_ERR_WORKSPACE", 7: "GDN_ERR_HIP", 8: "GDN_ERR_ALIAS",
           9: "GDN_ERR_DEVICE_INPUT"}


class GdnError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        self.status_name = _STATUS.get(status, f"status {status}")
        super().__init__(f"{self.status_name}: {message}")


class ChunkDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("chunk", ctypes.c_int32), ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class SwaDesc(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in ("batch", "seqlen", "keylen", "heads", "kv_heads", "dim", "num_seqs",
                                                    "window", "sinks", "dtype")] \
        + [("scale", ctypes.c_float), ("flags", ctypes.c_int32)]


class CacheDesc(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in ("slots", "kv_heads", "window", "sinks", "dim", "dtype")]


class ScanDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32), ("channels", ctypes.c_int32),
                ("num_seqs", ctypes.c_int32), ("in_dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


def lib_path() -> str:
    return os.environ.get("GDN_LIB", os.path.join(HERE, "libgdn.so"))


_lib = None


def load():
    """Load libgdn.so (raises if it is absent: build it with
    `python -m gated_delta_rule_24_amd.build`)."""
    global _lib
    if _lib is not None:
        return _lib
    p = lib_path()
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is not built; run `python -m gated_delta_rule_24_amd.build`")
    lib = ctypes.CDLL(p)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.gdn_abi_version.restype = ctypes.c_int
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_status_string.argtypes = [ctypes.c_int]
    lib.gdn_last_error_message.restype = ctypes.c_char_p
    lib.gdn_chunk_fwd_workspace_size.restype = ctypes.c_int
    lib.gdn_chunk_fwd_workspace_size.argtypes = [ctypes.POINTER(ChunkDesc), ctypes.POINTER(sz)]
    lib.gdn_chunk_fwd.restype = ctypes.c_int
    lib.gdn_chunk_fwd.argtypes = [ctypes.POINTER(ChunkDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gdn_chunk_bwd_workspace_size.restype = ctypes.c_int
    lib.gdn_chunk_bwd_workspace_size.argtypes = [ctypes.POINTER(ChunkDesc), ctypes.POINTER(sz)]
    lib.gdn_chunk_bwd.restype = ctypes.c_int
    lib.gdn_chunk_bwd.argtypes = [ctypes.POINTER(ChunkDesc)] + [vp] * 16 + [sz, vp]
    lib.gdn_chunk_fwd_noalloc.restype = ctypes.c_int
    lib.gdn_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(ChunkDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.gdn_chunk_fwd_check.restype = ctypes.c_int
    lib.gdn_chunk_fwd_check.argtypes = [vp, vp, ctypes.POINTER(i32)]
    lib.gdn_decode_step.restype = ctypes.c_int
    lib.gdn_decode_step.argtypes = [i32, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]
    i64, scan_desc, swa_desc = ctypes.c_int64, ctypes.POINTER(ScanDesc), ctypes.POINTER(SwaDesc)
    cache_desc = ctypes.POINTER(CacheDesc)
    for name, args in {
            "gdn_scan_workspace_size": [scan_desc, ctypes.POINTER(sz)],
            "gdn_scan_fwd": [scan_desc] + [vp] * 7 + [sz, vp],
            "gdn_scan_bwd": [scan_desc] + [vp] * 10 + [sz, vp],
            "gdn_scan_step": [i32] * 5 + [vp] * 5,
            "gdn_layernorm_fwd": [i64, i32, i32, i32, ctypes.c_float] + [vp] * 7,
            "gdn_layernorm_bwd_workspace_size": [i64, i32, ctypes.POINTER(sz)],
            "gdn_layernorm_bwd": [i64, i32, i32, i32] + [vp] * 9 + [sz, vp],
            "gdn_state_move": [i32, i32, i64, i32] + [vp] * 5,
            "gdn_swa_fwd_workspace_size": [swa_desc, ctypes.POINTER(sz)],
            "gdn_swa_bwd_workspace_size": [swa_desc, ctypes.POINTER(sz)],
            "gdn_swa_fwd": [swa_desc] + [vp] * 8 + [sz, vp],
            "gdn_swa_bwd": [swa_desc] + [vp] * 12 + [sz, vp],
            "gdn_swa_step_workspace_size": [cache_desc, i32, i32, ctypes.POINTER(sz)],
            "gdn_swa_step": [cache_desc, i32, i32, i32, ctypes.c_float] + [vp] * 9 + [sz, vp, vp],
            "gdn_cache_write": [cache_desc, i32, i32, i32] + [vp] * 9,
            "gdn_cache_read": [cache_desc, i32, i32, i32] + [vp] * 9}.items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = ctypes.c_int, args
    lib.gdn_profile_enable.restype = ctypes.c_int
    lib.gdn_profile_enable.argtypes = [i32]
    lib.gdn_profile_count.restype = ctypes.c_int
    lib.gdn_profile_count.argtypes = [ctypes.POINTER(i32)]
    lib.gdn_profile_read.restype = ctypes.c_int
    lib.gdn_profile_read.argtypes = [i32, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_int64),
                                     ctypes.POINTER(ctypes.c_double)]
    if lib.gdn_abi_version() != 5:
        raise RuntimeError(f"{p}: unexpected ABI version {lib.gdn_abi_version()}")
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise GdnError(status, load().gdn_last_error_message().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, name, dtypes, device, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _desc(B, T, H, dk, dv, N, in_dt, out_dt, chunk=CHUNK, flags=0):
    return ChunkDesc(B, T, H, dk, dv, N, chunk, in_dt, out_dt, flags)


def chunk_fwd_workspace_size(B, T, H, dk, dv, num_seqs, in_dtype=torch.bfloat16, out_dtype=torch.float32,
                             chunk=CHUNK) -> int:
    d = _desc(B, T, H, dk, dv, num_seqs, _DT[in_dtype], _DT[out_dtype], chunk)
    n = ctypes.c_size_t(0)
    _check(load().gdn_chunk_fwd_workspace_size(ctypes.byref(d), ctypes.byref(n)))
    return int(n.value)


def _chunk_call_args(q, k, v, log_alpha, beta, init_state, cu_seqlens, out_dtype, o, final_state, chunk,
                     qk_l2norm):
    """Checks and marshals the arguments shared by chunk_fwd and chunk_fwd_noalloc.
    Returns (descriptor, o, final_state or None, the leading pointer arguments)."""
    load()
    dev = q.device
    dts = (torch.float32, torch.bfloat16, torch.float16)
    _need(q, "q", dts, dev, 4)
    B, T, H, dk = q.shape
    _need(k, "k", (q.dtype,), dev, 4)
    _need(v, "v", (q.dtype,), dev, 4)
    dv = v.shape[3]
    if tuple(k.shape) != (B, T, H, dk) or tuple(v.shape[:3]) != (B, T, H):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    _need(log_alpha, "log_alpha", (torch.float32,), dev, 3)
    _need(beta, "beta", (torch.float32,), dev, 3)
    if tuple(log_alpha.shape) != (B, T, H) or tuple(beta.shape) != (B, T, H):
        raise ValueError("log_alpha and beta must be [B, T, H]")
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", (torch.int32,), dev, 1)
        N = cu_seqlens.shape[0] - 1
    else:
        N = B
    if init_state is not None:
        _need(init_state, "init_state", (torch.float32,), dev, 4)
        if tuple(init_state.shape) != (N, H, dv, dk):
            raise ValueError(f"init_state must be {(N, H, dv, dk)}, got {tuple(init_state.shape)}")
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=out_dtype, device=dev)
    else:
        _need(o, "o", (torch.float32, torch.bfloat16, torch.float16), dev, 4)
        if tuple(o.shape) != (B, T, H, dv):
            raise ValueError("o has the wrong shape")
    if final_state is True:
        final_state = torch.empty((N, H, dv, dk), dtype=torch.float32, device=dev)
    elif final_state is False:
        final_state = None
    elif final_state is not None:
        _need(final_state, "final_state", (torch.float32,), dev, 4)
        if tuple(final_state.shape) != (N, H, dv, dk):
            raise ValueError("final_state has the wrong shape")
    desc = _desc(B, T, H, dk, dv, N, _DT[q.dtype], _DT[o.dtype], chunk, GDN_QK_L2NORM if qk_l2norm else 0)
    ptrs = [_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(init_state), _ptr(cu_seqlens), _ptr(o),
            _ptr(final_state)]
    return desc, o, final_state, ptrs


def chunk_fwd(q, k, v, log_alpha, beta, init_state=None, cu_seqlens=None, *, out_dtype=torch.float32,
              o=None, final_state=True, workspace=None, chunk=CHUNK, qk_l2norm=False):
    """Chunkwise-parallel prefill.

    q, k [B,T,H,dk], v [B,T,H,dv] (fp32/bf16/fp16, same dtype);
    log_alpha, beta [B,T,H] fp32; init_state [N,H,dv,dk] fp32 or None;
    cu_seqlens int32 [N+1] (packed batch, B == 1) or None.
    final_state: True (allocate), False/None (not returned) or a tensor to
    write (it may be init_state itself).  qk_l2norm: normalise q and k per
    (token, head) inside the kernels.  Returns (o, final_state or None).
    """
    lib = load()
    desc, o, final_state, ptrs = _chunk_call_args(q, k, v, log_alpha, beta, init_state, cu_seqlens, out_dtype, o,
                                                  final_state, chunk, qk_l2norm)
    need = ctypes.c_size_t(0)
    _check(lib.gdn_chunk_fwd_workspace_size(ctypes.byref(desc), ctypes.byref(need)))
    if workspace is None:
        workspace = torch.empty(int(need.value), dtype=torch.uint8, device=q.device)
    _check(lib.gdn_chunk_fwd(ctypes.byref(desc), *ptrs, _ptr(workspace),
                             ctypes.c_size_t(workspace.numel() * workspace.element_size()), _stream(q.device)))
    return o, final_state


def chunk_fwd_noalloc(q, k, v, log_alpha, beta, init_state=None, cu_seqlens=None, *, out_dtype=torch.float32,
                      o=None, final_state=True, chunk=CHUNK, qk_l2norm=False):
    """chunk_fwd through gdn_chunk_fwd_noalloc: the library's per-GPU scratch
    array (NOALLOC_SCRATCH_BYTES) stands in for the workspace, so with `o` and
    `final_state` passed in (or final_state=False) nothing is allocated.
    Calls that overlap in time on one GPU race on the scratch array."""
    lib = load()
    desc, o, final_state, ptrs = _chunk_call_args(q, k, v, log_alpha, beta, init_state, cu_seqlens, out_dtype, o,
                                                  final_state, chunk, qk_l2norm)
    _check(lib.gdn_chunk_fwd_noalloc(ctypes.byref(desc), *ptrs, _stream(q.device)))
    return o, final_state


def chunk_bwd_workspace_size(B, T, H, dk, dv, num_seqs, in_dtype=torch.bfloat16, chunk=CHUNK,
                             qk_l2norm=False) -> int:
    d = _desc(B, T, H, dk, dv, num_seqs, _DT[in_dtype], GDN_FP32, chunk, GDN_QK_L2NORM if qk_l2norm else 0)
    n = ctypes.c_size_t(0)
    _check(load().gdn_chunk_bwd_workspace_size(ctypes.byref(d), ctypes.byref(n)))
    return int(n.value)


def chunk_bwd(q, k, v, log_alpha, beta, d_o, init_state=None, d_final=None, cu_seqlens=None, *,
              d_init=True, workspace=None, chunk=CHUNK, qk_l2norm=False):
    """Gradients of chunk_fwd's o and final state with respect to its inputs.

    q, k, v, log_alpha, beta, init_state, cu_seqlens, qk_l2norm as for
    chunk_fwd; d_o [B,T,H,dv] fp32; d_final [N,H,dv,dk] fp32 or None (zeros).
    d_init: True (allocate and return dL/d init_state) or False.
    Returns (dq, dk, dv, dlog_alpha, dbeta, d_init or None), all fp32.
    """
    lib = load()
    dev = q.device
    dts = (torch.float32, torch.bfloat16, torch.float16)
    _need(q, "q", dts, dev, 4)
    B, T, H, dk = q.shape
    _need(k, "k", (q.dtype,), dev, 4)
    _need(v, "v", (q.dtype,), dev, 4)
    dv = v.shape[3]
    if tuple(k.shape) != (B, T, H, dk) or tuple(v.shape[:3]) != (B, T, H):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    _need(log_alpha, "log_alpha", (torch.float32,), dev, 3)
    _need(beta, "beta", (torch.float32,), dev, 3)
    if tuple(log_alpha.shape) != (B, T, H) or tuple(beta.shape) != (B, T, H):
        raise ValueError("log_alpha and beta must be [B, T, H]")
    _need(d_o, "d_o", (torch.float32,), dev, 4)
    if tuple(d_o.shape) != (B, T, H, dv):
        raise ValueError(f"d_o must be {(B, T, H, dv)}, got {tuple(d_o.shape)}")
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", (torch.int32,), dev, 1)
        N = cu_seqlens.shape[0] - 1
    else:
        N = B
    for name, t in (("init_state", init_state), ("d_final", d_final)):
        if t is not None:
            _need(t, name, (torch.float32,), dev, 4)
            if tuple(t.shape) != (N, H, dv, dk):
                raise ValueError(f"{name} must be {(N, H, dv, dk)}, got {tuple(t.shape)}")
    f32 = dict(dtype=torch.float32, device=dev)
    dq, dk_, dv_ = torch.empty((B, T, H, dk), **f32), torch.empty((B, T, H, dk), **f32), torch.empty((B, T, H, dv), **f32)
    dla, db = torch.empty((B, T, H), **f32), torch.empty((B, T, H), **f32)
    di = torch.empty((N, H, dv, dk), **f32) if d_init else None
    desc = _desc(B, T, H, dk, dv, N, _DT[q.dtype], _DT[torch.float32], chunk, GDN_QK_L2NORM if qk_l2norm else 0)
    need = ctypes.c_size_t(0)
    _check(lib.gdn_chunk_bwd_workspace_size(ctypes.byref(desc), ctypes.byref(need)))
    if workspace is None:
        workspace = torch.empty(int(need.value), dtype=torch.uint8, device=dev)
    _check(lib.gdn_chunk_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                             _ptr(init_state), _ptr(cu_seqlens), _ptr(d_o), _ptr(d_final), _ptr(dq), _ptr(dk_),
                             _ptr(dv_), _ptr(dla), _ptr(db), _ptr(di), _ptr(workspace),
                             ctypes.c_size_t(workspace.numel() * workspace.element_size()), _stream(dev)))
    return dq, dk_, dv_, dla, db, di


def chunk_fwd_check(workspace: torch.Tensor) -> int:
    """Synchronise and return the device-side cu_seqlens check code of the last
    chunk_fwd that used `workspace` (0 = valid)."""
    code = ctypes.c_int32(0)
    st = load().gdn_chunk_fwd_check(_ptr(workspace), _stream(workspace.device), ctypes.byref(code))
    if st not in (0, 9):
        _check(st)
    return int(code.value)


def decode_step(state, q, k, v, log_alpha, beta, *, out_dtype=torch.float32, o=None, qk_l2norm=False):
    """One decode step, in place on `state` [N,H,dv,dk] fp32.
    q, k [N,H,dk], v [N,H,dv]; log_alpha, beta [N,H] fp32.  qk_l2norm:
    normalise q and k inside the kernel.  Returns o [N,H,dv]."""
    lib = load()
    dev = state.device
    _need(state, "state", (torch.float32,), dev, 4)
    N, H, dv, dk = state.shape
    dts = (torch.float32, torch.bfloat16, torch.float16)
    _need(q, "q", dts, dev, 3)
    _need(k, "k", (q.dtype,), dev, 3)
    _need(v, "v", (q.dtype,), dev, 3)
    if tuple(q.shape) != (N, H, dk) or tuple(k.shape) != (N, H, dk) or tuple(v.shape) != (N, H, dv):
        raise ValueError("q, k must be [N,H,dk] and v [N,H,dv] matching state")
    _need(log_alpha, "log_alpha", (torch.float32,), dev, 2)
    _need(beta, "beta", (torch.float32,), dev, 2)
    if tuple(log_alpha.shape) != (N, H) or tuple(beta.shape) != (N, H):
        raise ValueError("log_alpha and beta must be [N, H]")
    if o is None:
        o = torch.empty((N, H, dv), dtype=out_dtype, device=dev)
    else:
        _need(o, "o", dts, dev, 3)
    _check(lib.gdn_decode_step(N, H, dk, dv, _DT[q.dtype], _DT[o.dtype], GDN_QK_L2NORM if qk_l2norm else 0,
                               _ptr(state), _ptr(q), _ptr(k), _ptr(v),
                               _ptr(log_alpha), _ptr(beta), _ptr(o), _stream(dev)))
    return o


# ---- gated linear recurrence, layer norm, state moves ------------------------------

_FLOATS = tuple(_DT)


def _code(dtype):
    if dtype not in _DT:
        raise ValueError(f"dtype {dtype} is not one of {_FLOATS}")
    return _DT[dtype]


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _call(name, device, *args):
    """One library call with `device` current and its current stream as the last argument."""
    index = device.index
    if torch.cuda.current_device() == index:
        status = getattr(_lib or load(), name)(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = getattr(load(), name)(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != 0:
        _check(status)


def _cuda(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, expected a GPU")
    return t.device


def _shaped(t, name, shape, dtypes, device):
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and t.is_contiguous() \
            and t.device == device:
        return
    _need(t, name, dtypes, device, len(shape))
    raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")


def _workspace(workspace, size, device):
    if workspace is None:
        return torch.empty(size, dtype=torch.uint8, device=device), size
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {device}")
    return workspace, workspace.numel() * workspace.element_size()


def scan_workspace_size(B, T, D, num_seqs, in_dtype=torch.bfloat16, gate_dtype=torch.float32,
                        out_dtype=torch.float32) -> int:
    return _scan_desc(B, T, D, num_seqs, in_dtype, gate_dtype, out_dtype)[1]


@functools.lru_cache(maxsize=256)
def _scan_desc(B, T, D, N, in_dtype, gate_dtype, out_dtype):
    """Descriptor of these sizes and types, and its workspace size."""
    d = ScanDesc(B, T, D, N, _code(in_dtype), _code(gate_dtype), _code(out_dtype), 0)
    n = ctypes.c_size_t(0)
    _check(load().gdn_scan_workspace_size(ctypes.byref(d), ctypes.byref(n)))
    return d, int(n.value)


def _scan_call(B, T, D, in_dtype, gate_dtype, out_dtype, cu_seqlens, workspace, device):
    """Descriptor, number of sequences and workspace of a scan_fwd or scan_bwd call."""
    if cu_seqlens is None:
        N = B
    else:
        _need(cu_seqlens, "cu_seqlens", (torch.int32,), device, 1)
        N = cu_seqlens.shape[0] - 1
    desc, need = _scan_desc(B, T, D, N, in_dtype, gate_dtype, out_dtype)
    return desc, N, *_workspace(workspace, need, device)


def scan_fwd(x, log_alpha, init_state=None, cu_seqlens=None, *, out_dtype=torch.float32, h=None, final_state=True,
             workspace=None):
    """Gated linear recurrence h_t = exp(log_alpha_t) h_{t-1} + x_t per channel.

    x [B,T,D], log_alpha [B,T,D] (each fp32 or one 16-bit type); init_state
    [N,D] fp32 or None (zeros); cu_seqlens int32 [N+1] (packed batch, B == 1)
    or None.  final_state: True (allocate), False/None (not returned) or a
    tensor to write (it may be init_state itself).  Returns (h [B,T,D],
    final_state [N,D] or None).
    """
    dev = _cuda(x, "x")
    _need(x, "x", _FLOATS, dev, 3)
    B, T, D = shape = tuple(x.shape)
    _shaped(log_alpha, "log_alpha", shape, _FLOATS, dev)
    if h is None:
        h = torch.empty(shape, dtype=out_dtype, device=dev)
    else:
        _shaped(h, "h", shape, _FLOATS, dev)
    desc, N, workspace, size = _scan_call(B, T, D, x.dtype, log_alpha.dtype, h.dtype, cu_seqlens, workspace, dev)
    if init_state is not None:
        _shaped(init_state, "init_state", (N, D), (torch.float32,), dev)
    if final_state is True:
        final_state = torch.empty((N, D), dtype=torch.float32, device=dev)
    elif final_state is False:
        final_state = None
    elif final_state is not None:
        _shaped(final_state, "final_state", (N, D), (torch.float32,), dev)
    _call("gdn_scan_fwd", dev, desc, _addr(x), _addr(log_alpha), _addr(init_state), _addr(cu_seqlens), _addr(h),
          _addr(final_state), _addr(workspace), size)
    return h, final_state


def scan_bwd(log_alpha, h, d_h, init_state=None, d_final=None, cu_seqlens=None, *, dx_dtype=torch.float32,
             d_init=True, workspace=None):
    """Gradients of scan_fwd's h and final state with respect to its inputs.

    log_alpha, init_state, cu_seqlens as for scan_fwd; h is its output; d_h
    [B,T,D] in h's dtype; d_final [N,D] fp32 or None (zeros).  dx_dtype: the
    dtype of x.  d_init: True (allocate and return dL/d init_state) or False.
    Returns (dx in dx_dtype, dlog_alpha in log_alpha's dtype, d_init or None).
    """
    dev = _cuda(h, "h")
    _need(h, "h", _FLOATS, dev, 3)
    B, T, D = shape = tuple(h.shape)
    _shaped(log_alpha, "log_alpha", shape, _FLOATS, dev)
    _shaped(d_h, "d_h", shape, (h.dtype,), dev)
    dx = torch.empty(shape, dtype=dx_dtype, device=dev)
    dla = torch.empty(shape, dtype=log_alpha.dtype, device=dev)
    desc, N, workspace, size = _scan_call(B, T, D, dx_dtype, log_alpha.dtype, h.dtype, cu_seqlens, workspace, dev)
    for name, t in (("init_state", init_state), ("d_final", d_final)):
        if t is not None:
            _shaped(t, name, (N, D), (torch.float32,), dev)
    di = torch.empty((N, D), dtype=torch.float32, device=dev) if d_init else None
    _call("gdn_scan_bwd", dev, desc, _addr(log_alpha), _addr(h), _addr(init_state), _addr(cu_seqlens), _addr(d_h),
          _addr(d_final), _addr(dx), _addr(dla), _addr(di), _addr(workspace), size)
    return dx, dla, di


def scan_step(state, x, log_alpha, *, out_dtype=torch.float32, h=None):
    """One token of the gated linear recurrence, in place on `state` [N,D]
    fp32.  x, log_alpha [N,D].  Returns h [N,D], the new state in out_dtype."""
    dev = _cuda(state, "state")
    _need(state, "state", (torch.float32,), dev, 2)
    shape = tuple(state.shape)
    _shaped(x, "x", shape, _FLOATS, dev)
    _shaped(log_alpha, "log_alpha", shape, _FLOATS, dev)
    if h is None:
        h = torch.empty(shape, dtype=out_dtype, device=dev)
    else:
        _shaped(h, "h", shape, _FLOATS, dev)
    _call("gdn_scan_step", dev, *shape, _DT[x.dtype], _DT[log_alpha.dtype], _code(h.dtype), _addr(state), _addr(x),
          _addr(log_alpha), _addr(h))
    return h


def _rows(x, name):
    dev = _cuda(x, name)
    if x.dim() < 1:
        raise ValueError(f"{name} must have at least one dim")
    if x.dtype not in _FLOATS or not x.is_contiguous():
        _need(x, name, _FLOATS, dev, x.dim())
    D = x.shape[-1]
    return dev, x.numel() // D if D else 0, D


def layernorm_fwd(x, weight=None, bias=None, *, eps=1e-5, out_dtype=torch.float32, y=None, stats=True):
    """Layer norm over the last dimension of x [..., D] (fp32/bf16/fp16);
    weight, bias [D] fp32 or None (ones, zeros).  Returns (y [..., D], mean
    [...], rstd [...]), the statistics fp32, or None both without `stats`."""
    dev, rows, D = _rows(x, "x")
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _shaped(t, name, (D,), (torch.float32,), dev)
    if y is None:
        y = torch.empty(x.shape, dtype=out_dtype, device=dev)
    else:
        _shaped(y, "y", tuple(x.shape), _FLOATS, dev)
    mean = rstd = None
    if stats:
        mean, rstd = (torch.empty(x.shape[:-1], dtype=torch.float32, device=dev) for _ in range(2))
    _call("gdn_layernorm_fwd", dev, rows, D, _DT[x.dtype], _code(y.dtype), eps, _addr(x), _addr(weight), _addr(bias),
          _addr(y), _addr(mean), _addr(rstd))
    return y, mean, rstd


@functools.lru_cache(maxsize=256)
def layernorm_bwd_workspace_size(rows, dim) -> int:
    n = ctypes.c_size_t(0)
    _check(load().gdn_layernorm_bwd_workspace_size(rows, dim, ctypes.byref(n)))
    return int(n.value)


def layernorm_bwd(dy, x, mean, rstd, weight=None, *, dweight=True, dbias=True, workspace=None):
    """Gradients of layernorm_fwd: dy [..., D] in y's dtype; x, weight as given
    to it; mean, rstd [...] fp32 as it returned them.  Returns (dx in x's
    dtype, dweight [D] fp32 or None, dbias [D] fp32 or None)."""
    dev, rows, D = _rows(x, "x")
    _shaped(dy, "dy", tuple(x.shape), _FLOATS, dev)
    for name, t in (("mean", mean), ("rstd", rstd)):
        _shaped(t, name, tuple(x.shape[:-1]), (torch.float32,), dev)
    if weight is not None:
        _shaped(weight, "weight", (D,), (torch.float32,), dev)
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    dw, db = (torch.empty((D,), dtype=torch.float32, device=dev) if want else None for want in (dweight, dbias))
    size = 0
    if dweight or dbias:
        workspace, size = _workspace(workspace, layernorm_bwd_workspace_size(rows, D), dev)
    _call("gdn_layernorm_bwd", dev, rows, D, _DT[x.dtype], _DT[dy.dtype], _addr(dy), _addr(x), _addr(mean),
          _addr(rstd), _addr(weight), _addr(dx), _addr(dw), _addr(db), _addr(workspace), size)
    return dx, dw, db


def state_move(state, src, dst, *, layers=False, status=None):
    """Moves of resident states, in place: slot dst[m] of `state` gets what slot
    src[m] held before the call, zeros where src[m] is -1.  `state` [N, ...]
    is one layer's resident states (decode_step's, scan_step's), or with
    `layers` [L, N, ...] several layers' that all move alike.  src, dst int32
    [M] on the device, dst without repetition; bad indices leave the state as
    it was, and state_move_check tells of them if `status` (int32 [2] on the
    device) was given.  Forks, compacts, reorders and frees.  Returns state."""
    dev = _cuda(state, "state")
    lead = 2 if layers else 1
    if state.dim() < lead + 1:
        raise ValueError(f"state must have more than {lead} dims, got shape {tuple(state.shape)}")
    if not state.is_contiguous():
        raise ValueError("state must be contiguous")
    _need(src, "src", (torch.int32,), dev, 1)
    _shaped(dst, "dst", tuple(src.shape), (torch.int32,), dev)
    if status is not None:
        _shaped(status, "status", (2,), (torch.int32,), dev)
    _call("gdn_state_move", dev, state.shape[0] if layers else 1, state.shape[lead - 1],
          state.shape[lead:].numel() * state.element_size(), src.shape[0], _addr(state), _addr(src), _addr(dst),
          _addr(status))
    return state


def state_move_check(status: torch.Tensor) -> int:
    """Synchronise and return the code that state_move left in `status`: 0, or
    1 for a source out of range, 2 for a destination out of range, 3 for a
    destination given twice."""
    return chunk_fwd_check(status)


# ---- windowed attention and its resident cache --------------------------------------

_INT32 = 2 ** 31 - 1


def _scale(d, scale):
    """1 / sqrt(d) for None; heads of no elements are the library's to refuse."""
    return scale if scale is not None else max(d, 1) ** -0.5


@functools.lru_cache(maxsize=256)
def _swa_desc(which, *fields):
    """Descriptor of these sizes and types, and the workspace size of gdn_swa_<which>."""
    d = SwaDesc(*fields, 0)
    n = ctypes.c_size_t(0)
    _check(getattr(load(), f"gdn_swa_{which}_workspace_size")(ctypes.byref(d), ctypes.byref(n)))
    return d, int(n.value)


def _swa_call(which, q, k, v, window, sinks, cu_seqlens, cu_seqlens_k, scale):
    """Device, q's shape, key offsets, descriptor and workspace size of a swa_fwd or swa_bwd call."""
    dev, types = _cuda(q, "q"), (q.dtype,)
    if q.dtype not in _FLOATS or q.dim() != 4 or not q.is_contiguous():
        _need(q, "q", _FLOATS, dev, 4)
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        _need(k, "k", types, dev, 4)
    B, T, H, d = shape = q.shape
    Tk, KV = k.shape[1], k.shape[2]
    kshape = (B, Tk, KV, d)
    _shaped(k, "k", kshape, types, dev)
    _shaped(v, "v", kshape, types, dev)
    N = B
    if cu_seqlens is None:
        if cu_seqlens_k is not None:
            raise ValueError("cu_seqlens_k needs cu_seqlens")
    else:
        _need(cu_seqlens, "cu_seqlens", (torch.int32,), dev, 1)
        N = cu_seqlens.shape[0] - 1
        if cu_seqlens_k is None:
            if Tk != T:
                raise ValueError(f"k has {Tk} tokens and q {T}: cu_seqlens_k is needed")
            cu_seqlens_k = cu_seqlens
        else:
            _shaped(cu_seqlens_k, "cu_seqlens_k", (N + 1,), (torch.int32,), dev)
    if not -_INT32 <= sinks <= _INT32:
        raise ValueError(f"sinks {sinks} is no 32-bit number")
    desc, need = _swa_desc(which, B, T, Tk, H, KV, d, N, max(min(window, _INT32), -_INT32), sinks, _DT[q.dtype],
                           _scale(d, scale))
    return dev, shape, cu_seqlens_k, desc, need


def swa_fwd_workspace_size(B, T, Tk, H, KV, d, num_seqs, window, sinks=0, dtype=torch.bfloat16) -> int:
    return _swa_desc("fwd", B, T, Tk, H, KV, d, num_seqs, window, sinks, _code(dtype), 1.0)[1]


def swa_fwd(q, k, v, window, sinks=0, cu_seqlens=None, cu_seqlens_k=None, *, scale=None, o=None, lse=True,
            workspace=None):
    """Attention with a sliding window and sinks: a query sees the keys at most
    window - 1 positions back, and its sequence's first `sinks` keys.

    q [B,T,H,d], k, v [B,Tk,KV,d] (fp32/bf16/fp16, one dtype; H a multiple of
    KV); a row's queries are its last T positions.  cu_seqlens int32 [N+1]
    (packed batch, B == 1) or None, cu_seqlens_k the keys' (None: the same).
    scale: None for 1 / sqrt(d).  Returns (o [B,T,H,d], lse [B,T,H] fp32 or
    None without `lse`).
    """
    dev, shape, cu_k, desc, size = _swa_call("fwd", q, k, v, window, sinks, cu_seqlens, cu_seqlens_k, scale)
    if o is None:
        o = torch.empty_like(q)
    else:
        _shaped(o, "o", shape, (q.dtype,), dev)
    lse = torch.empty(shape[:3], dtype=torch.float32, device=dev) if lse else None
    if cu_seqlens is None:
        workspace, size = None, 0
    else:
        workspace, size = _workspace(workspace, size, dev)
    _call("gdn_swa_fwd", dev, desc, _addr(q), _addr(k), _addr(v), _addr(cu_seqlens), _addr(cu_k), _addr(o),
          _addr(lse), _addr(workspace), size)
    return o, lse


def swa_bwd_workspace_size(B, T, Tk, H, KV, d, num_seqs, window, sinks=0, dtype=torch.bfloat16) -> int:
    return _swa_desc("bwd", B, T, Tk, H, KV, d, num_seqs, window, sinks, _code(dtype), 1.0)[1]


def swa_bwd(d_o, q, k, v, o, lse, window, sinks=0, cu_seqlens=None, cu_seqlens_k=None, *, scale=None, workspace=None):
    """Gradients of swa_fwd's o with respect to q, k and v.

    q, k, v, window, sinks, cu_seqlens, cu_seqlens_k, scale as for swa_fwd; o
    and lse as it returned them; d_o [B,T,H,d] in their dtype.  Returns (dq, dk,
    dv) in that dtype.
    """
    dev, shape, cu_k, desc, size = _swa_call("bwd", q, k, v, window, sinks, cu_seqlens, cu_seqlens_k, scale)
    _shaped(d_o, "d_o", shape, (q.dtype,), dev)
    _shaped(o, "o", shape, (q.dtype,), dev)
    _shaped(lse, "lse", shape[:3], (torch.float32,), dev)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(k)
    workspace, size = _workspace(workspace, size, dev)
    _call("gdn_swa_bwd", dev, desc, _addr(d_o), _addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), _addr(cu_seqlens),
          _addr(cu_k), _addr(dq), _addr(dk), _addr(dv), _addr(workspace), size)
    return dq, dk, dv


_CACHE_DT = {**_DT, torch.float8_e4m3fn: GDN_E4M3}


@functools.lru_cache(maxsize=256)
def _cache_desc(shape, dtype, sinks):
    window = shape[3] - sinks
    if shape[0] != 2 or sinks < 0 or window < 1:
        raise ValueError(f"cache must be [2, slots, kv heads, {sinks} sinks + window, d], got {shape}")
    return CacheDesc(*shape[1:3], window, sinks, shape[4], _CACHE_DT[dtype])


def _cache_call(cache, scales, slots, lengths, sinks):
    """Device and descriptor of a call on `cache`."""
    dev = _cuda(cache, "cache")
    if cache.dtype not in _CACHE_DT or cache.dim() != 5 or not cache.is_contiguous():
        _need(cache, "cache", tuple(_CACHE_DT), dev, 5)
    if scales is not None:
        _shaped(scales, "scales", tuple(cache.shape[:4]), (torch.float32,), dev)
    if lengths is not None:
        _need(lengths, "lengths", (torch.int32,), dev, 1)
        if slots is not None:
            _shaped(slots, "slots", tuple(lengths.shape), (torch.int32,), dev)
    elif slots is not None:
        _need(slots, "slots", (torch.int32,), dev, 1)
    return dev, _cache_desc(tuple(cache.shape), cache.dtype, sinks)


def _cache_tokens(desc, k, v, lengths, slots, cu_seqlens, status, dev):
    """Number of sequences and tokens of a cache_write or cache_read call."""
    _need(k, "k", _FLOATS, dev, 4)
    B, T, KV, d = shape = tuple(k.shape)
    if (KV, d) != (desc.kv_heads, desc.dim):
        raise ValueError(f"k must be [.., {desc.kv_heads}, {desc.dim}], got {shape}")
    _shaped(v, "v", shape, (k.dtype,), dev)
    if cu_seqlens is None:
        N = B
    else:
        _need(cu_seqlens, "cu_seqlens", (torch.int32,), dev, 1)
        if B != 1:
            raise ValueError(f"cu_seqlens needs one row of tokens, got {B}")
        N = cu_seqlens.shape[0] - 1
    for name, t in (("lengths", lengths), ("slots", slots)):
        if t is not None and t.shape[0] != N:
            raise ValueError(f"{name} must have {N} entries, got {t.shape[0]}")
    if status is not None:
        _shaped(status, "status", (2,), (torch.int32,), dev)
    return N, B * T


def cache_write(cache, k, v, lengths=None, sinks=0, scales=None, slots=None, cu_seqlens=None, *, status=None):
    """Tokens into the resident cache of windowed attention, in place.

    cache [2, slots, KV, sinks + window, d] (fp32/bf16/fp16, k and v's dtype; or
    float8_e4m3fn with scales [2, slots, KV, sinks + window] fp32): the sinks'
    rows, then a ring.  k, v [B,T,KV,d]: T tokens for each of B sequences, or a
    packed batch with cu_seqlens int32 [N+1].  lengths int32 [N]: tokens that
    each sequence has already (None: 0); not changed.  slots int32 [N]: where
    each sequence is (None: in order), -1 to leave it out.  Bad indices leave
    the cache as it was, and cache_check tells of them if `status` (int32 [2] on
    the device) was given.  Returns cache.
    """
    dev, desc = _cache_call(cache, scales, slots, lengths, sinks)
    N, T = _cache_tokens(desc, k, v, lengths, slots, cu_seqlens, status, dev)
    _call("gdn_cache_write", dev, desc, N, T, _DT[k.dtype], _addr(k), _addr(v), _addr(cu_seqlens), _addr(lengths),
          _addr(slots), _addr(cache), _addr(scales), _addr(status))
    return cache


def cache_read(cache, lengths, sinks=0, scales=None, slots=None, cu_seqlens=None, *, out_dtype=None, k=None, v=None,
               status=None):
    """What the cache holds of each sequence, in the order of positions: its
    first `sinks` tokens and its last `window`, as many as it has.

    cache, lengths, sinks, scales, slots as for cache_write.  k, v: where the
    rows go, [N,R,KV,d] or with cu_seqlens [1,T,KV,d], each sequence's from its
    part's beginning on; rows behind them are left as they are.  Without them
    they are allocated with sinks + window rows a sequence (out_dtype: None for
    the cache's own, bf16 for an 8-bit one).  Returns (k, v).
    """
    dev, desc = _cache_call(cache, scales, slots, lengths, sinks)
    if lengths is None:
        raise ValueError("lengths is needed")
    if k is None or v is None:
        if k is not None or v is not None or cu_seqlens is not None:
            raise ValueError("k and v go together, and with cu_seqlens both are needed")
        if out_dtype is None:
            out_dtype = torch.bfloat16 if desc.dtype == GDN_E4M3 else cache.dtype
        k, v = (torch.empty((lengths.shape[0], cache.shape[3], *(cache.shape[i] for i in (2, 4))), dtype=out_dtype,
                            device=dev) for _ in range(2))
    N, T = _cache_tokens(desc, k, v, lengths, slots, cu_seqlens, status, dev)
    _call("gdn_cache_read", dev, desc, N, T, _DT[k.dtype], _addr(cache), _addr(scales), _addr(lengths), _addr(slots),
          _addr(cu_seqlens), _addr(k), _addr(v), _addr(status))
    return k, v


@functools.lru_cache(maxsize=256)
def _step_workspace(shape, dtype, sinks, N, H) -> int:
    n = ctypes.c_size_t(0)
    _check(load().gdn_swa_step_workspace_size(ctypes.byref(_cache_desc(shape, dtype, sinks)), N, H, ctypes.byref(n)))
    return int(n.value)


def swa_step(cache, q, k, v, lengths, sinks=0, scales=None, slots=None, *, scale=None, o=None, workspace=None,
             status=None):
    """One token of windowed attention for N resident sequences: k, v [N,KV,d]
    go into the cache (in place) at position lengths[n], and q [N,H,d] attends
    to what it then holds.  cache, lengths, sinks, scales, slots as for
    cache_write; scale: None for 1 / sqrt(d).  lengths is not changed: add one
    when all layers have run.  A sequence with slot -1 is left out, its o is
    zeros.  Returns o [N,H,d]."""
    dev, desc = _cache_call(cache, scales, slots, lengths, sinks)
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.dtype not in _FLOATS or not q.is_contiguous() \
            or q.device != dev:
        _need(q, "q", _FLOATS, dev, 3)
    N, H, d = shape = q.shape
    kshape = (N, desc.kv_heads, d)
    _shaped(k, "k", kshape, (q.dtype,), dev)
    _shaped(v, "v", kshape, (q.dtype,), dev)
    if d != desc.dim:
        raise ValueError(f"q must be [N, H, {desc.dim}], got {shape}")
    if lengths is None or lengths.shape[0] != N:
        raise ValueError(f"lengths must have {N} entries")
    if o is None:
        o = torch.empty_like(q)
    else:
        _shaped(o, "o", shape, (q.dtype,), dev)
    if status is not None:
        _shaped(status, "status", (2,), (torch.int32,), dev)
    need = _step_workspace(tuple(cache.shape), cache.dtype, sinks, N, H)
    size = 0
    if need:
        workspace, size = _workspace(workspace, need, dev)
    else:
        workspace = None
    _call("gdn_swa_step", dev, desc, N, H, _DT[q.dtype], _scale(d, scale), _addr(q), _addr(k),
          _addr(v), _addr(lengths), _addr(slots), _addr(cache), _addr(scales), _addr(o), _addr(workspace), size,
          _addr(status))
    return o


def cache_check(status: torch.Tensor) -> int:
    """Synchronise and return the code that cache_write, cache_read or swa_step
    left in `status`: 0, 1 to 3 for malformed cu_seqlens, 4 for a slot out of
    range, 5 for a slot given twice, 6 for a length out of range, 7 for a
    sequence with more rows to read than room for them."""
    return chunk_fwd_check(status)


class profile:
    """Context manager collecting per-kernel launch times recorded by the
    library (HIP events around each launch, on the launch stream).

        with profile() as p:
            ...
        p.results  ->  {kernel name: (launches, total ms)}
    """

    def __enter__(self):
        _check(load().gdn_profile_enable(1))
        self.results = {}
        return self

    def __exit__(self, *exc):
        lib = load()
        _check(lib.gdn_profile_enable(0))
        n = ctypes.c_int32(0)
        _check(lib.gdn_profile_count(ctypes.byref(n)))
        for i in range(n.value):
            name, cnt, ms = ctypes.c_char_p(), ctypes.c_int64(), ctypes.c_double()
            _check(lib.gdn_profile_read(i, ctypes.byref(name), ctypes.byref(cnt), ctypes.byref(ms)))
            self.results[name.value.decode()] = (int(cnt.value), float(ms.value))
        return False
