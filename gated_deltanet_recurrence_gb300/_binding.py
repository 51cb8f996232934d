"""ctypes binding of libgdn.so: same names as the C ABI (include/gdn.h), torch tensors in.

Argument marshalling only: shapes are read from the tensors, every tensor is checked to sit on
the call's device and to hold at least what the call touches (the library sees bare pointers),
outputs that the caller does not pass are allocated with torch, and the call goes to the library
with the tensors' device current, on that device's current torch stream (or the stream given).  Every computation happens in the library's CUDA kernels; there is no
fallback: if libgdn.so is missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libgdn.so")

GDN_F32, GDN_BF16 = 0, 1
GDN_DECAY_PER_HEAD, GDN_DECAY_PER_KEY_CHANNEL = 0, 1
GDN_CONV_KERNEL = 4
GDN_FORM_AUTO, GDN_FORM_OFF, GDN_FORM_ON = 0, 1, 2
GDN_NORM_RMS, GDN_NORM_L2 = 0, 1
STATUS = {0: "GDN_OK", -1: "GDN_ERR_ARG", -2: "GDN_ERR_DTYPE", -3: "GDN_ERR_CU_SEQLENS",
          -4: "GDN_ERR_WORKSPACE", -5: "GDN_ERR_LAUNCH", -6: "GDN_ERR_TIMEOUT",
          -7: "GDN_ERR_UNSUPPORTED", -8: "GDN_ERR_CUDA"}

_lib = None
_lock = threading.Lock()

_vp, _fp, _ip = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
_i, _f, _sz, _l = ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_long

SIGNATURES = {
    "gdn_chunk_fwd": (_i, [_vp, _vp, _vp, _fp, _fp, _ip, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i,
                           _fp, _fp, _fp, _fp, _fp, _fp, _fp, _f, _vp, _i, _vp, _sz, _vp]),
    "gdn_chunk_fwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "gdn_recurrent_step": (_i, [_vp, _vp, _vp, _fp, _fp, _fp, _i, _i, _i, _i, _i, _i, _i, _f, _i,
                                _fp, _fp, _fp, _fp, _fp, _f, _vp, _i, _vp]),
    "gdn_recurrent_multi_step": (_i, [_vp, _vp, _vp, _fp, _fp, _fp, _i, _ip, _i, _i, _i, _i, _i, _i, _i,
                                      _i, _f, _i, _fp, _fp, _fp, _fp, _fp, _f, _vp, _i, _vp]),
    "gdn_gate_rmsnorm_silu": (_i, [_vp, _i, _fp, _fp, _f, _vp, _i, _l, _i, _vp]),
    "gdn_decay_from_logits": (_i, [_fp, _fp, _fp, _fp, _fp, _fp, _l, _i, _vp]),
    "gdn_chunk_fwd_noalloc": (_i, [_vp, _vp, _vp, _fp, _fp, _ip, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i,
                                   _fp, _fp, _fp, _fp, _fp, _fp, _fp, _f, _vp, _i, _vp]),
    "gdn_chunk_bwd": (_i, [_vp, _vp, _vp, _fp, _fp, _ip, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i, _fp, _vp, _i,
                           _fp, _vp, _vp, _vp, _fp, _fp, _fp, _vp, _sz, _vp]),
    "gdn_chunk_bwd_zero_outside": (_i, [_ip, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _fp, _fp, _vp]),
    "gdn_chunk_bwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "gdn_gate_rmsnorm_silu_bwd": (_i, [_vp, _i, _vp, _i, _fp, _fp, _f, _vp, _fp, _fp, _l, _i, _vp, _sz, _vp]),
    "gdn_gate_groupnorm_silu": (_i, [_vp, _i, _fp, _fp, _fp, _f, _vp, _i, _l, _i, _i, _vp]),
    "gdn_gate_groupnorm_silu_bwd": (_i, [_vp, _i, _vp, _i, _fp, _fp, _fp, _f, _vp, _fp, _fp, _fp, _l, _i, _i,
                                         _vp, _sz, _vp]),
    "gdn_gate_bwd_workspace_size": (_sz, [_l, _i, _i]),
    "gdn_decay_from_logits_bwd": (_i, [_fp, _fp, _fp, _fp, _fp, _fp, _fp, _fp, _fp, _fp, _l, _i, _vp, _sz, _vp]),
    "gdn_decay_bwd_workspace_size": (_sz, [_l, _i]),
    "gdn_short_conv_fwd": (_i, [_vp, _l, _fp, _fp, _ip, _i, _i, _i, _i, _i, _fp, _fp, _vp, _vp]),
    "gdn_short_conv_step": (_i, [_vp, _l, _fp, _fp, _fp, _i, _ip, _i, _i, _i, _i, _i, _vp, _vp]),
    "gdn_short_conv_bwd": (_i, [_vp, _vp, _l, _fp, _fp, _ip, _i, _i, _i, _i, _i, _fp, _fp, _vp, _fp, _fp, _fp, _i,
                                _vp, _sz, _vp]),
    "gdn_short_conv_bwd_workspace_size": (_sz, [_i, _i, _i]),
    "gdn_ssm_chunk_fwd": (_i, [_vp, _l, _vp, _l, _vp, _l, _fp, _fp, _fp, _fp, _ip, _i, _i, _i, _i, _i, _i, _i, _fp,
                               _fp, _vp, _vp, _sz, _vp]),
    "gdn_ssm_chunk_fwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "gdn_ssm_step": (_i, [_vp, _l, _vp, _l, _vp, _l, _fp, _fp, _fp, _fp, _fp, _i, _ip, _i, _i, _i, _i, _i, _i, _i,
                          _vp, _vp]),
    "gdn_ssm_chunk_bwd": (_i, [_vp, _vp, _l, _vp, _l, _vp, _l, _fp, _fp, _fp, _fp, _ip, _i, _i, _i, _i, _i, _i, _i,
                               _fp, _fp, _vp, _vp, _vp, _fp, _fp, _fp, _fp, _fp, _i, _vp, _sz, _vp]),
    "gdn_ssm_chunk_bwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "gdn_qk_norm_rope": (_i, [_vp, _l, _vp, _l, _fp, _ip, _l, _fp, _fp, _i, _f, _i, _i, _i, _i, _i, _i, _i, _vp, _l,
                              _vp, _l, _vp]),
    "gdn_qk_norm_rope_bwd": (_i, [_vp, _vp, _vp, _l, _vp, _l, _fp, _ip, _l, _fp, _fp, _i, _f, _i, _i, _i, _i, _i, _i,
                                  _i, _vp, _l, _vp, _l, _fp, _fp, _vp, _sz, _vp]),
    "gdn_qk_norm_rope_bwd_workspace_size": (_sz, [_i, _i, _i, _i]),
    "gdn_get_device_error": (_i, [_vp, ctypes.POINTER(ctypes.c_int)]),
    "gdn_status_string": (ctypes.c_char_p, [_i]),
    "gdn_selftest_bounded_wait": (_i, [ctypes.c_ulonglong, _vp, _vp]),
    "gdn_set_kernel_forms": (_i, [_i, _i]),
}


class GdnError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} returned {status} ({STATUS.get(status, 'unknown')})")


def lib():
    """Load libgdn.so (building it first if it is missing or older than its sources)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            from . import build as _build
            if _build.is_stale():
                _build.build()
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libgdn.so not found at {LIB_PATH}")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _torch_dt(code: int):
    return torch.bfloat16 if code == GDN_BF16 else torch.float32


def _p(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("all tensors must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("all tensors must be contiguous")
    return t.data_ptr()


def _f32(t, name):
    if t is not None and t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    return t


def _sizes(ref, **tensors):
    """The library sees only pointers, so the binding refuses, before the call, a tensor on another
    device than `ref` or holding fewer elements than the call reads or writes through it.
    Each keyword is name=(tensor or None, elements the call touches)."""
    dev, cuda = ref.get_device(), ref.is_cuda
    for name, (t, numel) in tensors.items():
        if t is None:
            continue
        # the index alone tells CUDA tensors apart; on the host the devices themselves are compared
        if t.get_device() != dev or (not cuda and t.device != ref.device) or t.is_cuda != cuda:
            raise ValueError(f"{name} is on {t.device}, the call runs on {ref.device}")
        if t.numel() < numel:
            raise ValueError(f"{name} holds {t.numel()} elements; the call touches {numel}")


def _pointers(ref, names, tensors, sizes, fp32):
    """The checks of _f32, _sizes and _p in one pass, for calls whose host side is their time: for each of
    `tensors` (None where not given) its name, the elements the call touches, and whether it must be fp32.
    Returns the pointers."""
    dev, dense, out, f32 = ref.get_device(), True, [], torch.float32
    for name, t, numel, only32 in zip(names, tensors, sizes, fp32):
        if t is None:
            out.append(None)
            continue
        if only32 and t.dtype is not f32:
            raise TypeError(f"{name} must be float32")
        if t.get_device() != dev or (dev < 0 and t.device != ref.device):
            raise ValueError(f"{name} is on {t.device}, the call runs on {ref.device}")
        if t.numel() < numel:
            raise ValueError(f"{name} holds {t.numel()} elements; the call touches {numel}")
        if not t.is_contiguous():
            dense = False
        out.append(t.data_ptr())
    if not ref.is_cuda:
        raise ValueError("all tensors must be CUDA tensors")
    if not dense:
        raise ValueError("all tensors must be contiguous")
    return out


def _stream(stream, ref=None):
    if stream is None:
        if ref is not None and ref.is_cuda:  # the raw handle: a Stream object takes some microseconds more
            return torch._C._cuda_getCurrentRawStream(ref.get_device())
        return torch.cuda.current_stream(ref.device if ref is not None else None).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _run(ref, fn, *args):
    """Call library function `fn` with the device of `ref` current: the library launches its
    kernels on the calling thread's current device."""
    dev = ref.get_device()
    if dev == torch._C._cuda_getDevice():
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _check(fn, rc):
    if rc != 0:
        raise GdnError(fn, rc)


def _decay_mode(g, per_head_dims):
    """GDN_DECAY_PER_HEAD when g has the per-head shape, else one decay per key channel."""
    return GDN_DECAY_PER_HEAD if g.dim() == per_head_dims else GDN_DECAY_PER_KEY_CHANNEL


def _conv_f32(conv_weight, conv_state, conv_state_out):
    for name, t in (("conv_weight", conv_weight), ("conv_state", conv_state),
                    ("conv_state_out", conv_state_out)):
        _f32(t, name)


def gdn_chunk_fwd(q, k, v, g, beta, cu_seqlens=None, num_seqs=None, scale=0.0, use_qk_l2norm=True,
                  initial_state=None, final_state=None, output_final_state=True, conv_weight=None,
                  conv_state=None, conv_state_out=None, gate_z=None, norm_weight=None, norm_eps=1e-6,
                  out=None, out_dtype=None, workspace=None, stream=None):
    """Chunked prefill.  q, k [total_T, H_k, d_k]; v [total_T, H, d_v] (H a multiple of H_k);
    beta [total_T, H] fp32; g [total_T, H] fp32, or [total_T, H, d_k] for a decay per key channel;
    cu_seqlens int32 [num_seqs+1] (device) or None with num_seqs equal sequences (default 1).
    conv_weight [2 H_k d_k + H d_v, 4] fuses the short convolution (conv_state: carried input
    history [num_seqs, conv_dim, 3] or None; conv_state_out: filled with the final history if
    given, may be conv_state itself).
    Returns (out, final_state); final_state is allocated unless given or not requested."""
    total_T, H_k, d_k = q.shape
    H, d_v = v.shape[1], v.shape[-1]
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32:
            raise TypeError("cu_seqlens must be int32")
        num_seqs = cu_seqlens.numel() - 1
    elif num_seqs is None:
        num_seqs = 1
    dt = _dt(q)
    if _dt(k) != dt or _dt(v) != dt:
        raise TypeError("q, k, v must share one dtype")
    odt = dt if out_dtype is None else _dt(torch.empty(0, dtype=out_dtype))
    if out is None:
        out = torch.empty((total_T, H, d_v), dtype=_torch_dt(odt), device=q.device)
    else:
        odt = _dt(out)
    if final_state is None and output_final_state:
        final_state = torch.empty((num_seqs, H, d_v, d_k), dtype=torch.float32, device=q.device)
    for name, t in (("g", g), ("beta", beta), ("initial_state", initial_state),
                    ("final_state", final_state), ("gate_z", gate_z), ("norm_weight", norm_weight)):
        _f32(t, name)
    _conv_f32(conv_weight, conv_state, conv_state_out)
    conv_dim = 2 * H_k * d_k + H * d_v
    _sizes(q, k=(k, total_T * H_k * d_k), v=(v, total_T * H * d_v),
           g=(g, total_T * H * (1 if g.dim() == 2 else d_k)), beta=(beta, total_T * H),
           cu_seqlens=(cu_seqlens, num_seqs + 1), initial_state=(initial_state, num_seqs * H * d_v * d_k),
           final_state=(final_state, num_seqs * H * d_v * d_k), gate_z=(gate_z, total_T * H * d_v),
           norm_weight=(norm_weight, d_v), out=(out, total_T * H * d_v),
           conv_weight=(conv_weight, conv_dim * GDN_CONV_KERNEL),
           conv_state=(conv_state, num_seqs * conv_dim * (GDN_CONV_KERNEL - 1)),
           conv_state_out=(conv_state_out, num_seqs * conv_dim * (GDN_CONV_KERNEL - 1)),
           workspace=(workspace, 0))
    L = lib()
    ws_need = L.gdn_chunk_fwd_workspace_size(num_seqs, total_T, H, d_k, d_v, dt)
    if ws_need and workspace is None:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=q.device)
    rc = _run(q, L.gdn_chunk_fwd,
              _p(q), _p(k), _p(v), _p(g), _p(beta), _p(cu_seqlens), num_seqs, total_T, H, H_k, d_k,
              d_v, dt, _decay_mode(g, 2), float(scale), int(bool(use_qk_l2norm)), _p(conv_weight),
              _p(conv_state), _p(conv_state_out), _p(initial_state), _p(final_state), _p(gate_z),
              _p(norm_weight), float(norm_eps), _p(out), odt, _p(workspace),
              workspace.numel() * workspace.element_size() if workspace is not None else 0,
              _stream(stream, q))
    _check("gdn_chunk_fwd", rc)
    return out, final_state


def gdn_chunk_fwd_noalloc(q, k, v, g, beta, cu_seqlens=None, num_seqs=None, scale=0.0,
                          use_qk_l2norm=True, initial_state=None, final_state=None, conv_weight=None,
                          conv_state=None, conv_state_out=None, gate_z=None, norm_weight=None,
                          norm_eps=1e-6, out=None, stream=None):
    """gdn_chunk_fwd with the library's fixed scratch array instead of a workspace; `out` and
    `final_state` must be passed in (this call allocates nothing, here or in the library)."""
    total_T, H_k, d_k = q.shape
    H, d_v = v.shape[1], v.shape[-1]
    if out is None:
        raise ValueError("gdn_chunk_fwd_noalloc needs a preallocated `out`")
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32:
            raise TypeError("cu_seqlens must be int32")
        num_seqs = cu_seqlens.numel() - 1
    elif num_seqs is None:
        num_seqs = 1
    dt = _dt(q)
    for name, t in (("g", g), ("beta", beta), ("initial_state", initial_state),
                    ("final_state", final_state), ("gate_z", gate_z), ("norm_weight", norm_weight)):
        _f32(t, name)
    _conv_f32(conv_weight, conv_state, conv_state_out)
    conv_dim = 2 * H_k * d_k + H * d_v
    _sizes(q, k=(k, total_T * H_k * d_k), v=(v, total_T * H * d_v),
           g=(g, total_T * H * (1 if g.dim() == 2 else d_k)), beta=(beta, total_T * H),
           cu_seqlens=(cu_seqlens, num_seqs + 1), initial_state=(initial_state, num_seqs * H * d_v * d_k),
           final_state=(final_state, num_seqs * H * d_v * d_k), gate_z=(gate_z, total_T * H * d_v),
           norm_weight=(norm_weight, d_v), out=(out, total_T * H * d_v),
           conv_weight=(conv_weight, conv_dim * GDN_CONV_KERNEL),
           conv_state=(conv_state, num_seqs * conv_dim * (GDN_CONV_KERNEL - 1)),
           conv_state_out=(conv_state_out, num_seqs * conv_dim * (GDN_CONV_KERNEL - 1)))
    rc = _run(q, lib().gdn_chunk_fwd_noalloc,
              _p(q), _p(k), _p(v), _p(g), _p(beta), _p(cu_seqlens), num_seqs, total_T, H, H_k, d_k,
              d_v, dt, _decay_mode(g, 2), float(scale), int(bool(use_qk_l2norm)), _p(conv_weight),
              _p(conv_state), _p(conv_state_out), _p(initial_state), _p(final_state), _p(gate_z),
              _p(norm_weight), float(norm_eps), _p(out), _dt(out), _stream(stream, q))
    _check("gdn_chunk_fwd_noalloc", rc)
    return out, final_state


def gdn_recurrent_step(q, k, v, g, beta, state, scale=0.0, use_qk_l2norm=True, conv_weight=None,
                       conv_state=None, conv_state_out=None, gate_z=None, norm_weight=None,
                       norm_eps=1e-6, out=None, out_dtype=None, stream=None):
    """One decode token: q, k [N, H_k, d_k]; v [N, H, d_v]; beta [N, H]; g [N, H] or [N, H, d_k];
    state [N, H, d_v, d_k] fp32 updated in place.  conv_weight [conv_dim, 4] fuses the short
    convolution with history conv_state [N, conv_dim, 3] (None: zeros) and the new history written
    to conv_state_out (may be conv_state when H_k == H).  Returns out [N, H, d_v]."""
    N, H_k, d_k = q.shape
    H, d_v = v.shape[1], v.shape[-1]
    dt = _dt(q)
    odt = dt if out_dtype is None else _dt(torch.empty(0, dtype=out_dtype))
    if out is None:
        out = torch.empty((N, H, d_v), dtype=_torch_dt(odt), device=q.device)
    else:
        odt = _dt(out)
    for name, t in (("g", g), ("beta", beta), ("state", state), ("gate_z", gate_z),
                    ("norm_weight", norm_weight)):
        _f32(t, name)
    _conv_f32(conv_weight, conv_state, conv_state_out)
    conv_dim = 2 * H_k * d_k + H * d_v
    _sizes(q, k=(k, N * H_k * d_k), v=(v, N * H * d_v), g=(g, N * H * (1 if g.dim() == 2 else d_k)),
           beta=(beta, N * H), state=(state, N * H * d_v * d_k), gate_z=(gate_z, N * H * d_v),
           norm_weight=(norm_weight, d_v), out=(out, N * H * d_v),
           conv_weight=(conv_weight, conv_dim * GDN_CONV_KERNEL),
           conv_state=(conv_state, N * conv_dim * (GDN_CONV_KERNEL - 1)),
           conv_state_out=(conv_state_out, N * conv_dim * (GDN_CONV_KERNEL - 1)))
    rc = _run(q, lib().gdn_recurrent_step,
              _p(q), _p(k), _p(v), _p(g), _p(beta), _p(state), N, H, H_k, d_k, d_v, dt,
              _decay_mode(g, 2), float(scale), int(bool(use_qk_l2norm)), _p(conv_weight),
              _p(conv_state), _p(conv_state_out), _p(gate_z), _p(norm_weight), float(norm_eps),
              _p(out), odt, _stream(stream, q))
    _check("gdn_recurrent_step", rc)
    return out


def gdn_recurrent_multi_step(q, k, v, g, beta, state_pool, state_indices=None, scale=0.0,
                             use_qk_l2norm=True, conv_weight=None, conv_state=None,
                             conv_state_out=None, gate_z=None, norm_weight=None, norm_eps=1e-6,
                             out=None, out_dtype=None, stream=None):
    """T decode tokens per sequence on pooled states: q, k [N, T, H_k, d_k]; v [N, T, H, d_v];
    beta [N, T, H]; g [N, T, H] or [N, T, H, d_k]; state_pool [slots, H, d_v, d_k] fp32 updated in
    place; state_indices int32 [N] (negative = skip) or None; conv_state / conv_state_out
    [slots, conv_dim, 3] indexed like the pool.  Returns out [N, T, H, d_v]."""
    N, T, H_k, d_k = q.shape
    H, d_v = v.shape[2], v.shape[-1]
    dt = _dt(q)
    odt = dt if out_dtype is None else _dt(torch.empty(0, dtype=out_dtype))
    if out is None:
        out = torch.empty((N, T, H, d_v), dtype=_torch_dt(odt), device=q.device)
    else:
        odt = _dt(out)
    if state_indices is not None and state_indices.dtype != torch.int32:
        raise TypeError("state_indices must be int32")
    for name, t in (("g", g), ("beta", beta), ("state_pool", state_pool), ("gate_z", gate_z),
                    ("norm_weight", norm_weight)):
        _f32(t, name)
    _conv_f32(conv_weight, conv_state, conv_state_out)
    conv_dim, slots = 2 * H_k * d_k + H * d_v, state_pool.shape[0]
    _sizes(q, k=(k, N * T * H_k * d_k), v=(v, N * T * H * d_v),
           g=(g, N * T * H * (1 if g.dim() == 3 else d_k)), beta=(beta, N * T * H),
           state_pool=(state_pool, slots * H * d_v * d_k), state_indices=(state_indices, N),
           gate_z=(gate_z, N * T * H * d_v), norm_weight=(norm_weight, d_v), out=(out, N * T * H * d_v),
           conv_weight=(conv_weight, conv_dim * GDN_CONV_KERNEL),
           conv_state=(conv_state, slots * conv_dim * (GDN_CONV_KERNEL - 1)),
           conv_state_out=(conv_state_out, slots * conv_dim * (GDN_CONV_KERNEL - 1)))
    rc = _run(q, lib().gdn_recurrent_multi_step,
              _p(q), _p(k), _p(v), _p(g), _p(beta), _p(state_pool), state_pool.shape[0],
              _p(state_indices), N, T, H, H_k, d_k, d_v, dt, _decay_mode(g, 3), float(scale),
              int(bool(use_qk_l2norm)), _p(conv_weight), _p(conv_state), _p(conv_state_out),
              _p(gate_z), _p(norm_weight), float(norm_eps), _p(out), odt, _stream(stream, q))
    _check("gdn_recurrent_multi_step", rc)
    return out


def gdn_gate_rmsnorm_silu(y, z, norm_weight=None, eps=1e-6, out=None, out_dtype=None, stream=None):
    """out = w * y / rms(y) * silu(z) over the last dimension of y (fp32 or bf16)."""
    d_v = y.shape[-1]
    rows = y.numel() // d_v if d_v else 0
    odt = _dt(y) if out_dtype is None else _dt(torch.empty(0, dtype=out_dtype))
    if out is None:
        out = torch.empty(y.shape, dtype=_torch_dt(odt), device=y.device)
    else:
        odt = _dt(out)
    _f32(z, "z")
    _f32(norm_weight, "norm_weight")
    _sizes(y, z=(z, rows * d_v), norm_weight=(norm_weight, d_v), out=(out, rows * d_v))
    rc = _run(y, lib().gdn_gate_rmsnorm_silu,
              _p(y), _dt(y), _p(z), _p(norm_weight), float(eps), _p(out), odt, rows, d_v,
              _stream(stream, y))
    _check("gdn_gate_rmsnorm_silu", rc)
    return out


def gdn_decay_from_logits(a, A_log, dt_bias=None, b=None, g_out=None, beta_out=None, stream=None):
    """g = -exp(A_log) softplus(a + dt_bias) and beta = sigmoid(b); a, b [total_T, H] fp32."""
    total_T, H = a.shape
    for name, t in (("a", a), ("A_log", A_log), ("dt_bias", dt_bias), ("b", b)):
        _f32(t, name)
    if g_out is None:
        g_out = torch.empty_like(a)
    if b is not None and beta_out is None:
        beta_out = torch.empty_like(b)
    _sizes(a, A_log=(A_log, H), dt_bias=(dt_bias, H), b=(b, total_T * H), g_out=(g_out, total_T * H),
           beta_out=(beta_out, total_T * H))
    rc = _run(a, lib().gdn_decay_from_logits,
              _p(a), _p(A_log), _p(dt_bias), _p(b), _p(g_out), _p(beta_out), total_T, H,
              _stream(stream, a))
    _check("gdn_decay_from_logits", rc)
    return (g_out, beta_out) if b is not None else g_out


def _workspace(workspace, need, ref):
    """The caller's workspace, or one of `need` bytes from torch (None when none is needed), with its
    pointer and size."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=ref.device)
        return workspace, workspace.data_ptr(), need
    ptr, = _pointers(ref, ("workspace",), (workspace,), (0,), (False,))
    return workspace, ptr, workspace.numel() * workspace.element_size()


def _same_device(stream, ref):
    """Refuses a stream of another device than the call's: made current, it would leave the call on its own
    device's current stream instead, unordered with the given one."""
    if ref.is_cuda and stream.device != ref.device:
        raise ValueError(f"the stream is on {stream.device}, the call runs on {ref.device}")


def _on_stream(call):
    """With stream=..., runs the call with that stream current, so that what it allocates belongs to the
    stream that uses it (memory taken on one stream may still be read by that stream's pending work)."""
    @functools.wraps(call)
    def wrapped(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        first = next(t for t in (*args, *kw.values()) if isinstance(t, torch.Tensor))
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=first.device)
        _same_device(stream, first)
        with torch.cuda.stream(stream):
            return call(*args, **kw)
    return wrapped


# The tensors of the training calls, in the order of their pointers, and which of them are fp32 only.
_CHUNK_BWD_NAMES = ("q", "k", "v", "g", "beta", "cu_seqlens", "initial_state", "dout", "dfinal_state", "dq", "dk",
                  "dv", "dg", "dbeta", "dinitial_state")
_CHUNK_BWD_FP32 = tuple(n in ("g", "beta", "initial_state", "dfinal_state", "dg", "dbeta", "dinitial_state") for n
                  in _CHUNK_BWD_NAMES)
_RMSNORM_BWD_NAMES = ("dout", "y", "z", "norm_weight", "dy", "dz", "dnorm_weight")
_RMSNORM_BWD_FP32 = tuple(n in ("z", "norm_weight", "dz", "dnorm_weight") for n in _RMSNORM_BWD_NAMES)
_GROUPNORM_NAMES = ("y", "z", "weight", "bias", "out")
_GROUPNORM_FP32 = tuple(n in ("z", "weight", "bias") for n in _GROUPNORM_NAMES)
_GROUPNORM_BWD_NAMES = ("dout", "y", "z", "weight", "bias", "dy", "dz", "dweight", "dbias")
_GROUPNORM_BWD_FP32 = tuple(n in ("z", "weight", "bias", "dz", "dweight", "dbias") for n in _GROUPNORM_BWD_NAMES)
_DECAY_BWD_NAMES = ("a", "A_log", "dt_bias", "b", "dg", "dbeta", "da", "dA_log", "ddt_bias", "db")
_DECAY_BWD_FP32 = tuple(n in ("a", "A_log", "dt_bias", "b", "dg", "dbeta", "da", "dA_log", "ddt_bias", "db") for n
                  in _DECAY_BWD_NAMES)


@_on_stream
def gdn_chunk_bwd(q, k, v, g, beta, dout, cu_seqlens=None, num_seqs=None, scale=0.0, use_qk_l2norm=True,
                  initial_state=None, dfinal_state=None, output_dinitial_state=None, dq=None, dk=None, dv=None,
                  dg=None, dbeta=None, dinitial_state=None, workspace=None):
    """Gradients of gdn_chunk_fwd (without gate and convolution, one decay per head): q, k, v, g, beta,
    cu_seqlens, num_seqs, scale, use_qk_l2norm and initial_state as given to it, dout [total_T, H, d_v]
    (fp32 or bf16) the gradient of out, dfinal_state [num_seqs, H, d_v, d_k] fp32 that of final_state
    (None: zeros).  Returns (dq, dk, dv, dg, dbeta, dinitial_state): dq, dk, dv in the inputs' dtype,
    the others fp32; outputs are allocated unless given.  Rows of tokens outside the sequences of cu_seqlens are
    zeros in the outputs allocated here and left as they were in those given.  dinitial_state is None unless it is given,
    requested, or (output_dinitial_state=None) an initial_state is."""
    total_T, H_k, d_k = q.shape
    H, d_v = v.shape[1], v.shape[-1]
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32:
            raise TypeError("cu_seqlens must be int32")
        num_seqs = cu_seqlens.numel() - 1
    elif num_seqs is None:
        num_seqs = 1
    dt = _dt(q)
    if _dt(k) != dt or _dt(v) != dt:
        raise TypeError("q, k, v must share one dtype")
    own = [x is None for x in (dq, dk, dv, dg, dbeta)]
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if _dt(dq) != dt or _dt(dk) != dt or _dt(dv) != dt:
        raise TypeError("dq, dk, dv must have the dtype of q, k, v")
    if g.dim() != 2:
        raise ValueError("gdn_chunk_bwd takes one decay per head: g [total_T, H]")
    dg = torch.empty((total_T, H), dtype=torch.float32, device=q.device) if dg is None else dg
    dbeta = torch.empty((total_T, H), dtype=torch.float32, device=q.device) if dbeta is None else dbeta
    if dinitial_state is None and (output_dinitial_state or
                                   (output_dinitial_state is None and initial_state is not None)):
        dinitial_state = torch.empty((num_seqs, H, d_v, d_k), dtype=torch.float32, device=q.device)
    states, nk, nv, nh = num_seqs * H * d_v * d_k, total_T * H_k * d_k, total_T * H * d_v, total_T * H
    L = lib()
    p = _pointers(q, _CHUNK_BWD_NAMES,
                  (q, k, v, g, beta, cu_seqlens, initial_state, dout, dfinal_state, dq, dk, dv, dg, dbeta,
                   dinitial_state),
                  (nk, nk, nv, nh, nh, num_seqs + 1, states, nv, states, nk, nk, nv, nh, nh, states),
                  _CHUNK_BWD_FP32)
    need = L.gdn_chunk_bwd_workspace_size(num_seqs, total_T, H, H_k, d_k, d_v)
    workspace, ws, ws_bytes = _workspace(workspace, need, q)
    if cu_seqlens is not None and any(own):
        _check("gdn_chunk_bwd_zero_outside",
               _run(q, L.gdn_chunk_bwd_zero_outside, p[5], num_seqs, total_T, H, H_k, d_k, d_v, dt,
                    *(x if o else None for x, o in zip(p[9:14], own)), _stream(None, q)))
    rc = _run(q, L.gdn_chunk_bwd, *p[:6], num_seqs, total_T, H, H_k, d_k, d_v, dt, GDN_DECAY_PER_HEAD, float(scale),
              int(bool(use_qk_l2norm)), p[6], p[7], _dt(dout), *p[8:], ws, ws_bytes, _stream(None, q))
    _check("gdn_chunk_bwd", rc)
    return dq, dk, dv, dg, dbeta, dinitial_state


@_on_stream
def gdn_gate_rmsnorm_silu_bwd(dout, y, z, norm_weight=None, eps=1e-6, dy=None, dz=None, dnorm_weight=None,
                              workspace=None):
    """Gradients of gdn_gate_rmsnorm_silu: dout (fp32 or bf16), y and z as given to it.  Returns (dy in
    y's dtype, dz fp32, dnorm_weight fp32); dnorm_weight is None unless it or norm_weight is given."""
    d_v = y.shape[-1]
    rows = y.numel() // d_v if d_v else 0
    dy = torch.empty_like(y) if dy is None else dy
    dz = torch.empty_like(y, dtype=torch.float32) if dz is None else dz
    if dnorm_weight is None and norm_weight is not None:
        dnorm_weight = torch.empty_like(norm_weight)
    if dy.dtype != y.dtype:
        raise TypeError("dy must have the dtype of y")
    n, L = rows * d_v, lib()
    p = _pointers(y, _RMSNORM_BWD_NAMES,
                  (dout, y, z, norm_weight, dy, dz, dnorm_weight),
                  (n, n, n, d_v, n, n, d_v),
                  _RMSNORM_BWD_FP32)
    need = L.gdn_gate_bwd_workspace_size(rows, 1, d_v) if dnorm_weight is not None else 0
    workspace, ws, ws_bytes = _workspace(workspace, need, y)
    rc = _run(y, L.gdn_gate_rmsnorm_silu_bwd, p[0], _dt(dout), p[1], _dt(y), p[2], p[3], float(eps), p[4], p[5], p[6],
              rows, d_v, ws, ws_bytes, _stream(None, y))
    _check("gdn_gate_rmsnorm_silu_bwd", rc)
    return dy, dz, dnorm_weight


def _groups(y):
    if y.dim() < 2:
        raise ValueError("y must be [..., groups, group_size]")
    groups, size = y.shape[-2:]
    return (y.numel() // (groups * size) if groups * size else 0), groups, size


@_on_stream
def gdn_gate_groupnorm_silu(y, z=None, weight=None, bias=None, eps=1e-6, out=None, out_dtype=None):
    """Group norm over the heads, channels last, with a SiLU: y [..., groups, group_size] (fp32 or bf16),
    m = weight * (y - mean) / sqrt(var + eps) + bias per group, out = m * silu(z), or silu(m) without z.
    z like y, fp32; weight, bias [groups, group_size] fp32 or None."""
    rows, groups, size = _groups(y)
    if out is None:
        out = torch.empty_like(y, dtype=out_dtype)
    n, c = rows * groups * size, groups * size
    p = _pointers(y, _GROUPNORM_NAMES,
                  (y, z, weight, bias, out),
                  (n, n, c, c, n),
                  _GROUPNORM_FP32)
    rc = _run(y, lib().gdn_gate_groupnorm_silu, p[0], _dt(y), p[1], p[2], p[3], float(eps), p[4], _dt(out), rows,
              groups, size, _stream(None, y))
    _check("gdn_gate_groupnorm_silu", rc)
    return out


@_on_stream
def gdn_gate_groupnorm_silu_bwd(dout, y, z=None, weight=None, bias=None, eps=1e-6, dy=None, dz=None, dweight=None,
                                dbias=None, workspace=None):
    """Gradients of gdn_gate_groupnorm_silu: dout (fp32 or bf16) and the forward's inputs.  Returns (dy in
    y's dtype, dz fp32 or None without z, dweight, dbias fp32 [groups, group_size]); dweight (dbias) is
    None unless it or weight (bias) is given."""
    rows, groups, size = _groups(y)
    n, c = rows * groups * size, groups * size
    dy = torch.empty_like(y) if dy is None else dy
    if dy.dtype != y.dtype:
        raise TypeError("dy must have the dtype of y")
    if z is not None and dz is None:
        dz = torch.empty_like(z)
    if weight is not None and dweight is None:
        dweight = torch.empty_like(weight)
    if bias is not None and dbias is None:
        dbias = torch.empty_like(bias)
    L = lib()
    p = _pointers(y, _GROUPNORM_BWD_NAMES,
                  (dout, y, z, weight, bias, dy, dz, dweight, dbias),
                  (n, n, n, c, c, n, n, c, c),
                  _GROUPNORM_BWD_FP32)
    need = L.gdn_gate_bwd_workspace_size(rows, groups, size) if dweight is not None or dbias is not None else 0
    workspace, ws, ws_bytes = _workspace(workspace, need, y)
    rc = _run(y, L.gdn_gate_groupnorm_silu_bwd, p[0], _dt(dout), p[1], _dt(y), p[2], p[3], p[4], float(eps), p[5],
              p[6], p[7], p[8], rows, groups, size, ws, ws_bytes, _stream(None, y))
    _check("gdn_gate_groupnorm_silu_bwd", rc)
    return dy, dz, dweight, dbias


@_on_stream
def gdn_decay_from_logits_bwd(a, A_log, dt_bias, b, dg, dbeta, da=None, dA_log=None, ddt_bias=None, db=None,
                              workspace=None):
    """Gradients of gdn_decay_from_logits: a, A_log, dt_bias (or None), b (or None) as given to it, dg
    [total_T, H] and dbeta [total_T, H] (None exactly when b is) those of its outputs, fp32.  Returns
    (da, dA_log, ddt_bias, db); ddt_bias is None unless it or dt_bias is given, db is None without b."""
    total_T, H = a.shape
    if (b is None) != (dbeta is None):
        raise ValueError("b and dbeta are given together")
    da = torch.empty_like(a) if da is None else da
    dA_log = torch.empty_like(A_log) if dA_log is None else dA_log
    if dt_bias is not None and ddt_bias is None:
        ddt_bias = torch.empty_like(dt_bias)
    if b is not None and db is None:
        db = torch.empty_like(b)
    n, L = total_T * H, lib()
    p = _pointers(a, _DECAY_BWD_NAMES,
                  (a, A_log, dt_bias, b, dg, dbeta, da, dA_log, ddt_bias, db),
                  (n, H, H, n, n, n, n, H, H, n),
                  _DECAY_BWD_FP32)
    workspace, ws, ws_bytes = _workspace(workspace, L.gdn_decay_bwd_workspace_size(total_T, H), a)
    rc = _run(a, L.gdn_decay_from_logits_bwd, *p[:10], total_T, H, ws, ws_bytes, _stream(None, a))
    _check("gdn_decay_from_logits_bwd", rc)
    return da, dA_log, ddt_bias, db


def _rows(ref, name, t, shape, lead=1):
    """Pointer and stride of a token tensor that may be a slice of a wider one: `shape` (its first `lead` dimensions
    the tokens), each token's row contiguous, tokens one stride apart."""
    if t.shape != shape:
        raise ValueError(f"{name} is {tuple(t.shape)}, the call needs {tuple(shape)}")
    if t.get_device() != ref.get_device() or (not ref.is_cuda and t.device != ref.device):
        raise ValueError(f"{name} is on {t.device}, the call runs on {ref.device}")
    tokens, width = math.prod(shape[:lead]), math.prod(shape[lead:])
    stride = width if tokens > 1 else -(-width // 8) * 8  # one row has no stride
    if t.is_contiguous():
        return t.data_ptr(), stride
    strides, width = t.stride(), 1
    for n, st in zip(reversed(shape[lead:]), reversed(strides[lead:])):
        if n != 1 and st != width:
            raise ValueError(f"{name}: the rows of a token must be contiguous")
        width *= n
    if tokens > 1:
        stride = strides[lead - 1]
        if lead == 2:
            if shape[1] == 1:
                stride = strides[0]
            elif shape[0] > 1 and strides[0] != shape[1] * stride:
                raise ValueError(f"{name}: tokens must be one stride apart over all sequences")
    return t.data_ptr(), stride


def _seqs(cu_seqlens, num_seqs):
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32:
            raise TypeError("cu_seqlens must be int32")
        return cu_seqlens.numel() - 1
    return 1 if num_seqs is None else num_seqs


def _same_dtype(dt, **tensors):
    dtype = _torch_dt(dt)
    for name, t in tensors.items():
        if t is not None and t.dtype is not dtype:
            raise TypeError(f"{name} must have the dtype of the inputs")


def _tokens(t, dims, name):
    """A step call's tensor with its token dimension: [N, T, ...] as given, or [N, ...] as one token."""
    if t.dim() == dims:
        return t
    if t.dim() == dims - 1:
        return t.unsqueeze(1)
    raise ValueError(f"{name} must have {dims - 1} or {dims} dimensions")


_CONV_NAMES = ("weight", "bias", "cu_seqlens", "conv_state", "conv_state_out", "out")
_CONV_FP32 = (True, True, False, True, True, False)
_CONV_STEP_NAMES = ("weight", "bias", "conv_state", "state_indices", "out")
_CONV_STEP_FP32 = (True, True, True, False, False)
_CONV_BWD_NAMES = ("dout", "weight", "bias", "cu_seqlens", "conv_state", "dconv_state_out", "dx", "dweight", "dbias",
                   "dconv_state")
_CONV_BWD_FP32 = (False, True, True, False, True, True, False, True, True, True)
_SSM_NAMES = ("a", "A_log", "dt_bias", "D", "cu_seqlens", "initial_state", "final_state", "out")
_SSM_FP32 = (True, True, True, True, False, True, True, False)
_SSM_STEP_NAMES = ("a", "A_log", "dt_bias", "D", "state", "state_indices", "out")
_SSM_STEP_FP32 = (True, True, True, True, True, False, False)
_SSM_BWD_NAMES = ("dout", "a", "A_log", "dt_bias", "D", "cu_seqlens", "initial_state", "dfinal_state", "dx", "dB", "dC",
                  "da", "dA_log", "ddt_bias", "dD", "dinitial_state")
_SSM_BWD_FP32 = (False, True, True, True, True, False, True, True, False, False, False, True, True, True, True, True)
_QK_NAMES = ("cos_sin", "positions", "q_weight", "k_weight", "dq_weight", "dk_weight")
_QK_FP32 = (True, False, True, True, True, True)


@_on_stream
def gdn_short_conv_fwd(x, weight, bias=None, cu_seqlens=None, num_seqs=None, conv_state=None, conv_state_out=None,
                       output_final_state=True, silu=True, out=None):
    """The causal short convolution (four taps, SiLU) over packed sequences: x [total_T, dim] (fp32 or bf16; may be a
    slice of a wider tensor, rows one stride apart), weight [dim, 4], bias [dim] or None, conv_state
    [num_seqs, dim, 3] the carried inputs (None: zeros).  Returns (out [total_T, dim], conv_state_out), which is
    allocated unless given (it may be conv_state itself) or not requested."""
    total_T, dim = x.shape
    num_seqs, dt = _seqs(cu_seqlens, num_seqs), _dt(x)
    px, stride = _rows(x, "x", x, (total_T, dim))
    if out is None:
        out = torch.empty((total_T, dim), dtype=x.dtype, device=x.device)
    _same_dtype(dt, out=out)
    if conv_state_out is None and output_final_state:
        conv_state_out = torch.empty((num_seqs, dim, 3), dtype=torch.float32, device=x.device)
    st = num_seqs * dim * 3
    p = _pointers(x, _CONV_NAMES, (weight, bias, cu_seqlens, conv_state, conv_state_out, out),
                  (dim * GDN_CONV_KERNEL, dim, num_seqs + 1, st, st, total_T * dim), _CONV_FP32)
    _check("gdn_short_conv_fwd",
           _run(x, lib().gdn_short_conv_fwd, px, stride, p[0], p[1], p[2], num_seqs, total_T, dim, dt,
                int(bool(silu)), p[3], p[4], p[5], _stream(None, x)))
    return out, conv_state_out


@_on_stream
def gdn_short_conv_step(x, weight, conv_state, bias=None, state_indices=None, silu=True, out=None):
    """The convolution of T more tokens of N sequences: x [N, T, dim] or [N, dim] (a slice of a wider tensor is
    taken as it is), conv_state [slots, dim, 3] fp32 updated in place, state_indices int32 [N] (negative = skip) or None.
    Returns out like x."""
    x3 = _tokens(x, 3, "x")
    N, T, dim = x3.shape
    dt = _dt(x)
    px, stride = _rows(x, "x", x3, (N, T, dim), lead=2)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _same_dtype(dt, out=out)
    if state_indices is not None and state_indices.dtype != torch.int32:
        raise TypeError("state_indices must be int32")
    slots = conv_state.shape[0]
    p = _pointers(x, _CONV_STEP_NAMES, (weight, bias, conv_state, state_indices, out),
                  (dim * GDN_CONV_KERNEL, dim, slots * dim * 3, N, N * T * dim), _CONV_STEP_FP32)
    _check("gdn_short_conv_step",
           _run(x, lib().gdn_short_conv_step, px, stride, p[0], p[1], p[2], slots, p[3], N, T, dim, dt,
                int(bool(silu)), p[4], _stream(None, x)))
    return out


@_on_stream
def gdn_short_conv_bwd(dout, x, weight, bias=None, cu_seqlens=None, num_seqs=None, conv_state=None,
                       dconv_state_out=None, silu=True, dx=None, dweight=None, dbias=None, dconv_state=None,
                       workspace=None):
    """Gradients of gdn_short_conv_fwd: dout [total_T, dim] in x's dtype, the forward's inputs, dconv_state_out the
    gradient of its final history (None: zeros).  Returns (dx, dweight, dbias, dconv_state): dx in x's dtype, the
    others fp32; dbias is None unless it or bias is given, dconv_state unless it or conv_state is.  Rows of tokens
    outside the sequences of cu_seqlens are zeros in a dx allocated here and left as they were in one given."""
    total_T, dim = x.shape
    num_seqs, dt = _seqs(cu_seqlens, num_seqs), _dt(x)
    px, stride = _rows(x, "x", x, (total_T, dim))
    zeros = dx is None
    if dx is None:
        dx = torch.empty((total_T, dim), dtype=x.dtype, device=x.device)
    _same_dtype(dt, dout=dout, dx=dx)
    if dweight is None:
        dweight = torch.empty((dim, GDN_CONV_KERNEL), dtype=torch.float32, device=x.device)
    if dbias is None and bias is not None:
        dbias = torch.empty((dim,), dtype=torch.float32, device=x.device)
    if dconv_state is None and conv_state is not None:
        dconv_state = torch.empty((num_seqs, dim, 3), dtype=torch.float32, device=x.device)
    st, n, L = num_seqs * dim * 3, total_T * dim, lib()
    p = _pointers(x, _CONV_BWD_NAMES,
                  (dout, weight, bias, cu_seqlens, conv_state, dconv_state_out, dx, dweight, dbias, dconv_state),
                  (n, dim * GDN_CONV_KERNEL, dim, num_seqs + 1, st, st, n, dim * GDN_CONV_KERNEL, dim, st),
                  _CONV_BWD_FP32)
    workspace, ws, ws_bytes = _workspace(workspace, L.gdn_short_conv_bwd_workspace_size(num_seqs, total_T, dim), x)
    _check("gdn_short_conv_bwd",
           _run(x, L.gdn_short_conv_bwd, p[0], px, stride, p[1], p[2], p[3], num_seqs, total_T, dim, dt,
                int(bool(silu)), p[4], p[5], p[6], p[7], p[8], p[9], int(zeros), ws, ws_bytes, _stream(None, x)))
    return dx, dweight, dbias, dconv_state


def _ssm_inputs(x, B, C, lead):
    """Sizes, dtype and the pointers with strides of x [..., H, P], B and C [..., G, N]."""
    H, P = x.shape[lead:]
    G, N = B.shape[lead:]
    dt = _dt(x)
    _same_dtype(dt, B=B, C=C)
    tok = tuple(x.shape[:lead])
    rows = (*_rows(x, "x", x, tok + (H, P), lead), *_rows(x, "B", B, tok + (G, N), lead),
            *_rows(x, "C", C, tok + (G, N), lead))
    return H, P, G, N, dt, rows


@_on_stream
def gdn_ssm_chunk_fwd(x, B, C, a, A_log, dt_bias=None, D=None, cu_seqlens=None, num_seqs=None, initial_state=None,
                      final_state=None, output_final_state=True, out=None, workspace=None):
    """The selective state space scan over packed prompts: S_t = exp(-exp(A_log) dt_t) S_{t-1} + dt_t x_t B_t^T,
    y_t = S_t C_t + D x_t, dt = softplus(a + dt_bias).  x [total_T, H, P], B, C [total_T, G, N] (fp32 or bf16; slices of
    a wider tensor are taken as they are), a [total_T, H], A_log, dt_bias, D [H] fp32, states [num_seqs, H, P, N] fp32.
    Returns (out [total_T, H, P], final_state), which is allocated unless given or not requested."""
    total_T = x.shape[0]
    H, P, G, N, dt, rows = _ssm_inputs(x, B, C, 1)
    num_seqs = _seqs(cu_seqlens, num_seqs)
    if out is None:
        out = torch.empty((total_T, H, P), dtype=x.dtype, device=x.device)
    _same_dtype(dt, out=out)
    if final_state is None and output_final_state:
        final_state = torch.empty((num_seqs, H, P, N), dtype=torch.float32, device=x.device)
    st, L = num_seqs * H * P * N, lib()
    p = _pointers(x, _SSM_NAMES, (a, A_log, dt_bias, D, cu_seqlens, initial_state, final_state, out),
                  (total_T * H, H, H, H, num_seqs + 1, st, st, total_T * H * P), _SSM_FP32)
    need = L.gdn_ssm_chunk_fwd_workspace_size(num_seqs, total_T, H, G, P, N, dt)
    workspace, ws, ws_bytes = _workspace(workspace, need, x)
    _check("gdn_ssm_chunk_fwd",
           _run(x, L.gdn_ssm_chunk_fwd, *rows, *p[:5], num_seqs, total_T, H, G, P, N, dt, *p[5:], ws, ws_bytes,
                _stream(None, x)))
    return out, final_state


@_on_stream
def gdn_ssm_step(x, B, C, a, A_log, state, dt_bias=None, D=None, state_indices=None, out=None):
    """T tokens of the scan for N sequences: x [N, T, H, P], B, C [N, T, G, N_state], a [N, T, H] (or without T, for one
    token), state [slots, H, P, N_state] fp32 updated in place, state_indices int32 [N] (negative = skip) or None.
    Returns out like x."""
    x4, a3 = _tokens(x, 4, "x"), _tokens(a, 3, "a")
    n_seq, T = x4.shape[:2]
    H, P, G, N, dt, rows = _ssm_inputs(x4, _tokens(B, 4, "B"), _tokens(C, 4, "C"), 2)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _same_dtype(dt, out=out)
    if state_indices is not None and state_indices.dtype != torch.int32:
        raise TypeError("state_indices must be int32")
    slots = state.shape[0]
    p = _pointers(x, _SSM_STEP_NAMES, (a3, A_log, dt_bias, D, state, state_indices, out),
                  (n_seq * T * H, H, H, H, slots * H * P * N, n_seq, n_seq * T * H * P), _SSM_STEP_FP32)
    _check("gdn_ssm_step",
           _run(x, lib().gdn_ssm_step, *rows, *p[:5], slots, p[5], n_seq, T, H, G, P, N, dt, p[6], _stream(None, x)))
    return out


@_on_stream
def gdn_ssm_chunk_bwd(dout, x, B, C, a, A_log, dt_bias=None, D=None, cu_seqlens=None, num_seqs=None,
                      initial_state=None, dfinal_state=None, output_dinitial_state=None, dx=None, dB=None, dC=None,
                      da=None, dA_log=None, ddt_bias=None, dD=None, dinitial_state=None, workspace=None):
    """Gradients of gdn_ssm_chunk_fwd: dout [total_T, H, P] in x's dtype, the forward's inputs, dfinal_state the
    gradient of final_state (None: zeros).  Returns (dx, dB, dC, da, dA_log, ddt_bias, dD, dinitial_state): the first
    three in x's dtype, the others fp32; ddt_bias (dD) is None unless it or dt_bias (D) is given, dinitial_state unless
    it is given, requested, or (output_dinitial_state=None) an initial_state is.  Rows of tokens outside the sequences
    of cu_seqlens are zeros when dx, dB, dC and da are all allocated here, and left as they were otherwise."""
    total_T = x.shape[0]
    H, P, G, N, dt, rows = _ssm_inputs(x, B, C, 1)
    num_seqs = _seqs(cu_seqlens, num_seqs)
    zeros = dx is None and dB is None and dC is None and da is None

    def new(t, shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=x.device) if t is None else t

    dx, da = new(dx, (total_T, H, P), x.dtype), new(da, (total_T, H))
    dB, dC = new(dB, (total_T, G, N), x.dtype), new(dC, (total_T, G, N), x.dtype)
    _same_dtype(dt, dout=dout, dx=dx, dB=dB, dC=dC)
    dA_log = new(dA_log, (H,))
    if dt_bias is not None:
        ddt_bias = new(ddt_bias, (H,))
    if D is not None:
        dD = new(dD, (H,))
    if output_dinitial_state or (output_dinitial_state is None and initial_state is not None):
        dinitial_state = new(dinitial_state, (num_seqs, H, P, N))
    st, nx, nb, L = num_seqs * H * P * N, total_T * H * P, total_T * G * N, lib()
    p = _pointers(x, _SSM_BWD_NAMES,
                  (dout, a, A_log, dt_bias, D, cu_seqlens, initial_state, dfinal_state, dx, dB, dC, da, dA_log,
                   ddt_bias, dD, dinitial_state),
                  (nx, total_T * H, H, H, H, num_seqs + 1, st, st, nx, nb, nb, total_T * H, H, H, H, st),
                  _SSM_BWD_FP32)
    need = L.gdn_ssm_chunk_bwd_workspace_size(num_seqs, total_T, H, G, P, N, dt)
    workspace, ws, ws_bytes = _workspace(workspace, need, x)
    _check("gdn_ssm_chunk_bwd",
           _run(x, L.gdn_ssm_chunk_bwd, p[0], *rows, *p[1:6], num_seqs, total_T, H, G, P, N, dt, *p[6:],
                int(zeros), ws, ws_bytes, _stream(None, x)))
    return dx, dB, dC, da, dA_log, ddt_bias, dD, dinitial_state


def _qk_inputs(q, k, cos_sin, positions, q_weight, k_weight, dq_weight=None, dk_weight=None):
    T, H, d = q.shape
    H_k, dt = (0 if k is None else k.shape[1]), _dt(q)
    _same_dtype(dt, k=k)
    max_positions, rot = (0, 0) if cos_sin is None else cos_sin.shape
    if positions is not None and positions.dtype != torch.int32:
        raise TypeError("positions must be int32")
    p = _pointers(q, _QK_NAMES, (cos_sin, positions, q_weight, k_weight, dq_weight, dk_weight),
                  (max_positions * rot, T, d, d, d, d), _QK_FP32)
    rows = (*_rows(q, "q", q, (T, H, d)), *((None, 0) if k is None else _rows(q, "k", k, (T, H_k, d))))
    return T, H, H_k, d, rot, dt, max_positions, p, rows


def _qk_output(q, name, out, T, heads, d):
    """An output of the norm and rotation, its pointer and stride; allocated unless given."""
    if heads == 0:
        return None, None, 0
    if out is None:
        out = q.new_empty((T, heads, d))
        return out, out.data_ptr(), heads * d
    _same_dtype(_dt(q), **{name: out})
    return out, *_rows(q, name, out, (T, heads, d))


@_on_stream
def gdn_qk_norm_rope(q, k, cos_sin, positions=None, q_weight=None, k_weight=None, norm=GDN_NORM_RMS, eps=1e-6,
                     interleaved=False, q_out=None, k_out=None):
    """Queries and keys normalised per head (GDN_NORM_RMS, or GDN_NORM_L2: to length one) and rotated by their
    position: q [T, H, d], k [T, H_k, d] or None (fp32 or bf16; slices of a wider tensor are taken as they are), cos_sin
    [max_positions, d_rot] fp32 (the cosines of a position's d_rot / 2 angles, then the sines; None: no rotation),
    positions int32 [T] or None (row t has position t), weights [d] fp32 or None.  Pairs are channels i and
    d_rot / 2 + i, or neighbours when interleaved.  Returns (q_out, k_out), allocated unless given (they may be q and k)."""
    T, H, H_k, d, rot, dt, most, p, rows = _qk_inputs(q, k, cos_sin, positions, q_weight, k_weight)
    q_out, pq, sq = _qk_output(q, "q_out", q_out, T, H, d)
    k_out, pk, sk = _qk_output(q, "k_out", k_out, T, H_k, d)
    _check("gdn_qk_norm_rope",
           _run(q, lib().gdn_qk_norm_rope, *rows, p[0], p[1], most, p[2], p[3], int(norm), float(eps),
                int(bool(interleaved)), T, H, H_k, d, rot, dt, pq, sq, pk, sk, _stream(None, q)))
    return q_out, k_out


@_on_stream
def gdn_qk_norm_rope_bwd(dq_out, dk_out, q, k, cos_sin, positions=None, q_weight=None, k_weight=None, norm=GDN_NORM_RMS,
                         eps=1e-6, interleaved=False, dq=None, dk=None, dq_weight=None, dk_weight=None, workspace=None):
    """Gradients of gdn_qk_norm_rope: dq_out, dk_out (contiguous, in q's dtype) and the forward's inputs.  Returns
    (dq, dk in q's dtype, dq_weight, dk_weight fp32); a weight's gradient is None unless it or the weight is given."""
    if q_weight is not None and dq_weight is None:
        dq_weight = torch.empty_like(q_weight)
    if k_weight is not None and dk_weight is None and k is not None:
        dk_weight = torch.empty_like(k_weight)
    T, H, H_k, d, rot, dt, most, p, rows = _qk_inputs(q, k, cos_sin, positions, q_weight, k_weight, dq_weight, dk_weight)
    dq, pq, sq = _qk_output(q, "dq", dq, T, H, d)
    dk, pk, sk = _qk_output(q, "dk", dk, T, H_k, d)
    _same_dtype(dt, dq_out=dq_out, dk_out=dk_out)
    g = _pointers(q, ("dq_out", "dk_out"), (dq_out, dk_out), (T * H * d, T * H_k * d), (False, False))
    L = lib()
    need = L.gdn_qk_norm_rope_bwd_workspace_size(T, H, H_k, d) if dq_weight is not None or dk_weight is not None else 0
    workspace, ws, ws_bytes = _workspace(workspace, need, q)
    _check("gdn_qk_norm_rope_bwd",
           _run(q, L.gdn_qk_norm_rope_bwd, *g, *rows, p[0], p[1], most, p[2], p[3], int(norm), float(eps),
                int(bool(interleaved)), T, H, H_k, d, rot, dt, pq, sq, pk, sk, p[4], p[5], ws, ws_bytes, _stream(None, q)))
    return dq, dk, dq_weight, dk_weight


def gdn_selftest_bounded_wait(limit_ns, status=None, stream=None):
    """Run the library's bounded device wait on a phase that never completes (limit_ns in
    [1e3, 1e9]); returns the int32 device tensor the kernel writes its status to
    (GDN_ERR_TIMEOUT = -6 once the wait has given up)."""
    if status is None:
        status = torch.full((1,), 1, dtype=torch.int32, device="cuda")
    if status.dtype != torch.int32 or status.numel() < 1:
        raise ValueError("status must be an int32 tensor with at least one element")
    rc = _run(status, lib().gdn_selftest_bounded_wait, int(limit_ns), _p(status),
              _stream(stream, status))
    _check("gdn_selftest_bounded_wait", rc)
    return status


def gdn_get_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device-side status word."""
    st = ctypes.c_int(0)
    _check("gdn_get_device_error", lib().gdn_get_device_error(_stream(stream), ctypes.byref(st)))
    return st.value


def gdn_set_kernel_forms(prefill_fused=GDN_FORM_AUTO, decode_blocks=GDN_FORM_AUTO):
    """Process-wide choice between the library's equivalent kernel forms (GDN_FORM_AUTO / _OFF /
    _ON for the fused prefill launch and for the four-token block decode); for comparisons and
    tests.  Call it with no arguments to restore the automatic choice."""
    _check("gdn_set_kernel_forms", lib().gdn_set_kernel_forms(int(prefill_fused), int(decode_blocks)))
