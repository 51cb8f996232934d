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
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libgdn.so")

GDN_F32, GDN_BF16 = 0, 1
GDN_DECAY_PER_HEAD, GDN_DECAY_PER_KEY_CHANNEL = 0, 1
GDN_CONV_KERNEL = 4
GDN_FORM_AUTO, GDN_FORM_OFF, GDN_FORM_ON = 0, 1, 2
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
