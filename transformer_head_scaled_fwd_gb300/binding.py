"""Thin ctypes binding of ``libmha.so`` (the C ABI in ``include/mha.h``).

Argument marshalling only: tensors are passed as raw pointers, every step of
the forward pass runs in the library's CUDA kernels. There is no fallback:
if the library is missing or a call fails, an exception is raised.

Function names match the C entry points: ``mha_forward``,
``mha_qkv_projection``, ``mha_attention_core``, ``mha_output_projection``,
``mha_forward_host``, ``mha_workspace_size``, ``mha_host_staging_size``,
``mha_check_device_status``; the serving operators ``mha_rotary``,
``mha_paged_append``, ``mha_paged_attention``, ``mha_attention``,
``mha_document_spans``, ``mha_rmsnorm``, ``mha_paged_resize``, ``mha_coded_append``,
``mha_coded_attention`` and the ``make_*`` descriptions they take.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmha.so")

MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED, MHA_ERR_CUDA = 0, 1, 2, 3
MHA_F32, MHA_BF16 = 0, 1

# every symbol include/mha.h declares
EXPORTS = ("mha_workspace_size", "mha_forward", "mha_qkv_projection", "mha_attention_core",
           "mha_output_projection", "mha_host_staging_size", "mha_forward_host", "mha_last_error",
           "mha_check_device_status", "mha_version", "mha_forward_noalloc", "mha_ffn_workspace_size",
           "mha_ffn_forward", "mha_sublayer_workspace_size", "mha_sublayer_forward",
           "mha_decode_workspace_size", "mha_kv_cache_prefill", "mha_decode_step",
           "mha_selftest_wait_timeout", "mha_rotary_frequencies", "mha_rotary", "mha_paged_append",
           "mha_paged_attention_workspace_size", "mha_paged_attention", "mha_document_spans",
           "mha_attention", "mha_rmsnorm", "mha_paged_resize", "mha_coded_append",
           "mha_coded_attention_workspace_size", "mha_coded_attention")
MHA_SELFTEST_WAIT_CODE = 0x7f1


class MHAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"status {status}: {message}")
        self.status = status


class MaskT(ctypes.Structure):
    _fields_ = [("causal", ctypes.c_int), ("key_valid_lens", ctypes.c_void_p),
                ("dense", ctypes.c_void_p), ("dense_mq", ctypes.c_int)]


class StridesT(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("l", ctypes.c_int64), ("h", ctypes.c_int64)]


class RotaryT(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("scale", ctypes.c_float)]


class PagedCacheT(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("n_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("max_pages", ctypes.c_int)]


class CodedCacheT(ctypes.Structure):
    _fields_ = [("pages", PagedCacheT), ("code", ctypes.c_int), ("block", ctypes.c_int), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p)]


class ScoresT(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("cap", ctypes.c_float), ("slopes", ctypes.c_void_p)]


class SpanMaskT(ctypes.Structure):
    _fields_ = [("causal", ctypes.c_int), ("q_offset", ctypes.c_int), ("key_valid_lens", ctypes.c_void_p),
                ("prefix_lens", ctypes.c_void_p), ("doc_spans", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None


def load(path: str | None = None):
    """Load libmha.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise ImportError(f"{p} not found: build it with transformer_head_scaled_fwd_gb300.build.build()")
        lib = ctypes.CDLL(p)
        vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.mha_workspace_size.restype = sz
        lib.mha_workspace_size.argtypes = [i] * 6
        lib.mha_forward.restype = i
        lib.mha_forward.argtypes = [i] + [vp] * 11 + [i] * 5 + [ctypes.POINTER(MaskT), vp, vp, vp, sz, vp]
        lib.mha_qkv_projection.restype = i
        lib.mha_qkv_projection.argtypes = [i] + [vp] * 9 + [i] * 5 + [vp, sz, vp]
        lib.mha_attention_core.restype = i
        lib.mha_attention_core.argtypes = [i] * 6 + [ctypes.POINTER(MaskT), vp, vp, sz, vp]
        lib.mha_output_projection.restype = i
        lib.mha_output_projection.argtypes = [i, vp, vp] + [i] * 5 + [vp, vp, sz, vp]
        lib.mha_host_staging_size.restype = sz
        lib.mha_host_staging_size.argtypes = [i] * 7
        lib.mha_forward_host.restype = i
        lib.mha_forward_host.argtypes = ([i] + [vp] * 11 + [i] * 5
                                         + [ctypes.POINTER(MaskT), vp, vp, sz, vp, sz, vp])
        lib.mha_last_error.restype = ctypes.c_char_p
        lib.mha_last_error.argtypes = []
        lib.mha_check_device_status.restype = i
        lib.mha_check_device_status.argtypes = [ctypes.POINTER(ctypes.c_int), i]
        lib.mha_version.restype = ctypes.c_char_p
        lib.mha_version.argtypes = []
        lib.mha_ffn_workspace_size.restype = sz
        lib.mha_ffn_workspace_size.argtypes = [i] * 5
        lib.mha_ffn_forward.restype = i
        lib.mha_ffn_forward.argtypes = [i] + [vp] * 5 + [i] * 4 + [vp, vp, sz, vp]
        lib.mha_sublayer_workspace_size.restype = sz
        lib.mha_sublayer_workspace_size.argtypes = [i] * 6
        lib.mha_sublayer_forward.restype = i
        lib.mha_sublayer_forward.argtypes = ([i, vp, vp, vp, vp, ctypes.c_float, i] + [vp] * 8 + [i] * 5
                                             + [ctypes.POINTER(MaskT), vp, vp, sz, vp])
        lib.mha_decode_workspace_size.restype = sz
        lib.mha_decode_workspace_size.argtypes = [i] * 4
        lib.mha_kv_cache_prefill.restype = i
        lib.mha_kv_cache_prefill.argtypes = [i] + [vp] * 5 + [i] * 4 + [vp, vp, i, vp]
        lib.mha_decode_step.restype = i
        lib.mha_decode_step.argtypes = [i] + [vp] * 9 + [i] * 3 + [vp, vp, vp, i, vp, vp, sz, vp]
        lib.mha_selftest_wait_timeout.restype = i
        lib.mha_selftest_wait_timeout.argtypes = [vp]
        lib.mha_forward_noalloc.restype = i
        lib.mha_forward_noalloc.argtypes = [i] + [vp] * 11 + [i] * 5 + [ctypes.POINTER(MaskT), vp, vp, vp]
        i64, f = ctypes.c_int64, ctypes.c_float
        lib.mha_rotary_frequencies.restype = i
        lib.mha_rotary_frequencies.argtypes = [vp, vp, i, ctypes.c_double, i] + [ctypes.c_double] * 4
        lib.mha_rotary.restype = i
        lib.mha_rotary.argtypes = [i] + [vp] * 8 + [i] * 5 + [vp] * 3
        lib.mha_paged_append.restype = i
        lib.mha_paged_append.argtypes = [i] + [vp] * 10 + [i] * 5 + [vp] * 5
        lib.mha_paged_attention_workspace_size.restype = sz
        lib.mha_paged_attention_workspace_size.argtypes = [i] * 5
        lib.mha_paged_attention.restype = i
        lib.mha_paged_attention.argtypes = [i] + [vp] * 4 + [i] * 4 + [vp] * 4 + [sz, vp]
        lib.mha_document_spans.restype = i
        lib.mha_document_spans.argtypes = [vp, i, i, vp, vp]
        lib.mha_attention.restype = i
        lib.mha_attention.argtypes = [i] + [vp] * 8 + [i] * 6 + [vp] * 3
        lib.mha_rmsnorm.restype = i
        lib.mha_rmsnorm.argtypes = [i, vp, i64, vp, i64, vp, i64, vp, f, i64, i, vp, i64, vp, i, vp]
        lib.mha_paged_resize.restype = i
        lib.mha_paged_resize.argtypes = [vp, vp, i, i, vp, i64, i, vp, i, vp, vp, vp, i, vp, vp]
        lib.mha_coded_append.restype = i
        lib.mha_coded_append.argtypes = [i] + [vp] * 10 + [i] * 5 + [vp] * 5
        lib.mha_coded_attention_workspace_size.restype = sz
        lib.mha_coded_attention_workspace_size.argtypes = [i] * 5
        lib.mha_coded_attention.restype = i
        lib.mha_coded_attention.argtypes = [i] + [vp] * 4 + [i] * 4 + [vp] * 4 + [sz, vp]
        _lib = lib
        return lib


def _check(status: int):
    if status != MHA_OK:
        raise MHAError(status, load().mha_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return MHA_BF16
    if t.dtype == torch.float32:
        return MHA_F32
    raise TypeError(f"unsupported dtype {t.dtype}: use torch.bfloat16 or torch.float32")


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_mask(causal=False, key_valid_lens=None, dense=None):
    """Build the C mask struct. The struct holds references to the two tensors, so
    they stay allocated for as long as the struct is alive."""
    if not causal and key_valid_lens is None and dense is None:
        return None
    m = MaskT()
    m.causal = int(bool(causal))
    m.key_valid_lens = _ptr(key_valid_lens)
    m.dense = _ptr(dense)
    m.dense_mq = int(dense.shape[1]) if dense is not None else 0
    m._tensors = (key_valid_lens, dense)
    return m


def workspace_size(dt: int, B: int, Lq: int, Lk: int, d_model: int, h: int) -> int:
    return int(load().mha_workspace_size(dt, B, Lq, Lk, d_model, h))


def mha_forward(query, key, value, w_q, b_q, w_k, b_k, w_v, b_v, w_o, b_o, h, *, out, workspace,
                mask=None, p_attn=None, stream=None):
    """Enqueue the whole sublayer on ``stream``. All tensors are CUDA tensors."""
    B, Lq, d = query.shape
    Lk = key.shape[1]
    _check(load().mha_forward(
        _dtype_code(query), _ptr(query), _ptr(key), _ptr(value), _ptr(w_q), _ptr(b_q), _ptr(w_k),
        _ptr(b_k), _ptr(w_v), _ptr(b_v), _ptr(w_o), _ptr(b_o), B, Lq, Lk, d, h,
        ctypes.byref(mask) if mask is not None else None, _ptr(out), _ptr(p_attn), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def mha_qkv_projection(query, key, value, w_q, b_q, w_k, b_k, w_v, b_v, h, *, workspace, stream=None):
    B, Lq, d = query.shape
    Lk = key.shape[1]
    _check(load().mha_qkv_projection(
        _dtype_code(query), _ptr(query), _ptr(key), _ptr(value), _ptr(w_q), _ptr(b_q), _ptr(w_k),
        _ptr(b_k), _ptr(w_v), _ptr(b_v), B, Lq, Lk, d, h, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def mha_attention_core(dt: int, B, Lq, Lk, d_model, h, *, workspace, mask=None, p_attn=None, stream=None):
    _check(load().mha_attention_core(
        dt, B, Lq, Lk, d_model, h, ctypes.byref(mask) if mask is not None else None, _ptr(p_attn),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def mha_output_projection(w_o, b_o, B, Lq, Lk, h, *, out, workspace, stream=None):
    d = w_o.shape[0]
    _check(load().mha_output_projection(
        _dtype_code(w_o), _ptr(w_o), _ptr(b_o), B, Lq, Lk, d, h, _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def host_staging_size(dt: int, B, Lq, Lk, d_model, kv_distinct: bool, q_distinct: bool) -> int:
    return int(load().mha_host_staging_size(dt, B, Lq, Lk, d_model, int(kv_distinct), int(q_distinct)))


def mha_forward_host(h_query, h_key, h_value, w_q, b_q, w_k, b_k, w_v, b_v, w_o, b_o, h, *, h_out,
                     staging, workspace, mask=None, stream=None):
    """Host activations (pinned CPU tensors) in and out; weights and workspace on the device."""
    B, Lq, d = h_query.shape
    Lk = h_key.shape[1]
    _check(load().mha_forward_host(
        _dtype_code(h_query), _ptr(h_query), _ptr(h_key), _ptr(h_value), _ptr(w_q), _ptr(b_q),
        _ptr(w_k), _ptr(b_k), _ptr(w_v), _ptr(b_v), _ptr(w_o), _ptr(b_o), B, Lq, Lk, d, h,
        ctypes.byref(mask) if mask is not None else None, _ptr(h_out), _ptr(staging),
        staging.numel() * staging.element_size(), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def mha_forward_noalloc(query, key, value, w_q, b_q, w_k, b_k, w_v, b_v, w_o, b_o, h, *, out,
                        mask=None, p_attn=None, stream=None):
    """mha_forward without a workspace: uses the library's fixed scratch (see include/mha.h)."""
    B, Lq, d = query.shape
    Lk = key.shape[1]
    _check(load().mha_forward_noalloc(
        _dtype_code(query), _ptr(query), _ptr(key), _ptr(value), _ptr(w_q), _ptr(b_q), _ptr(w_k),
        _ptr(b_k), _ptr(w_v), _ptr(b_v), _ptr(w_o), _ptr(b_o), B, Lq, Lk, d, h,
        ctypes.byref(mask) if mask is not None else None, _ptr(out), _ptr(p_attn), _stream(stream)))


def decode_workspace_size(B: int, d_model: int, h: int, L_max: int) -> int:
    return int(load().mha_decode_workspace_size(B, d_model, h, L_max))


def mha_kv_cache_prefill(x, w_k, b_k, w_v, b_v, h, *, k_cache, v_cache, stream=None):
    """Project x [B, T, d_model] into positions 0..T-1 of the caches [B, h, L_max, 64]."""
    B, T, d = x.shape
    _check(load().mha_kv_cache_prefill(
        _dtype_code(x), _ptr(x), _ptr(w_k), _ptr(b_k), _ptr(w_v), _ptr(b_v), B, T, d, h, _ptr(k_cache),
        _ptr(v_cache), k_cache.shape[2], _stream(stream)))


def mha_decode_step(x_new, w_q, b_q, w_k, b_k, w_v, b_v, w_o, b_o, h, *, k_cache, v_cache, cache_len, out,
                    workspace, stream=None):
    """One decoding step: x_new [B, d_model] -> out [B, d_model]; appends to the caches, bumps cache_len."""
    B, d = x_new.shape
    _check(load().mha_decode_step(
        _dtype_code(x_new), _ptr(x_new), _ptr(w_q), _ptr(b_q), _ptr(w_k), _ptr(b_k), _ptr(w_v), _ptr(b_v),
        _ptr(w_o), _ptr(b_o), B, d, h, _ptr(k_cache), _ptr(v_cache), _ptr(cache_len), k_cache.shape[2],
        _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


LN_UNBIASED_STD, LN_TORCH = 0, 1


def sublayer_workspace_size(dt: int, B: int, L: int, L_mem: int, d_model: int, h: int) -> int:
    return int(load().mha_sublayer_workspace_size(dt, B, L, L_mem, d_model, h))


def mha_sublayer_forward(x, ln_gain, ln_bias, ln_eps, ln_kind, w_q, b_q, w_k, b_k, w_v, b_v, w_o, b_o, h, *,
                         out, workspace, memory=None, mask=None, stream=None):
    """out = x + MHA(LayerNorm(x), kv, kv, mask), kv = LayerNorm(x) or memory (CUDA tensors)."""
    B, L, d = x.shape
    L_mem = memory.shape[1] if memory is not None else 0
    _check(load().mha_sublayer_forward(
        _dtype_code(x), _ptr(x), _ptr(memory), _ptr(ln_gain), _ptr(ln_bias), float(ln_eps), int(ln_kind),
        _ptr(w_q), _ptr(b_q), _ptr(w_k), _ptr(b_k), _ptr(w_v), _ptr(b_v), _ptr(w_o), _ptr(b_o), B, L, L_mem, d, h,
        ctypes.byref(mask) if mask is not None else None, _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def ffn_workspace_size(dt: int, B: int, L: int, d_model: int, d_ff: int) -> int:
    return int(load().mha_ffn_workspace_size(dt, B, L, d_model, d_ff))


def mha_ffn_forward(x, w_1, b_1, w_2, b_2, *, out, workspace, stream=None):
    """Position-wise FFN: out = max(0, x W_1^T + b_1) W_2^T + b_2 (CUDA tensors)."""
    B, L, d = x.shape
    d_ff = w_1.shape[0]
    _check(load().mha_ffn_forward(
        _dtype_code(x), _ptr(x), _ptr(w_1), _ptr(b_1), _ptr(w_2), _ptr(b_2), B, L, d, d_ff, _ptr(out),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


# ------------------------------------------------------------------ serving operators
MHA_PAGED_BAD_PAGE = 0x501
MHA_CODE_E4M3, MHA_CODE_INT8 = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_BASE, ROPE_BANDED, ROPE_RAMP = range(5)


# These calls are made once a layer and token, so what a call costs on the host counts. Each goes to its namesake in
# _front (csrc/front.cpp), which checks and makes the call in native code; where that finds anything out of order, or is
# not built, the Python below checks again, names the fault, or makes the call through ctypes.
_pack_strides = struct.Struct("4q").pack        # mha_strides_t is the first three
_pack_mask = struct.Struct("@2i3P").pack        # mha_span_mask_t


def _torch():
    """torch's entry points used below, looked up once: (current device, current stream handle of a device)."""
    global _current_device, _raw_stream, _bf16, _f32, _i32, _i64, _e4m3, _i8, _front
    import torch
    torch.cuda.init()
    try:
        from . import _front as front
        if torch.__version__.split("+")[0] == front.torch_version.split("+")[0]:
            front.set_library(*(ctypes.cast(getattr(load(), n), ctypes.c_void_p).value for n in _FRONT))
            _front = front
    except ImportError:
        pass
    if _front is None:
        warnings.warn("_front.so is not built for this torch: serving calls cost more on the host")
    _bf16, _f32, _i32, _i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
    _e4m3, _i8 = torch.float8_e4m3fn, torch.int8
    _current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


_current_device = _raw_stream = _bf16 = _f32 = _i32 = _i64 = _e4m3 = _i8 = _front = None
_FRONT = ("mha_rotary", "mha_paged_append", "mha_paged_attention", "mha_document_spans", "mha_attention", "mha_rmsnorm",
          "mha_paged_resize", "mha_coded_append", "mha_coded_attention")


def _here(t):
    """Index of t's device, which has to be the current CUDA device: work is enqueued there."""
    if not t.is_cuda:
        raise ValueError(f"tensors must be on the current CUDA device, not on {t.device}")
    if _current_device is None:
        _torch()
    dev = t.get_device()
    if dev != _current_device():
        raise ValueError(f"tensors must be on the current CUDA device, not on {t.device}")
    return dev


def _code(dtype):
    if dtype is _bf16:
        return MHA_BF16
    if dtype is _f32:
        return MHA_F32
    raise TypeError(f"unsupported dtype {dtype}: use torch.bfloat16 or torch.float32")


def _want(t, name, dtype, shape, dev):
    """t is a CUDA tensor of this dtype, shape and device."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")


def _view(t, name, dtype, shape, dev):
    """(pointer, packed strides) of a [B, L, H, d] tensor of this dtype, shape and device, its last dimension adjacent."""
    st = t.stride()
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _want(t, name, dtype, shape, dev)
    if st[3] != 1 and shape[3] != 1:
        raise ValueError(f"the last dimension of {name} must be adjacent (stride {st[3]})")
    return t.data_ptr(), _pack_strides(*st)


def _ints(t, name, shape, dev):
    """Pointer of a contiguous int32 tensor, or None."""
    if t is None:
        return None
    if t.dtype is not _i32 or t.shape != shape or t.get_device() != dev:
        _want(t, name, _i32, shape, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _floats(t, name):
    dev = _here(t)
    _want(t, name, _f32, (t.numel(),), dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: int = ROPE_PLAIN, factor: float = 1.0,
                       original_length: float = 0.0, low: float = 1.0, high: float = 4.0):
    """(inv_freq, scale): the rot_dim / 2 frequencies (a CPU fp32 tensor) and the factor of cos and sin
    for a scaled context."""
    import torch
    table = torch.empty(max(rot_dim // 2, 1), dtype=torch.float32)
    scale = ctypes.c_float(1.0)
    _check(load().mha_rotary_frequencies(table.data_ptr(), ctypes.addressof(scale), rot_dim, base, scaling, factor,
                                         original_length, low, high))
    return table, scale.value


def make_rotary(inv_freq, interleaved: bool = False, scale: float = 1.0):
    """Rotary description: inv_freq is a CUDA fp32 tensor of rot_dim / 2 frequencies. Holds a reference to it."""
    r = RotaryT(_floats(inv_freq, "inv_freq"), 2 * inv_freq.numel(), int(interleaved), scale)
    r._tensors = inv_freq
    r._ref = ctypes.byref(r)
    r._device = inv_freq.get_device()
    r._native = struct.pack("Pq", ctypes.addressof(r), r._device)
    return r


def make_paged_cache(k_pages, v_pages, block_table):
    """Cache description: k_pages and v_pages [n_pages, page_size, h_kv, d_k] with the same strides (any order of
    the dimensions in memory but the last), block_table int32 [B, max_pages]. Holds references to the three."""
    dev = _here(k_pages)
    n, size, h_kv, d = k_pages.shape
    _code(k_pages.dtype)
    _want(v_pages, "v_pages", k_pages.dtype, k_pages.shape, dev)
    if k_pages.stride() != v_pages.stride():
        raise ValueError("k_pages and v_pages must have the same strides")
    if k_pages.stride(3) != 1 and d != 1:
        raise ValueError("the last dimension of the pages must be adjacent")
    _want(block_table, "block_table", _i32, block_table.shape, dev)
    if block_table.dim() != 2 or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be [B, max_pages] with adjacent rows")
    c = PagedCacheT(k_pages.data_ptr(), v_pages.data_ptr(), *k_pages.stride()[:3], n, size, block_table.data_ptr(),
                    block_table.stride(0), block_table.shape[1])
    c._tensors = (k_pages, v_pages, block_table)
    c._ref = ctypes.byref(c)
    c._heads = h_kv
    c._for = (block_table.shape[0], d, k_pages.dtype, dev)
    c._native = struct.pack("P5q", ctypes.addressof(c), block_table.shape[0], d, _code(k_pages.dtype), dev, h_kv)
    return c


_CODED = 2       # in place of a dtype code, in what the native front reads


def make_coded_cache(k_pages, v_pages, k_scales, v_scales, block_table):
    """Description of a cache in 8 bits: pages as for make_paged_cache, torch.float8_e4m3fn or torch.int8; the scales fp32
    [n_pages, blocks of a page, h_kv], contiguous. Holds references to the five."""
    dev = _here(k_pages)
    n, size, h_kv, d = k_pages.shape
    if k_pages.dtype is not _e4m3 and k_pages.dtype is not _i8:
        raise TypeError(f"unsupported dtype {k_pages.dtype} of coded pages: use torch.float8_e4m3fn or torch.int8")
    _want(v_pages, "v_pages", k_pages.dtype, k_pages.shape, dev)
    if k_pages.stride() != v_pages.stride():
        raise ValueError("k_pages and v_pages must have the same strides")
    if k_pages.stride(3) != 1 and d != 1:
        raise ValueError("the last dimension of the pages must be adjacent")
    _want(block_table, "block_table", _i32, block_table.shape, dev)
    if block_table.dim() != 2 or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be [B, max_pages] with adjacent rows")
    if k_scales.dim() != 3:
        raise ValueError("k_scales must be [n_pages, blocks of a page, h_kv]")
    blocks = k_scales.shape[1]
    if blocks < 1 or size % blocks != 0:
        raise ValueError(f"k_scales has {blocks} blocks a page, which do not divide its {size} slots")
    for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
        _want(t, name, _f32, (n, blocks, h_kv), dev)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    pages = PagedCacheT(k_pages.data_ptr(), v_pages.data_ptr(), *k_pages.stride()[:3], n, size, block_table.data_ptr(),
                        block_table.stride(0), block_table.shape[1])
    c = CodedCacheT(pages, MHA_CODE_INT8 if k_pages.dtype is _i8 else MHA_CODE_E4M3, size // blocks, k_scales.data_ptr(),
                    v_scales.data_ptr())
    c._tensors = (k_pages, v_pages, k_scales, v_scales, block_table)
    c._ref = ctypes.byref(c)
    c._heads = h_kv
    c._for = (block_table.shape[0], d, "coded", dev)
    c._native = struct.pack("P5q", ctypes.addressof(c), block_table.shape[0], d, _CODED, dev, h_kv)
    return c


def make_scores(scale: float = 0.0, cap: float = 0.0, slopes=None):
    """Score description: scale (0: 1 / sqrt(d_k)), tanh cap (0: none), slopes a CUDA fp32 [h] or None."""
    s = ScoresT(scale, cap, None if slopes is None else _floats(slopes, "slopes"))
    s._tensors = slopes
    s._ref = ctypes.byref(s)
    s._for = None if slopes is None else (slopes.numel(), slopes.get_device())
    s._native = struct.pack("P2q", ctypes.addressof(s), *(s._for or (-1, -1)))
    return s


class _SpanMask:
    __slots__ = ("causal", "q_offset", "tensors")


def make_span_mask(causal=False, q_offset=0, key_valid_lens=None, prefix_lens=None, doc_spans=None):
    """Mask description for mha_attention. Holds references to the tensors (CUDA int32)."""
    m = _SpanMask()
    m.causal, m.q_offset, m.tensors = (1 if causal else 0), q_offset, (key_valid_lens, prefix_lens, doc_spans)
    return m


def _scores_ref(scores, h, dev):
    if scores is None:
        return None
    if scores._for is not None and scores._for != (h, dev):
        raise ValueError(f"slopes has {scores._for[0]} entries on cuda:{scores._for[1]}, not {h} on cuda:{dev}")
    return scores._ref


def _rotary_ref(rotary, dev):
    if rotary._device != dev:
        raise ValueError(f"inv_freq is on cuda:{rotary._device}, not on cuda:{dev}")
    return rotary._ref


def mha_rotary(q, *, rotary, q_out, k=None, k_out=None, positions=None, stream=None):
    """Turn q [B, T, h, d_k] into q_out and k [B, T, h_kv, d_k] into k_out (an output may be its input)."""
    if _front is not None and _front.rotary(q, rotary, q_out, k, k_out, positions, stream):
        return
    dev = _here(q)
    dtype, shape = q.dtype, q.shape
    B, T, h, d = shape
    qp, qs = _view(q, "q", dtype, shape, dev)
    qop, qos = _view(q_out, "q_out", dtype, shape, dev)
    kp = ks = kop = kos = None
    h_kv = 0
    if k is not None:
        h_kv = k.shape[2]
        k_shape = (B, T, h_kv, d)
        kp, ks = _view(k, "k", dtype, k_shape, dev)
        kop, kos = _view(k_out, "k_out", dtype, k_shape, dev)
    st = (_lib or load()).mha_rotary(
        _code(dtype), qp, qs, qop, qos, kp, ks, kop, kos, B, T, h, h_kv, d, _ints(positions, "positions", (B, T), dev),
        _rotary_ref(rotary, dev), _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _check(st)


def mha_paged_append(k, v, start, *, cache, q=None, q_out=None, k_out=None, new_lens=None, rotary=None, stream=None):
    """Append k, v [B, T, h_kv, d_k] to the cache at positions start[b] + t, turning k (and q into q_out)."""
    if _front is not None and _front.paged_append(k, v, start, cache, q, q_out, k_out, new_lens, rotary, stream):
        return
    _append((_lib or load()).mha_paged_append, k.dtype, k, v, start, cache, q, q_out, k_out, new_lens, rotary, stream)


def mha_coded_append(k, v, start, *, cache, q=None, q_out=None, k_out=None, new_lens=None, rotary=None, stream=None):
    """mha_paged_append into a cache in 8 bits (make_coded_cache)."""
    if _front is not None and _front.coded_append(k, v, start, cache, q, q_out, k_out, new_lens, rotary, stream):
        return
    _append((_lib or load()).mha_coded_append, "coded", k, v, start, cache, q, q_out, k_out, new_lens, rotary, stream)


def _append(entry, kind, k, v, start, cache, q, q_out, k_out, new_lens, rotary, stream):
    dev = _here(k)
    dtype, shape = k.dtype, k.shape
    B, T, h_kv, d = shape
    if cache._for != (B, d, kind, dev) or cache._heads != h_kv:
        raise ValueError("the cache's batch, heads, head width, dtype or device differ from k's")
    kp, ks = _view(k, "k", dtype, shape, dev)
    vp, vs = _view(v, "v", dtype, shape, dev)
    qp = qs = qop = qos = kop = kos = None
    h = 0
    if q is not None:
        h = q.shape[2]
        q_shape = (B, T, h, d)
        qp, qs = _view(q, "q", dtype, q_shape, dev)
        qop, qos = _view(q_out, "q_out", dtype, q_shape, dev)
    if k_out is not None:
        kop, kos = _view(k_out, "k_out", dtype, shape, dev)
    if start is None:
        raise ValueError("start must be an int32 tensor [B]")
    one = (B,)
    st = entry(
        _code(dtype), qp, qs, qop, qos, kp, ks, kop, kos, vp, vs, B, T, h, h_kv, d, _ints(start, "start", one, dev),
        _ints(new_lens, "new_lens", one, dev), None if rotary is None else _rotary_ref(rotary, dev), cache._ref,
        _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _check(st)


def paged_attention_workspace_size(dt: int, B: int, h: int, h_kv: int, d_k: int) -> int:
    return int(load().mha_paged_attention_workspace_size(dt, B, h, h_kv, d_k))


def mha_paged_attention(q, kv_lens, *, cache, out, workspace, scores=None, stream=None):
    """Attention of one new token a sequence, q [B, h, d_k], over the kv_lens[b] cached positions -> out."""
    if _front is not None and _front.paged_attention(q, kv_lens, cache, out, workspace, scores, stream):
        return
    _decode((_lib or load()).mha_paged_attention, q.dtype, q, kv_lens, cache, out, workspace, scores, stream)


def coded_attention_workspace_size(dt: int, B: int, h: int, h_kv: int, d_k: int) -> int:
    return int(load().mha_coded_attention_workspace_size(dt, B, h, h_kv, d_k))


def mha_coded_attention(q, kv_lens, *, cache, out, workspace, scores=None, stream=None):
    """mha_paged_attention over a cache in 8 bits (make_coded_cache)."""
    if _front is not None and _front.coded_attention(q, kv_lens, cache, out, workspace, scores, stream):
        return
    _decode((_lib or load()).mha_coded_attention, "coded", q, kv_lens, cache, out, workspace, scores, stream)


def _decode(entry, kind, q, kv_lens, cache, out, workspace, scores, stream):
    dev = _here(q)
    dtype, shape = q.dtype, q.shape
    B, h, d = shape
    _want(out, "out", dtype, shape, dev)
    if cache._for != (B, d, kind, dev):
        raise ValueError("the cache's batch, head width, dtype or device differ from q's")
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on cuda:{dev}")
    if kv_lens is None:
        raise ValueError("kv_lens must be an int32 tensor [B]")
    qb, qh, qd = q.stride()
    ob, oh, od = out.stride()
    if qd != 1 or od != 1:
        raise ValueError("the last dimension of q and out must be adjacent")
    st = entry(
        _code(dtype), q.data_ptr(), _pack_strides(qb, 0, qh, 1), out.data_ptr(), _pack_strides(ob, 0, oh, 1), B, h,
        cache._heads, d, _ints(kv_lens, "kv_lens", (B,), dev), _scores_ref(scores, h, dev), cache._ref,
        workspace.data_ptr(), workspace.nbytes, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _check(st)


def mha_paged_resize(held, want, *, block_table, page_size: int, free_pages, free_count, lens, new_lens=None, slots=None,
                     stream=None):
    """Take the sequences from held to want positions (int32 [B]): pages move between block_table int32 [B, max_pages] and
    the stack free_pages int32 [n_pages], of which free_count int32 [1] are free. lens and new_lens int32 [B] get the positions
    reached and how many are new, slots int64 [B, T] the new tokens' slots."""
    if _front is not None and _front.paged_resize(held, want, block_table, page_size, free_pages, free_count, lens, new_lens, slots,
                                                  stream):
        return
    dev = _here(held)
    B, = held.shape
    one = (B,)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    max_pages = block_table.shape[1]
    _want(block_table, "block_table", _i32, (B, max_pages), dev)
    if max_pages > 1 and block_table.stride(1) != 1:
        raise ValueError("the rows of block_table must be adjacent")
    sp, T = None, 0
    if slots is not None:
        if slots.dim() != 2:
            raise ValueError("slots must be [B, T]")
        T = slots.shape[1]
        _want(slots, "slots", _i64, (B, T), dev)
        if not slots.is_contiguous():
            raise ValueError("slots must be contiguous")
        sp = slots.data_ptr()
    st = (_lib or load()).mha_paged_resize(
        _ints(held, "held", one, dev), _ints(want, "want", one, dev), B, page_size, block_table.data_ptr(), block_table.stride(0),
        max_pages, _ints(free_pages, "free_pages", (free_pages.numel(),), dev), free_pages.numel(),
        _ints(free_count, "free_count", (1,), dev), _ints(lens, "lens", one, dev), _ints(new_lens, "new_lens", one, dev), T, sp,
        _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _check(st)


def mha_document_spans(doc_ids, *, spans, stream=None):
    """spans int32 [B, L, 2] of the documents in doc_ids int32 [B, L] (one run each; < 0 is padding)."""
    if _front is not None and _front.document_spans(doc_ids, spans, stream):
        return
    dev = _here(doc_ids)
    B, L = doc_ids.shape
    st = (_lib or load()).mha_document_spans(_ints(doc_ids, "doc_ids", (B, L), dev), B, L,
                                             _ints(spans, "spans", (B, L, 2), dev), _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _check(st)


def mha_attention(q, k, v, *, out, scores=None, mask=None, stream=None):
    """Attention of q [B, L_q, h, d_k] over k, v [B, L_k, h_kv, d_k] -> out [B, L_q, h, d_k]."""
    if _front is not None and _front.attention(q, k, v, out, scores, mask, stream):
        return
    dev = _here(q)
    dtype, shape = q.dtype, q.shape
    B, Lq, h, d = shape
    Lk, h_kv = k.shape[1], k.shape[2]
    k_shape = (B, Lk, h_kv, d)
    qp, qs = _view(q, "q", dtype, shape, dev)
    kp, ks = _view(k, "k", dtype, k_shape, dev)
    vp, vs = _view(v, "v", dtype, k_shape, dev)
    op, os_ = _view(out, "out", dtype, shape, dev)
    ref = None
    if mask is not None:
        valid, prefix, spans = mask.tensors
        ref = _pack_mask(mask.causal, mask.q_offset, _ints(valid, "key_valid_lens", (B,), dev) or 0,
                         _ints(prefix, "prefix_lens", (B,), dev) or 0, _ints(spans, "doc_spans", (B, Lq, 2), dev) or 0)
    st = (_lib or load()).mha_attention(
        _code(dtype), qp, qs, kp, ks, vp, vs, op, os_, B, Lq, Lk, h, h_kv, d, _scores_ref(scores, h, dev), ref,
        _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _check(st)


def _rows(t, name, dtype, shape, dev):
    """(pointer, row stride) of a [rows, d] tensor of this dtype, shape and device with adjacent rows."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _want(t, name, dtype, shape, dev)
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] != 1:
        raise ValueError(f"the rows of {name} must be adjacent")
    return t.data_ptr(), s0


def mha_rmsnorm(x, gain, eps: float, *, y, residual=None, sum_out=None, scales=None, stream=None):
    """y = gain * z / rms(z), z = x + residual (written to sum_out), rows of length d = x.shape[-1], x [rows, d].
    y has x's dtype, or torch.float8_e4m3fn with scales fp32 [rows, groups] (one group: the row)."""
    if _front is not None and _front.rmsnorm(x, gain, eps, y, residual, sum_out, scales, stream):
        return
    dev = _here(x)
    dtype, shape = x.dtype, x.shape
    rows, d = shape
    xp, xs = _rows(x, "x", dtype, shape, dev)
    group = rs = zs = 0
    rp = zp = gp = cp = None
    if scales is None:
        yp, ys = _rows(y, "y", dtype, shape, dev)
    else:
        yp, ys = _rows(y, "y", _e4m3, shape, dev)
        groups = scales.shape[1]
        _want(scales, "scales", _f32, (rows, groups), dev)
        if not scales.is_contiguous() or groups < 1 or d % groups != 0:
            raise ValueError("scales must be contiguous [rows, groups] with groups dividing d")
        if groups > 1:
            group = d // groups
        cp = scales.data_ptr()
    if residual is not None:
        rp, rs = _rows(residual, "residual", dtype, shape, dev)
    if sum_out is not None:
        if residual is None:
            raise ValueError("sum_out needs a residual")
        zp, zs = _rows(sum_out, "sum_out", dtype, shape, dev)
    if gain is not None:
        if gain.dtype is not dtype or gain.shape != (d,) or gain.get_device() != dev or not gain.is_contiguous():
            _want(gain, "gain", dtype, (d,), dev)
            raise ValueError("gain must be contiguous")
        gp = gain.data_ptr()
    st = (_lib or load()).mha_rmsnorm(_code(dtype), xp, xs, rp, rs, zp, zs, gp, eps, rows, d, yp, ys, cp, group,
                                      _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _check(st)


def mha_selftest_wait_timeout(stream=None):
    """Enqueue the diagnostic kernel whose bounded pipeline wait runs out (it records
    MHA_SELFTEST_WAIT_CODE in the device status word)."""
    _check(load().mha_selftest_wait_timeout(_stream(stream)))


def mha_check_device_status(reset: bool = True) -> int:
    """Synchronise and return the kernels' bounded-wait status word (0 = clean)."""
    v = ctypes.c_int(0)
    _check(load().mha_check_device_status(ctypes.byref(v), int(reset)))
    return v.value


def version() -> str:
    return load().mha_version().decode()
