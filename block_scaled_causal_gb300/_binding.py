"""ctypes binding of libbsc.so: argument marshalling only (every step runs in the CUDA library).

The functions keep the C names of include/bsc.h.  Tensors are torch CUDA tensors; outputs are
allocated with torch when not given.  A missing library raises at import time: there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct

import torch

from . import build as _build

BSHD = 0
SBHD = 1

BSC_OK = 0
BSC_ERR_DEVICE_TIMEOUT = 6


def _load():
    path = _build.LIB_PATH
    if not os.path.exists(path):
        raise ImportError("libbsc.so is not built (%s); run `python -m block_scaled_causal_gb300.build`" % path)
    lib = ctypes.CDLL(path)
    vp, i32, u8p = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
    lib.bsc_abi_version.restype = i32
    lib.bsc_status_string.restype = ctypes.c_char_p
    lib.bsc_status_string.argtypes = [i32]
    for name in ("mxfp8_quantize_qk_rowwise", "mxfp8_quantize_v_colwise", "v_token_normalize"):
        f = getattr(lib, name)
        f.restype = i32
        f.argtypes = [vp, i32, i32, i32, i32, i32, u8p, u8p, vp]
    lib.mxfp8_quantize_v_fused.restype = i32
    lib.mxfp8_quantize_v_fused.argtypes = [vp, i32, i32, i32, i32, i32, u8p, u8p, u8p, u8p, vp]
    lib.mxfp8_causal_attn_fwd.restype = i32
    lib.mxfp8_causal_attn_fwd.argtypes = [ctypes.POINTER(AttnFwdParams), vp]
    lib.mxfp8_quantize_qkv.restype = i32
    lib.mxfp8_quantize_qkv.argtypes = [ctypes.POINTER(QkvQuantParams), vp]
    lib.mxfp8_quantize.restype = i32
    lib.mxfp8_quantize.argtypes = [ctypes.POINTER(QuantParams), vp]
    lib.bf16_attn_bwd.restype = i32
    lib.bf16_attn_bwd.argtypes = [ctypes.POINTER(AttnBwdParams), vp]
    lib.bf16_attn_bwd_static.restype = i32
    lib.bf16_attn_bwd_static.argtypes = [ctypes.POINTER(AttnBwdParams), vp]
    lib.bf16_attn_bwd_static_capacity.restype = ctypes.c_size_t
    lib.bf16_attn_bwd_static_capacity.argtypes = []
    lib.bf16_attn_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.bf16_attn_bwd_workspace_bytes.argtypes = [i32, i32, i32, i32]
    for name, params in (("mx_cache_write", CacheWriteParams), ("mx_cache_read", CacheReadParams),
                         ("mx_cache_attn", CacheAttnParams)):
        f = getattr(lib, name)
        f.restype = i32
        f.argtypes = [ctypes.POINTER(params), vp]
    lib.mx_cache_attn_workspace_bytes.restype = ctypes.c_size_t
    lib.mx_cache_attn_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, ctypes.c_longlong]
    for name, params in (("rms_norm", RmsNormParams), ("rms_norm_bwd", RmsNormBwdParams), ("rope", RopeParams),
                         ("mxfp8_rope_quantize_qk", RopeQuantParams), ("mx_cache_write_rope", CacheWriteRopeParams),
                         ("mx_cache_bounds", CacheBoundsParams), ("mx_cache_sparse_attn", CacheSparseAttnParams)):
        f = getattr(lib, name)
        f.restype = i32
        f.argtypes = [ctypes.POINTER(params), vp]
    lib.rms_norm_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.rms_norm_bwd_workspace_bytes.argtypes = [ctypes.c_longlong, i32]
    lib.mx_cache_sparse_attn_workspace_bytes.restype = ctypes.c_size_t
    lib.mx_cache_sparse_attn_workspace_bytes.argtypes = [i32] * 8
    lib.mxfp8_dequantize.restype = i32
    lib.mxfp8_dequantize.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, vp, vp]
    lib.bsc_rope_turns.restype = i32
    lib.bsc_rope_turns.argtypes = [ctypes.POINTER(RopeConfig), vp, ctypes.POINTER(ctypes.c_float)]
    lib.bsc_rope_magnitude.restype = ctypes.c_double
    lib.bsc_rope_magnitude.argtypes = [ctypes.POINTER(RopeConfig)]
    lib.bsc_read_device_status.restype = i32
    lib.bsc_read_device_status.argtypes = [vp, vp]
    return lib


class AttnFwdParams(ctypes.Structure):
    """Mirror of bsc_attn_fwd_params."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("q_sc", ctypes.c_void_p),
        ("k", ctypes.c_void_p), ("k_sc", ctypes.c_void_p),
        ("v_t", ctypes.c_void_p), ("v_sc", ctypes.c_void_p),
        ("vtn", ctypes.c_void_p), ("vtn_sc", ctypes.c_void_p),
        ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("B", ctypes.c_int), ("S", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
        ("D", ctypes.c_int), ("layout", ctypes.c_int), ("softmax_scale", ctypes.c_float),
        ("p_terms", ctypes.c_int), ("leaky", ctypes.c_int),
        ("dev_status", ctypes.c_void_p), ("wait_timeout_ms", ctypes.c_uint32),
        ("debug_stall", ctypes.c_int),
        ("o_e4m3", ctypes.c_void_p), ("o_sc", ctypes.c_void_p),
    ]


class QuantParams(ctypes.Structure):
    """Mirror of bsc_quant_params."""
    _fields_ = [
        ("kind", ctypes.c_int), ("x", ctypes.c_void_p),
        ("B", ctypes.c_int), ("S", ctypes.c_int), ("H", ctypes.c_int), ("D", ctypes.c_int),
        ("layout", ctypes.c_int), ("rule", ctypes.c_int),
        ("e4m3", ctypes.c_void_p), ("sc", ctypes.c_void_p),
        ("vtn_e4m3", ctypes.c_void_p), ("vtn_sc", ctypes.c_void_p),
    ]


class QkvQuantParams(ctypes.Structure):
    """Mirror of bsc_qkv_quant_params."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("B", ctypes.c_int), ("S", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("layout", ctypes.c_int), ("rule", ctypes.c_int),
        ("q_e4m3", ctypes.c_void_p), ("q_sc", ctypes.c_void_p), ("k_e4m3", ctypes.c_void_p), ("k_sc", ctypes.c_void_p),
        ("v_e4m3_t", ctypes.c_void_p), ("v_sc", ctypes.c_void_p),
        ("vtn_e4m3", ctypes.c_void_p), ("vtn_sc", ctypes.c_void_p),
    ]


QUANT_ROWWISE, QUANT_V_COLWISE, QUANT_V_TOKEN_NORM, QUANT_V_FUSED = 0, 1, 2, 3
SCALE_FLOOR, SCALE_CEIL = 0, 1


class AttnBwdParams(ctypes.Structure):
    """Mirror of bsc_attn_bwd_params."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("q_sc", ctypes.c_void_p),
        ("k", ctypes.c_void_p), ("k_sc", ctypes.c_void_p),
        ("vtn", ctypes.c_void_p), ("vtn_sc", ctypes.c_void_p),
        ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("d_o", ctypes.c_void_p),
        ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p), ("dv", ctypes.c_void_p),
        ("B", ctypes.c_int), ("S", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
        ("D", ctypes.c_int), ("layout", ctypes.c_int), ("softmax_scale", ctypes.c_float),
        ("dev_status", ctypes.c_void_p), ("wait_timeout_ms", ctypes.c_uint32),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class CachePools(ctypes.Structure):
    """Mirror of bsc_mx_cache."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "k_sc", "v", "v_sc")] + \
        [(n, ctypes.c_longlong) for n in ("k_page_stride", "k_sc_page_stride", "v_page_stride", "v_sc_page_stride")] + \
        [(n, ctypes.c_int) for n in ("format", "num_pages", "page_size", "Hkv", "D")]


def _strides(*names):
    return [("%s_stride_%s" % (n, d), ctypes.c_longlong) for n in names for d in "bth"]


class CacheWriteParams(ctypes.Structure):
    """Mirror of bsc_mx_cache_write_params."""
    _fields_ = [("cache", CachePools), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + _strides("k", "v") + \
        [(n, ctypes.c_int) for n in ("B", "T", "dtype", "rule")] + \
        [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_longlong), ("max_pages", ctypes.c_int),
         ("seq_lens", ctypes.c_void_p), ("new_lens", ctypes.c_void_p), ("dev_status", ctypes.c_void_p)]


class CacheReadParams(ctypes.Structure):
    """Mirror of bsc_mx_cache_read_params."""
    _fields_ = [("cache", CachePools), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + _strides("k", "v") + \
        [(n, ctypes.c_int) for n in ("B", "T", "dtype")] + \
        [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_longlong), ("max_pages", ctypes.c_int),
         ("seq_lens", ctypes.c_void_p), ("starts", ctypes.c_void_p), ("dev_status", ctypes.c_void_p)]


class CacheAttnParams(ctypes.Structure):
    """Mirror of bsc_mx_cache_attn_params."""
    _fields_ = [("cache", CachePools), ("q", ctypes.c_void_p), ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p)] + \
        _strides("q", "o") + [(n, ctypes.c_int) for n in ("B", "T", "Hq", "dtype")] + \
        [("softmax_scale", ctypes.c_float), ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_longlong),
         ("max_pages", ctypes.c_int), ("seq_lens", ctypes.c_void_p), ("new_lens", ctypes.c_void_p),
         ("dev_status", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


_TABLE = [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_longlong), ("max_pages", ctypes.c_int),
          ("seq_lens", ctypes.c_void_p), ("new_lens", ctypes.c_void_p), ("dev_status", ctypes.c_void_p)]


def _row_strides(*names):
    return [(n + d, ctypes.c_longlong) for n in names for d in ("_stride", "_inner_stride")]


class RmsNormParams(ctypes.Structure):
    """Mirror of bsc_rms_norm_params."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "residual", "weight", "y", "sum", "rstd", "y_e4m3", "y_sc")] + \
        [("rows", ctypes.c_longlong)] + _row_strides("x", "residual", "y", "sum") + \
        [(n, ctypes.c_int) for n in ("inner", "N", "dtype", "weight_dtype", "rule")] + [("eps", ctypes.c_float)]


class RmsNormBwdParams(ctypes.Structure):
    """Mirror of bsc_rms_norm_bwd_params."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("dy", "s", "weight", "rstd", "d_sum", "dx", "dweight")] + \
        [("rows", ctypes.c_longlong)] + _row_strides("dy", "s", "d_sum", "dx") + \
        [(n, ctypes.c_int) for n in ("inner", "N", "dtype", "weight_dtype")] + \
        [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class RopeConfig(ctypes.Structure):
    """Mirror of bsc_rope_config."""
    _fields_ = [("rot", ctypes.c_int), ("scaling", ctypes.c_int)] + \
        [(n, ctypes.c_double) for n in ("base", "factor", "original_length", "low_turns", "high_turns")]


class RopeAngles(ctypes.Structure):
    """Mirror of bsc_rope_angles."""
    _fields_ = [("turns", ctypes.c_void_p), ("magnitude", ctypes.c_float), ("rot", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("magnitude_low", ctypes.c_float)]


_POSITIONS = [("positions", ctypes.c_void_p), ("position_stride_b", ctypes.c_longlong),
              ("position_stride_t", ctypes.c_longlong)]


class RopeParams(ctypes.Structure):
    """Mirror of bsc_rope_params."""
    _fields_ = [("angles", RopeAngles)] + [(n, ctypes.c_void_p) for n in ("q", "k", "q_out", "k_out")] + \
        _strides("q", "k", "q_out", "k_out") + _POSITIONS + \
        [(n, ctypes.c_int) for n in ("B", "T", "Hq", "Hkv", "D", "dtype", "inverse")]


class RopeQuantParams(ctypes.Structure):
    """Mirror of bsc_rope_quant_params."""
    _fields_ = [("angles", RopeAngles), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p)] + _strides("q", "k") + \
        [(n, ctypes.c_void_p) for n in ("q_e4m3", "q_sc", "k_e4m3", "k_sc")] + _POSITIONS + \
        [(n, ctypes.c_int) for n in ("B", "T", "Hq", "Hkv", "D", "dtype", "layout", "rule")]


class CacheWriteRopeParams(ctypes.Structure):
    """Mirror of bsc_mx_cache_write_rope_params."""
    _fields_ = [("cache", CachePools), ("angles", RopeAngles)] + [(n, ctypes.c_void_p) for n in ("q", "k", "v", "q_out")] + \
        _strides("q", "k", "v", "q_out") + [(n, ctypes.c_int) for n in ("B", "T", "Hq", "dtype", "rule")] + _TABLE


class CacheBoundsParams(ctypes.Structure):
    """Mirror of bsc_mx_cache_bounds_params."""
    _fields_ = [("cache", CachePools), ("codes", ctypes.c_void_p), ("exps", ctypes.c_void_p), ("B", ctypes.c_int),
                ("T", ctypes.c_int)] + _TABLE


class CacheSparseAttnParams(ctypes.Structure):
    """Mirror of bsc_mx_cache_sparse_attn_params."""
    _fields_ = [("cache", CachePools)] + [(n, ctypes.c_void_p) for n in ("codes", "exps", "q", "o", "lse", "blocks")] + \
        _strides("q", "o") + [(n, ctypes.c_int) for n in ("B", "T", "Hq", "dtype")] + [("softmax_scale", ctypes.c_float)] + \
        [(n, ctypes.c_int) for n in ("top", "first", "last")] + _TABLE + \
        [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


ROPE_PLAIN, ROPE_LINEAR, ROPE_BASE, ROPE_BY_PARTS = 0, 1, 2, 3

CACHE_MXFP8, CACHE_MXFP4 = 0, 1
_ACT = {torch.bfloat16: 0, torch.float16: 1}

lib = _load()


class BscError(RuntimeError):
    def __init__(self, status: int):
        super().__init__(lib.bsc_status_string(status).decode())
        self.status = status


def _check(status: int):
    if status != BSC_OK:
        raise BscError(status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _bshd_dims(x: torch.Tensor, layout: int):
    if x.dim() != 4:
        raise ValueError("expected a 4-D tensor")
    if layout == BSHD:
        B, S, H, D = x.shape
    else:
        S, B, H, D = x.shape
    return B, S, H, D


def _require(x: torch.Tensor, dtype, name):
    if not x.is_cuda or x.dtype != dtype or not x.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA %s tensor" % (name, dtype))


def mxfp8_quantize_qk_rowwise(x, layout=BSHD, out=None, out_sc=None, stream=None):
    """Returns (E4M3 bytes shaped like x, scales [B, H, S, D/32])."""
    _require(x, torch.bfloat16, "x")
    B, S, H, D = _bshd_dims(x, layout)
    out = torch.empty(x.shape, dtype=torch.uint8, device=x.device) if out is None else out
    out_sc = torch.empty((B, H, S, D // 32), dtype=torch.uint8, device=x.device) if out_sc is None else out_sc
    _check(lib.mxfp8_quantize_qk_rowwise(_ptr(x), B, S, H, D, layout, _ptr(out), _ptr(out_sc), _stream(stream)))
    return out, out_sc


def _v_outputs(v, B, S, H, D, col, tn):
    dev = v.device
    r = []
    if col:
        r += [torch.empty((B, H, D, S), dtype=torch.uint8, device=dev),
              torch.empty((B, H, S // 32, D), dtype=torch.uint8, device=dev)]
    if tn:
        r += [torch.empty(v.shape, dtype=torch.uint8, device=dev),
              torch.empty((B, H, S), dtype=torch.uint8, device=dev)]
    return r


def mxfp8_quantize_v_colwise(v, layout=BSHD, stream=None):
    """Returns (E4M3 bytes of V transposed [B, H, D, S], scales [B, H, S/32, D])."""
    _require(v, torch.bfloat16, "v")
    B, S, H, D = _bshd_dims(v, layout)
    vt, vsc = _v_outputs(v, B, S, H, D, True, False)
    _check(lib.mxfp8_quantize_v_colwise(_ptr(v), B, S, H, D, layout, _ptr(vt), _ptr(vsc), _stream(stream)))
    return vt, vsc


def v_token_normalize(v, layout=BSHD, stream=None):
    """Returns (E4M3 bytes shaped like v, token amplitudes [B, H, S])."""
    _require(v, torch.bfloat16, "v")
    B, S, H, D = _bshd_dims(v, layout)
    vtn, vtn_sc = _v_outputs(v, B, S, H, D, False, True)
    _check(lib.v_token_normalize(_ptr(v), B, S, H, D, layout, _ptr(vtn), _ptr(vtn_sc), _stream(stream)))
    return vtn, vtn_sc


def mxfp8_quantize_v_fused(v, layout=BSHD, out=None, stream=None):
    """Both V quantisations in one pass: (v_t, v_sc, vtn, vtn_sc)."""
    _require(v, torch.bfloat16, "v")
    B, S, H, D = _bshd_dims(v, layout)
    vt, vsc, vtn, vtn_sc = _v_outputs(v, B, S, H, D, True, True) if out is None else out
    _check(lib.mxfp8_quantize_v_fused(_ptr(v), B, S, H, D, layout, _ptr(vt), _ptr(vsc), _ptr(vtn), _ptr(vtn_sc),
                                      _stream(stream)))
    return vt, vsc, vtn, vtn_sc


def make_attn_params(q, q_sc, k, k_sc, v_t, v_sc, vtn, vtn_sc, o, lse, layout, softmax_scale, p_terms=2, leaky=0,
                     dev_status=None, wait_timeout_ms=0, debug_stall=0, o8=None, o_sc=None):
    B, S, Hq, D = _bshd_dims(q, layout)
    Hkv = _bshd_dims(k, layout)[2]
    return AttnFwdParams(q=q.data_ptr(), q_sc=q_sc.data_ptr(), k=k.data_ptr(), k_sc=k_sc.data_ptr(),
                         v_t=v_t.data_ptr(), v_sc=v_sc.data_ptr(),
                         vtn=0 if vtn is None else vtn.data_ptr(), vtn_sc=0 if vtn_sc is None else vtn_sc.data_ptr(),
                         o=0 if o is None else o.data_ptr(), lse=lse.data_ptr(), B=B, S=S, Hq=Hq, Hkv=Hkv, D=D,
                         layout=layout, softmax_scale=softmax_scale, p_terms=p_terms, leaky=leaky,
                         dev_status=0 if dev_status is None else dev_status.data_ptr(),
                         wait_timeout_ms=wait_timeout_ms, debug_stall=debug_stall,
                         o_e4m3=0 if o8 is None else o8.data_ptr(), o_sc=0 if o_sc is None else o_sc.data_ptr())


def mxfp8_causal_attn_fwd(q, q_sc, k, k_sc, v_t, v_sc, vtn, vtn_sc, layout=BSHD, softmax_scale=None, p_terms=2,
                          leaky=0, o=None, lse=None, dev_status=None, wait_timeout_ms=0, debug_stall=0,
                          stream=None, o8_out=False, bf16_out=True, o8=None, o_sc=None):
    """Leak-free causal MXFP8 attention forward on quantised operands.

    Returns (O bf16, LSE fp32); with o8_out=True, (O bf16 or None, LSE, O E4M3 bytes laid out like
    q, O scales [B, Hq, S, D/32]).  p_terms: E4M3 terms of P for the completed blocks (2: the
    tolerance-preserving default; 1: faster, one E4M3 rounding of P).
    """
    B, S, Hq, D = _bshd_dims(q, layout)
    if softmax_scale is None:
        softmax_scale = D ** -0.5
    if bf16_out:
        o = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device) if o is None else o
    else:
        o = None
    lse = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device) if lse is None else lse
    if o8_out:
        o8 = torch.empty(q.shape, dtype=torch.uint8, device=q.device) if o8 is None else o8
        o_sc = torch.empty((B, Hq, S, D // 32), dtype=torch.uint8, device=q.device) if o_sc is None else o_sc
    else:
        o8 = o_sc = None
    p = make_attn_params(q, q_sc, k, k_sc, v_t, v_sc, vtn, vtn_sc, o, lse, layout, softmax_scale, p_terms, leaky,
                         dev_status, wait_timeout_ms, debug_stall, o8, o_sc)
    _check(lib.mxfp8_causal_attn_fwd(ctypes.byref(p), _stream(stream)))
    return (o, lse, o8, o_sc) if o8_out else (o, lse)


def bsc_read_device_status(dev_status, stream=None):
    """Synchronises the stream; returns the library status for the device status word."""
    return lib.bsc_read_device_status(_ptr(dev_status), _stream(stream))


def _rotated_elsewhere(q, k, v, rope, stream):
    """Checks of what forward takes with a Rope (K and V are quantised by two calls, neither of which sees the other), and
    _elsewhere for it, so that all of its calls run and allocate in one place."""
    if rope is None:
        return None
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    if k.device != q.device or v.device != q.device:
        raise ValueError("q, k and v must be on one device")
    return _elsewhere_with(rope, q, stream)


def _operands(q, k, v, layout, token_norm, rope, positions, stream):
    """The eight operands of the attention: Q and K rotated where `rope` is given."""
    if rope is None:
        if positions is not None:
            raise ValueError("positions are for rope")
        return mxfp8_quantize_qkv(q, k, v, layout, token_norm=token_norm, stream=stream)
    qk = mxfp8_rope_quantize_qk(q, k, rope, positions, layout, stream=stream)
    if token_norm:
        return qk + tuple(mxfp8_quantize_v_fused(v, layout, stream=stream))
    return qk + tuple(mxfp8_quantize_v_colwise(v, layout, stream=stream)) + (None, None)


def forward(q, k, v, layout=BSHD, softmax_scale=None, p_terms=2, leaky=0, o=None, lse=None, stream=None,
            o8_out=False, bf16_out=True, rope=None, positions=None):
    """The whole hot path on bf16 inputs: quantise Q, K rowwise, V columnwise + token-normalised,
    then the leak-free causal attention forward.  Returns (O bf16, LSE fp32); `o` and `lse` may be
    given (laid out like q and [B, Hq, S]).  With o8_out=True the MXFP8 O is returned as well, as
    in mxfp8_causal_attn_fwd.  With `rope` (a Rope) Q and K are rotated on their way into MXFP8, at
    `positions` as in mxfp8_rope_quantize_qk; attention is causal by the tokens' order all the same."""
    there = _rotated_elsewhere(q, k, v, rope, stream)
    if there is not None:
        with there:
            return forward(q, k, v, layout, softmax_scale, p_terms, leaky, o, lse, None, o8_out, bf16_out, rope, positions)
    qq, qs, kq, ks, vt, vsc, vtn, vtn_sc = _operands(q, k, v, layout, not leaky, rope, positions, stream)
    return mxfp8_causal_attn_fwd(qq, qs, kq, ks, vt, vsc, vtn, vtn_sc, layout, softmax_scale, p_terms, leaky,
                                 o=o, lse=lse, stream=stream, o8_out=o8_out, bf16_out=bf16_out)


def bf16_attn_bwd_workspace_bytes(B, S, Hq, Hkv):
    """Bytes of scratch the backward needs (the C call of the same name)."""
    return int(lib.bf16_attn_bwd_workspace_bytes(B, S, Hq, Hkv))


def _bwd_params(q, q_sc, k, k_sc, vtn, vtn_sc, o, lse, do, layout, softmax_scale, dq, dk, dv, dev_status,
                wait_timeout_ms, workspace):
    B, S, Hq, D = _bshd_dims(q, layout)
    Hkv = _bshd_dims(k, layout)[2]
    if softmax_scale is None:
        softmax_scale = D ** -0.5
    _require(do, torch.bfloat16, "do")
    _require(o, torch.bfloat16, "o")
    dq = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device) if dq is None else dq
    dk = torch.empty(k.shape, dtype=torch.bfloat16, device=q.device) if dk is None else dk
    dv = torch.empty(k.shape, dtype=torch.bfloat16, device=q.device) if dv is None else dv
    p = AttnBwdParams(q=q.data_ptr(), q_sc=q_sc.data_ptr(), k=k.data_ptr(), k_sc=k_sc.data_ptr(),
                      vtn=vtn.data_ptr(), vtn_sc=vtn_sc.data_ptr(), o=o.data_ptr(), lse=lse.data_ptr(),
                      d_o=do.data_ptr(), dq=dq.data_ptr(), dk=dk.data_ptr(), dv=dv.data_ptr(), B=B, S=S, Hq=Hq,
                      Hkv=Hkv, D=D, layout=layout, softmax_scale=softmax_scale,
                      dev_status=0 if dev_status is None else dev_status.data_ptr(), wait_timeout_ms=wait_timeout_ms,
                      workspace=0 if workspace is None else workspace.data_ptr(),
                      workspace_bytes=0 if workspace is None else workspace.numel() * workspace.element_size())
    return p, dq, dk, dv


def bf16_attn_bwd(q, q_sc, k, k_sc, vtn, vtn_sc, o, lse, do, layout=BSHD, softmax_scale=None, dq=None, dk=None,
                  dv=None, dev_status=None, wait_timeout_ms=0, stream=None, workspace=None):
    """Backward on decoded operands (quantised Q, K and token-normalised V, the forward's O, LSE);
    returns (dQ, dK, dV) in bf16, laid out like q and k.  `workspace`: a device tensor of at least
    bf16_attn_bwd_workspace_bytes(B, S, Hq, Hkv) bytes, else one is allocated here."""
    if workspace is None:
        B, S, Hq, _ = _bshd_dims(q, layout)
        ws_bytes = bf16_attn_bwd_workspace_bytes(B, S, Hq, _bshd_dims(k, layout)[2])
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device)
    p, dq, dk, dv = _bwd_params(q, q_sc, k, k_sc, vtn, vtn_sc, o, lse, do, layout, softmax_scale, dq, dk, dv,
                                dev_status, wait_timeout_ms, workspace)
    _check(lib.bf16_attn_bwd(ctypes.byref(p), _stream(stream)))
    return dq, dk, dv


def bf16_attn_bwd_static(q, q_sc, k, k_sc, vtn, vtn_sc, o, lse, do, layout=BSHD, softmax_scale=None, dq=None,
                         dk=None, dv=None, dev_status=None, wait_timeout_ms=0, stream=None):
    """bf16_attn_bwd with the library's fixed device workspace (nothing allocated for scratch)."""
    p, dq, dk, dv = _bwd_params(q, q_sc, k, k_sc, vtn, vtn_sc, o, lse, do, layout, softmax_scale, dq, dk, dv,
                                dev_status, wait_timeout_ms, None)
    _check(lib.bf16_attn_bwd_static(ctypes.byref(p), _stream(stream)))
    return dq, dk, dv


def bf16_attn_bwd_static_capacity():
    """Bytes of the fixed workspace bf16_attn_bwd_static uses."""
    return int(lib.bf16_attn_bwd_static_capacity())


def forward_backward(q, k, v, do, layout=BSHD, softmax_scale=None, p_terms=2, stream=None, rope=None, positions=None):
    """Forward then the backward on decoded operands; returns (O, LSE, dQ, dK, dV).  With `rope` (see forward) dQ and
    dK are those of the unrotated q and k: bf16 as the backward gives them, turned back and rounded once more."""
    there = _rotated_elsewhere(q, k, v, rope, stream)
    if there is not None:
        with there:
            return forward_backward(q, k, v, do, layout, softmax_scale, p_terms, None, rope, positions)
    qq, qs, kq, ks, vt, vsc, vtn, vtn_sc = _operands(q, k, v, layout, True, rope, positions, stream)
    o, lse = mxfp8_causal_attn_fwd(qq, qs, kq, ks, vt, vsc, vtn, vtn_sc, layout, softmax_scale, p_terms,
                                   stream=stream)
    dq, dk, dv = bf16_attn_bwd(qq, qs, kq, ks, vtn, vtn_sc, o, lse, do, layout, softmax_scale, stream=stream)
    if rope is not None:
        apply_rope(dq, dk, rope, positions, layout, inverse=True, q_out=dq, k_out=dk, stream=stream)
    return o, lse, dq, dk, dv


def mxfp8_quantize(kind, x, layout=BSHD, rule=SCALE_FLOOR, stream=None):
    """Any quantisation with a chosen scale rule.  Returns the outputs of the matching call:
    (bytes, [B,H,S,D/32] scales) for QUANT_ROWWISE, (V^T bytes, [B,H,S/32,D] scales) for QUANT_V_COLWISE,
    (token-normalised bytes, amplitudes) for QUANT_V_TOKEN_NORM, all four for QUANT_V_FUSED."""
    _require(x, torch.bfloat16, "x")
    B, S, H, D = _bshd_dims(x, layout)
    u8 = dict(dtype=torch.uint8, device=x.device)
    e4m3 = sc = vtn = vtn_sc = None
    if kind == QUANT_ROWWISE:
        e4m3, sc = torch.empty(x.shape, **u8), torch.empty((B, H, S, D // 32), **u8)
    if kind in (QUANT_V_COLWISE, QUANT_V_FUSED):
        e4m3, sc = torch.empty((B, H, D, S), **u8), torch.empty((B, H, S // 32, D), **u8)
    if kind in (QUANT_V_TOKEN_NORM, QUANT_V_FUSED):
        vtn, vtn_sc = torch.empty(x.shape, **u8), torch.empty((B, H, S), **u8)
    p = QuantParams(kind=kind, x=x.data_ptr(), B=B, S=S, H=H, D=D, layout=layout, rule=rule,
                    e4m3=_ptr(e4m3), sc=_ptr(sc), vtn_e4m3=_ptr(vtn), vtn_sc=_ptr(vtn_sc))
    _check(lib.mxfp8_quantize(ctypes.byref(p), _stream(stream)))
    if kind == QUANT_V_FUSED:
        return e4m3, sc, vtn, vtn_sc
    if kind == QUANT_V_TOKEN_NORM:
        return vtn, vtn_sc
    return e4m3, sc


def mxfp8_quantize_qkv(q, k, v, layout=BSHD, rule=SCALE_FLOOR, token_norm=True, out=None, stream=None):
    """Q and K rowwise and V columnwise (+ token-normalised unless token_norm=False) in one launch.
    Returns (q_e4m3, q_sc, k_e4m3, k_sc, v_e4m3_t, v_sc, vtn_e4m3, vtn_sc), the last two None when
    token_norm=False; `out` may give all eight (the last two may be None)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, torch.bfloat16, n)
    B, S, Hq, D = _bshd_dims(q, layout)
    Hkv = _bshd_dims(k, layout)[2]
    if tuple(k.shape) != tuple(v.shape):
        raise ValueError("k and v must have the same shape")
    if out is None:
        u8 = dict(dtype=torch.uint8, device=q.device)
        out = (torch.empty(q.shape, **u8), torch.empty((B, Hq, S, D // 32), **u8),
               torch.empty(k.shape, **u8), torch.empty((B, Hkv, S, D // 32), **u8),
               torch.empty((B, Hkv, D, S), **u8), torch.empty((B, Hkv, S // 32, D), **u8),
               torch.empty(v.shape, **u8) if token_norm else None,
               torch.empty((B, Hkv, S), **u8) if token_norm else None)
    qq, qs, kq, ks, vt, vsc, vtn, vtn_sc = out
    p = QkvQuantParams(q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, layout=layout,
                       rule=rule, q_e4m3=_ptr(qq), q_sc=_ptr(qs), k_e4m3=_ptr(kq), k_sc=_ptr(ks), v_e4m3_t=_ptr(vt),
                       v_sc=_ptr(vsc), vtn_e4m3=_ptr(vtn), vtn_sc=_ptr(vtn_sc))
    _check(lib.mxfp8_quantize_qkv(ctypes.byref(p), _stream(stream)))
    return qq, qs, kq, ks, vt, vsc, vtn, vtn_sc


class MxCache:
    """The key/value cache: a handle on the caller's four uint8 CUDA pools (bsc_mx_cache in bsc.h).

    k, v [num_pages, Hkv, page_size, D] (CACHE_MXFP8) or [..., D/2] (CACHE_MXFP4); k_sc, v_sc
    [num_pages, Hkv, page_size, D/32].  Dimensions after the first are contiguous; the page stride is
    free, so pools may be slices of one allocation.  The handle keeps the tensors alive and holds no
    other state.  `mx_cache_alloc` makes one with new pools.

    The calls' `stream` works like torch.cuda.stream(stream) around them: the caller sees to it that what other
    streams wrote is ready, and that the tensors live until the call has run."""

    __slots__ = ("k", "k_sc", "v", "v_sc", "fmt", "num_pages", "page_size", "Hkv", "D", "device", "index", "params", "packed")

    def __init__(self, k, k_sc, v, v_sc, fmt=CACHE_MXFP4):
        if fmt not in (CACHE_MXFP8, CACHE_MXFP4):
            raise ValueError("fmt must be CACHE_MXFP8 or CACHE_MXFP4")
        pools = (k, k_sc, v, v_sc)
        for t, n in zip(pools, ("k", "k_sc", "v", "v_sc")):
            if not t.is_cuda or t.dtype != torch.uint8 or t.dim() != 4 or t.device != k.device:
                raise ValueError("%s must be a 4-D CUDA uint8 tensor on one device with the others" % n)
            if t.shape[0] and not t[0].is_contiguous():
                raise ValueError("%s must be contiguous within a page" % n)
        pages, Hkv, page_size, row = k.shape
        D = row * 2 if fmt == CACHE_MXFP4 else row
        if k.shape != v.shape or k_sc.shape != v_sc.shape or tuple(k_sc.shape) != (pages, Hkv, page_size, D // 32):
            raise ValueError("k, v must be [pages, Hkv, page_size, row] and k_sc, v_sc [pages, Hkv, page_size, D/32]")
        self.k, self.k_sc, self.v, self.v_sc = pools
        self.fmt, self.num_pages, self.page_size, self.Hkv, self.D = fmt, pages, page_size, Hkv, D
        self.device, self.index = k.device, k.get_device()
        self.params = CachePools(*(t.data_ptr() for t in pools), *(t.stride(0) for t in pools), fmt, pages, page_size,
                                 Hkv, D)
        self.packed = bytes(self.params)


def mx_cache_alloc(num_pages, page_size, Hkv, D=128, fmt=CACHE_MXFP4, device="cuda"):
    """An MxCache with new, zeroed pools (zero bytes stand for zeros)."""
    shape = (num_pages, Hkv, page_size)
    row = D // 2 if fmt == CACHE_MXFP4 else D
    k, k_sc, v, v_sc = (torch.zeros(shape + (n,), dtype=torch.uint8, device=device) for n in (row, D // 32) * 2)
    return MxCache(k, k_sc, v, v_sc, fmt)


def _act_dims(x, layout, cache, name, D=None):
    """(B, T, H), element strides (b, t, h) and the dtype code of an activation of head size D (None: the cache's) on the
    device of `cache` (or of a Rope)."""
    code, shape = _ACT.get(x.dtype), x.shape
    if code is None or len(shape) != 4 or x.get_device() != cache.index:
        raise ValueError("%s must be a 4-D bfloat16 or float16 tensor on the cache's device" % name)
    B, T, H, width = shape
    sb, st, sh, sd = x.stride()
    if layout == SBHD:
        B, T, sb, st = T, B, st, sb
    elif layout != BSHD:
        raise ValueError("layout must be BSHD or SBHD")
    if width != (cache.D if D is None else D):
        raise ValueError("%s does not have the cache's head size" % name)
    if sd != 1 and x.numel():
        raise ValueError("%s must be contiguous along D" % name)
    return (B, T, H), (sb, st, sh), code


def _dense(layout, B, T, H, D):
    """Shape of a contiguous activation and its strides (b, t, h)."""
    if layout == BSHD:
        return (B, T, H, D), (T * H * D, H * D, D)
    if layout == SBHD:
        return (T, B, H, D), (H * D, B * H * D, D)
    raise ValueError("layout must be BSHD or SBHD")


def _out_like(x, out, dims, layout, cache, name, dtype, D=None):
    """An output of the shape and dtype of activation x (dims, dtype code): `out` if given, else a new contiguous one; and its
    element strides (b, t, h)."""
    if out is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format), _dense(layout, *dims, x.shape[3])[1]
    dims_o, strides, dtype_o = _act_dims(out, layout, cache, name, D)
    if dims_o != dims or dtype_o != dtype:
        raise ValueError("%s must have its input's shape and dtype" % name)
    return out, strides


def _index(t, B, cache, name):
    """Pointer of an int32 index array of B entries (None: NULL)."""
    if t is None:
        return 0
    if t.dtype is not torch.int32 or t.shape != (B,) or t.get_device() != cache.index:
        raise ValueError("%s must be an int32 tensor of shape (%d,) on the cache's device" % (name, B))
    if B > 1 and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _table(t, B, cache):
    """Pointer, row stride and columns of a page table of B rows."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != B or t.dtype is not torch.int32 or t.get_device() != cache.index:
        raise ValueError("page_table must be an int32 tensor [B, max_pages] on the cache's device")
    row, col = t.stride()
    if col != 1 and shape[1] > 1:
        raise ValueError("page_table must have contiguous rows")
    return t.data_ptr(), row, shape[1]


def _status(t, cache):
    if t is None:
        return 0
    if t.dtype != torch.int32 or t.device != cache.device or t.numel() < 1:
        raise ValueError("dev_status must be an int32 tensor on the cache's device")
    return t.data_ptr()


def _elsewhere(cache, stream):
    """The context a call has to enter before it allocates and launches: None where the current device is the
    cache's and no stream is given; else the stream's (memory allocated inside belongs to the stream that
    uses it) or the device's."""
    if stream is None and _current_device() == cache.index:
        return None
    if stream is not None:
        if stream.device != cache.device:
            raise ValueError("stream must be on the cache's device")
        return torch.cuda.stream(stream)
    return torch.cuda.device(cache.device)


def _elsewhere_of(x, name, stream):
    """_elsewhere for a call whose device is that of tensor x."""
    if not x.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if stream is not None:
        if stream.device != x.device:
            raise ValueError("stream must be on %s's device" % name)
        return torch.cuda.stream(stream)
    return torch.cuda.device(x.device)


# The current stream's handle without a Stream object around it (a call's largest host cost after the launches).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _packed_call(name, params, fields, ahead=ctypes.sizeof(CachePools)):
    """The C call `name` taking its parameters as packed bytes, and the packer of what follows the cache (`ahead` bytes)
    in them (native sizes and alignment, as ctypes lays `params` out): a quarter of a ctypes structure's time."""
    f = lib[name]
    f.restype, f.argtypes = ctypes.c_int, [ctypes.c_char_p, ctypes.c_void_p]
    packer = struct.Struct("@" + fields)
    assert ahead + packer.size == ctypes.sizeof(params)
    return f, packer.pack


# pointers and strides, sizes and codes, then from page_table on
_c_write, _pack_write = _packed_call("mx_cache_write", CacheWriteParams, "8q4i2qi3q")
_c_read, _pack_read = _packed_call("mx_cache_read", CacheReadParams, "8q3i2qi3q")
_c_attn, _pack_attn = _packed_call("mx_cache_attn", CacheAttnParams, "9q4if2qi5q")


def mx_cache_write(cache, k, v, page_table, seq_lens, new_lens=None, layout=BSHD, rule=SCALE_FLOOR, dev_status=None,
                   stream=None):
    """Quantises new tokens into the cache.  k, v: bf16 or fp16 [B, T, Hkv, D] (BSHD) or [T, B, Hkv, D]
    (SBHD), any strides with D contiguous.  Token t < new_lens[b] (None: all T) of sequence b goes to position
    seq_lens[b] - new_lens[b] + t; page_table [B, max_pages], seq_lens, new_lens [B]: int32 on the device."""
    there = _elsewhere(cache, stream)
    if there is not None:
        with there:
            return mx_cache_write(cache, k, v, page_table, seq_lens, new_lens, layout, rule, dev_status)
    dims, ks, dt = _act_dims(k, layout, cache, "k")
    dims_v, vs, dt_v = _act_dims(v, layout, cache, "v")
    B, T, H = dims
    if dims_v != dims or dt_v != dt or H != cache.Hkv:
        raise ValueError("k and v must both have the cache's heads, one shape and one dtype")
    p = cache.packed + _pack_write(k.data_ptr(), v.data_ptr(), *ks, *vs, B, T, dt, rule,
                         *_table(page_table, B, cache), _index(seq_lens, B, cache, "seq_lens"),
                         _index(new_lens, B, cache, "new_lens"), _status(dev_status, cache))
    _check(_c_write(p, _raw_stream(cache.index)))


def mx_cache_read(cache, page_table, seq_lens, T, starts=None, layout=BSHD, dtype=torch.bfloat16, k_out=None,
                  v_out=None, dev_status=None, stream=None):
    """Reads positions starts[b] .. starts[b] + T - 1 (None: from 0) of every sequence back as values:
    (k, v), shaped [B, T, Hkv, D] or [T, B, Hkv, D]; zeros outside [0, seq_lens[b])."""
    there = _elsewhere(cache, stream)
    if there is not None:
        with there:
            return mx_cache_read(cache, page_table, seq_lens, T, starts, layout, dtype, k_out, v_out, dev_status)
    B, Hkv = page_table.shape[0], cache.Hkv
    shape, ks = _dense(layout, B, T, Hkv, cache.D)
    vs, dt = ks, _ACT.get(dtype)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=cache.device)
    else:
        dims, ks, dt = _act_dims(k_out, layout, cache, "k_out")
        if dims != (B, T, Hkv):
            raise ValueError("k_out must be [B, T, Hkv, D] in the layout")
    if v_out is None:
        v_out = torch.empty(shape, dtype=dtype, device=cache.device)
        dt_v = _ACT.get(dtype)
    else:
        dims, vs, dt_v = _act_dims(v_out, layout, cache, "v_out")
        if dims != (B, T, Hkv):
            raise ValueError("v_out must be [B, T, Hkv, D] in the layout")
    if dt is None or dt != dt_v:
        raise ValueError("k_out and v_out must be bfloat16 or float16, of one dtype")
    p = cache.packed + _pack_read(k_out.data_ptr(), v_out.data_ptr(), *ks, *vs, B, T, dt,
                        *_table(page_table, B, cache), _index(seq_lens, B, cache, "seq_lens"),
                        _index(starts, B, cache, "starts"), _status(dev_status, cache))
    _check(_c_read(p, _raw_stream(cache.index)))
    return k_out, v_out


@functools.lru_cache(maxsize=256)
def mx_cache_attn_workspace_bytes(B, T, Hq, Hkv, D=128, max_tokens=1 << 30):
    """Bytes of scratch mx_cache_attn needs at these sizes (the C call of the same name); max_tokens: page_table
    columns times page size (left out: enough for any table)."""
    return int(lib.mx_cache_attn_workspace_bytes(B, T, Hq, Hkv, D, max_tokens))


def mx_cache_attn(q, cache, page_table, seq_lens, new_lens=None, layout=BSHD, softmax_scale=None, o=None, lse=None,
                  workspace=None, dev_status=None, stream=None):
    """Attention of T queries per sequence over the cache; returns (O shaped and typed like q, LSE fp32
    [B, Hq, T]).  Query t < new_lens[b] (None: all T) is the token at position seq_lens[b] - new_lens[b] + t and
    attends the positions up to its own.  `workspace`: a device tensor of at least
    mx_cache_attn_workspace_bytes(...) bytes that no other running call uses, else one is allocated here
    where the call needs any."""
    there = _elsewhere(cache, stream)
    if there is not None:
        with there:
            return mx_cache_attn(q, cache, page_table, seq_lens, new_lens, layout, softmax_scale, o, lse, workspace,
                                 dev_status)
    dims, qs, dt = _act_dims(q, layout, cache, "q")
    B, T, Hq = dims
    table = _table(page_table, B, cache)
    device = cache.device
    o, o_s = _out_like(q, o, dims, layout, cache, "o", dt)
    if lse is None:
        lse = torch.empty((B, Hq, T), dtype=torch.float32, device=device)
    elif lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, T) or lse.device != device or \
            not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 tensor [B, Hq, T] on the cache's device")
    if workspace is None:
        need = mx_cache_attn_workspace_bytes(B, T, Hq, cache.Hkv, cache.D, table[2] * cache.page_size)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the cache's device")
        need = workspace.numel() * workspace.element_size()
    p = cache.packed + _pack_attn(q.data_ptr(), o.data_ptr(), lse.data_ptr(), *qs, *o_s, B, T, Hq, dt,
                        cache.D ** -0.5 if softmax_scale is None else softmax_scale, *table, _index(seq_lens, B, cache, "seq_lens"),
                        _index(new_lens, B, cache, "new_lens"), _status(dev_status, cache),
                        workspace.data_ptr() if need else 0, need)
    _check(_c_attn(p, _raw_stream(cache.index)))
    return o, lse


# ------------------------------------------------------------------------------- norm and rotary positions
# `stream` is that of the cache's calls (MxCache): like torch.cuda.stream(stream) around the call.
_WEIGHT = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_ANGLES = ctypes.sizeof(RopeAngles)
_c_norm, _pack_norm = _packed_call("rms_norm", RmsNormParams, "8q9q5if", 0)
_c_norm_bwd, _pack_norm_bwd = _packed_call("rms_norm_bwd", RmsNormBwdParams, "7q9q4i2q", 0)
_c_rope, _pack_rope = _packed_call("rope", RopeParams, "4q12q3q7i0q", _ANGLES)
_c_rope_quant, _pack_rope_quant = _packed_call("mxfp8_rope_quantize_qk", RopeQuantParams, "2q6q4q3q8i", _ANGLES)
_c_write_rope, _pack_write_rope = _packed_call("mx_cache_write_rope", CacheWriteRopeParams, "4q12q5i2qi3q",
                                               ctypes.sizeof(CachePools) + _ANGLES)
_c_bounds, _pack_bounds = _packed_call("mx_cache_bounds", CacheBoundsParams, "2i2qi3q", ctypes.sizeof(CachePools) + 16)
_c_sparse, _pack_sparse = _packed_call("mx_cache_sparse_attn", CacheSparseAttnParams, "10q4if3i2qi5q", ctypes.sizeof(CachePools) + 16)


def _same_rows(t, shape, dtype, dev, name):
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError("%s must have the first tensor's shape, device and dtype" % name)


def _row_layout(tensors):
    """(rows, inner, [(stride, inner stride)]) of tensors [..., N] of one shape (None: (0, 0)): one split of the leading
    dimensions into two groups, within each of which every tensor's rows are evenly spaced."""
    first = tensors[0]
    lead, N = first.shape[:-1], first.shape[-1]
    rows = 1
    for n in lead:
        rows *= n
    if all([t is None or t.is_contiguous() for t in tensors]):
        return rows, 1, [(0, 0) if t is None else (N, 0) for t in tensors]
    for t in tensors:
        if t is not None and t.stride(-1) != 1 and N > 1 and t.numel():
            raise ValueError("rows must be contiguous")

    def even(t, dims):
        """Stride of rows numbered over `dims`, or None."""
        step = None
        for d in reversed(dims):
            if t.shape[d] == 1:
                continue
            if step is None:
                step, count = t.stride(d), t.shape[d]
            elif t.stride(d) == step * count:
                count *= t.shape[d]
            else:
                return None
        return step or 0

    if rows == 0:
        return 0, 1, [(0, 0)] * len(tensors)
    for cut in range(len(lead), -1, -1):
        outer, inner = range(cut), range(cut, len(lead))
        pairs = [(0, 0) if t is None else (even(t, outer), even(t, inner)) for t in tensors]
        if all(a is not None and b is not None for a, b in pairs):
            n = 1
            for d in inner:
                n *= lead[d]
            return rows, n, pairs
    raise ValueError("the rows of every tensor must be spaced by at most two strides")


def _weight_code(weight, N, dtype, dev):
    wd = weight.dtype
    if weight.shape != (N,) or weight.get_device() != dev or not weight.is_contiguous() or \
            (wd is not dtype and wd is not torch.float32):
        raise ValueError("weight must be a contiguous [N] tensor of the activations' dtype or float32")
    return _WEIGHT[wd]


def _rstd_of(rstd, lead, dev):
    if rstd.shape != lead or rstd.dtype is not torch.float32 or rstd.get_device() != dev or not rstd.is_contiguous():
        raise ValueError("rstd must be a contiguous float32 tensor of the activations' leading dimensions")


def rms_norm(x, weight, eps=1e-6, residual=None, y=None, sum_out=None, rstd=None, y8_out=False, y_out=True, y8=None,
             y_sc=None, rule=SCALE_FLOOR, stream=None):
    """Root-mean-square norm of the rows of x [..., N] (bf16 or fp16), with the residual's addition.

    s = x + residual (held in x's dtype), rstd = (mean s^2 + eps)^-1/2, y = s * rstd * weight.  Returns (y, s, rstd), s being
    x itself without a residual and rstd float32 [...]; with y8_out=True, (y or None, s, rstd, y as E4M3 bytes [..., N], its
    scales [..., N/32]).  weight: [N], x's dtype or float32.  y, sum_out and rstd may be given; y and sum_out may be x or
    residual themselves."""
    dev = x.get_device()
    if stream is not None or dev < 0 or _current_device() != dev:
        with _elsewhere_of(x, "x", stream):
            return rms_norm(x, weight, eps, residual, y, sum_out, rstd, y8_out, y_out, y8, y_sc, rule)
    dtype, shape = x.dtype, x.shape
    dt = _ACT.get(dtype)
    if dt is None or not shape:
        raise ValueError("x must be a bfloat16 or float16 tensor [..., N]")
    N, lead = shape[-1], shape[:-1]
    wt = _weight_code(weight, N, dtype, dev)
    fresh = x.is_contiguous()                  # an output that is allocated here is laid out like x
    if y_out:
        if y is None:
            y = torch.empty_like(x, memory_format=torch.contiguous_format)
        else:
            _same_rows(y, shape, dtype, dev, "y")
            fresh = False
        y_ptr = y.data_ptr()
    elif y8_out:
        y, y_ptr = None, 0
    else:
        raise ValueError("y_out=False needs y8_out=True")
    if residual is None:
        if sum_out is not None:
            raise ValueError("sum_out is for a residual")
        r_ptr = s_ptr = 0
    else:
        _same_rows(residual, shape, dtype, dev, "residual")
        fresh = fresh and residual.is_contiguous()
        if sum_out is None:
            sum_out = torch.empty_like(x, memory_format=torch.contiguous_format)
        else:
            _same_rows(sum_out, shape, dtype, dev, "sum_out")
            fresh = False
        r_ptr, s_ptr = residual.data_ptr(), sum_out.data_ptr()
    if rstd is None:
        rstd = torch.empty(lead, dtype=torch.float32, device=x.device)
    else:
        _rstd_of(rstd, lead, dev)
    y8_ptr = sc_ptr = 0
    if y8_out:
        shapes = (shape, lead + (N // 32,))
        y8, y_sc = (torch.empty(n, dtype=torch.uint8, device=x.device) if t is None else t for t, n in zip((y8, y_sc), shapes))
        for t, n in ((y8, shapes[0]), (y_sc, shapes[1])):
            if t.dtype != torch.uint8 or t.shape != n or t.device != x.device or not t.is_contiguous():
                raise ValueError("y8 and y_sc must be contiguous uint8 tensors [..., N] and [..., N/32]")
        y8_ptr, sc_ptr = y8.data_ptr(), y_sc.data_ptr()
    if fresh:
        rows, inner, xs, rs, ys, ss = x.numel() // max(N, 1), 1, (N, 0), (N, 0), (N, 0), (N, 0)
    else:
        rows, inner, (xs, rs, ys, ss) = _row_layout((x, residual, y, sum_out))
    p = _pack_norm(x.data_ptr(), r_ptr, weight.data_ptr(), y_ptr, s_ptr, rstd.data_ptr(), y8_ptr, sc_ptr, rows, *xs, *rs, *ys,
                   *ss, inner, N, dt, wt, rule, eps)
    _check(_c_norm(p, _raw_stream(dev)))
    s = x if residual is None else sum_out
    return (y, s, rstd, y8, y_sc) if y8_out else (y, s, rstd)


def rms_norm_bwd_workspace_bytes(rows, N):
    """Bytes of scratch rms_norm_bwd needs (the C call of the same name)."""
    return int(lib.rms_norm_bwd_workspace_bytes(rows, N))


def rms_norm_bwd(dy, s, weight, rstd, ds=None, dx=None, dweight=None, workspace=None, stream=None):
    """Gradients of rms_norm at s (its second output) with its rstd: (dx, dweight).  dx is the gradient of x and of the
    residual alike, with `ds`, the gradient that reaches s by the residual stream, added; dweight has weight's dtype.
    dx may be dy, s or ds themselves.  `workspace`: a device tensor of rms_norm_bwd_workspace_bytes(rows, N) bytes that no
    other running call uses, else one is allocated here."""
    dev = s.get_device()
    if stream is not None or dev < 0 or _current_device() != dev:
        with _elsewhere_of(s, "s", stream):
            return rms_norm_bwd(dy, s, weight, rstd, ds, dx, dweight, workspace)
    dtype, shape = s.dtype, s.shape
    dt = _ACT.get(dtype)
    if dt is None or not shape:
        raise ValueError("s must be a bfloat16 or float16 tensor [..., N]")
    N = shape[-1]
    wt = _weight_code(weight, N, dtype, dev)
    _same_rows(dy, shape, dtype, dev, "dy")
    if ds is not None:
        _same_rows(ds, shape, dtype, dev, "ds")
    _rstd_of(rstd, shape[:-1], dev)
    if dx is None:
        dx = torch.empty_like(s, memory_format=torch.contiguous_format)
    else:
        _same_rows(dx, shape, dtype, dev, "dx")
    rows, inner, (dys, ss, dss, dxs) = _row_layout((dy, s, ds, dx))
    if dweight is None:
        dweight = torch.empty_like(weight)
    elif dweight.shape != weight.shape or dweight.dtype != weight.dtype or dweight.device != s.device or \
            not dweight.is_contiguous():
        raise ValueError("dweight must be a contiguous tensor like weight")
    if rows == 0:
        dweight.zero_()                        # the call has nothing to do
    if workspace is None:
        need = rms_norm_bwd_workspace_bytes(rows, N)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=s.device)
    else:
        if workspace.device != s.device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the activations' device")
        need = workspace.numel() * workspace.element_size()
    p = _pack_norm_bwd(dy.data_ptr(), s.data_ptr(), weight.data_ptr(), rstd.data_ptr(), 0 if ds is None else ds.data_ptr(),
                       dx.data_ptr(), dweight.data_ptr(), rows, *dys, *ss, *dss, *dxs, inner, N, dt, wt, workspace.data_ptr(),
                       need)
    _check(_c_norm_bwd(p, _raw_stream(dev)))
    return dx, dweight


_UNSAID = object()


def mxfp8_dequantize(x, sc, layout=_UNSAID, dtype=torch.bfloat16, out=None, stream=None):
    """MXFP8 rows back to values.  layout BSHD or SBHD: x uint8 [B, S, H, D] or [S, B, H, D] with sc [B, H, S, D/32], as the
    rowwise quantisers return them.  None: x [..., N] with sc [..., N/32], as rms_norm does.  A 4-D x may be either, so its
    layout has to be said; any other is taken for the second."""
    dev = x.get_device()
    if stream is not None or dev < 0 or _current_device() != dev:
        with _elsewhere_of(x, "x", stream):
            return mxfp8_dequantize(x, sc, layout, dtype, out)
    code = _ACT.get(dtype)
    if code is None:
        raise ValueError("dtype must be bfloat16 or float16")
    for t, n in ((x, "x"), (sc, "sc")):
        if t.dtype is not torch.uint8 or t.get_device() != dev or not t.is_contiguous():
            raise ValueError("%s must be a contiguous CUDA uint8 tensor on one device with the other" % n)
    shape = x.shape
    if len(shape) != 4 and layout is _UNSAID:
        layout = None
    if layout is not None:
        if layout is _UNSAID or len(shape) != 4:
            raise ValueError("a 4-D x needs its layout, BSHD, SBHD or None; any other has None")
        B, S, H, D = shape
        if layout == SBHD:
            B, S = S, B
        elif layout != BSHD:
            raise ValueError("layout must be BSHD or SBHD")
        want = (B, H, S, D // 32)
    elif shape:
        B, H, D = 1, 1, shape[-1]
        S, want, layout = x.numel() // max(D, 1), shape[:-1] + (D // 32,), BSHD
    else:
        raise ValueError("x must have at least one dimension")
    if sc.shape != want:
        raise ValueError("sc must have the shape %s" % (tuple(want),))
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
    elif out.shape != x.shape or out.dtype != dtype or out.device != x.device or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor shaped like x, of dtype")
    _check(lib.mxfp8_dequantize(x.data_ptr(), sc.data_ptr(), B, S, H, D, layout, code, out.data_ptr(),
                                _raw_stream(dev)))
    return out


class Rope:
    """Rotary positions' frequencies: one per pair of the first `rot` elements of a head, on the device, in turns per token
    (bsc_rope_turns and bsc_rope_angles in bsc.h).  Any 32-bit position may be rotated by it; it holds no other state.

    interleaved: pairs are neighbours (x_2i, x_2i+1), else (x_i, x_{i + rot/2}).  scaling: ROPE_PLAIN; ROPE_LINEAR (positions
    / factor); ROPE_BASE (base * factor^(rot/(rot-2))); ROPE_BY_PARTS (pairs of fewer than low_turns turns in
    original_length tokens are interpolated by factor, those of more than high_turns are kept, what lies between is mixed, linear
    in turns).
    magnitude: the factor on what is rotated (None: 0.1 ln(factor) + 1 by parts, else 1)."""

    __slots__ = ("rot", "interleaved", "magnitude", "turns", "device", "index", "params", "packed")

    def __init__(self, rot, base=10000.0, interleaved=False, scaling=ROPE_PLAIN, factor=1.0, original_length=0,
                 low_turns=1.0, high_turns=32.0, magnitude=None, device="cuda"):
        config = RopeConfig(rot, scaling, base, factor, original_length, low_turns, high_turns)
        host, m = (ctypes.c_ulonglong * 128)(), ctypes.c_float()
        _check(lib.bsc_rope_turns(ctypes.byref(config), host, ctypes.byref(m)))
        signed = (ctypes.c_longlong * (rot // 2)).from_buffer(host)
        self.turns = torch.tensor(list(signed), dtype=torch.int64).to(device)
        self.rot, self.interleaved = rot, bool(interleaved)
        self.magnitude = lib.bsc_rope_magnitude(ctypes.byref(config)) if magnitude is None else float(magnitude)
        high = ctypes.c_float(self.magnitude).value
        low = self.magnitude - high if 1e-30 < abs(high) < math.inf else 0.0
        self.device, self.index = self.turns.device, self.turns.get_device()
        self.params = RopeAngles(self.turns.data_ptr(), high, rot, int(self.interleaved), low)
        self.packed = bytes(self.params)


def _positions(t, B, T, rope):
    """Pointer and strides (b, t) of positions: None, [B] (of the first tokens) or [B, T] int32."""
    if t is None:
        return 0, 0, 0
    shape = t.shape
    if t.dtype is not torch.int32 or t.get_device() != rope.index or (shape != (B, T) and shape != (B,)):
        raise ValueError("positions must be an int32 tensor of shape (%d,) or (%d, %d) on rope's device" % (B, B, T))
    stride = t.stride()
    if len(shape) == 1:
        return t.data_ptr(), stride[0], 0
    if T > 1 and stride[1] == 0:
        raise ValueError("positions must not be expanded along the tokens")
    return t.data_ptr(), stride[0], stride[1] or 1


def _elsewhere_with(rope, q, stream):
    """_elsewhere for a call on q by a Rope."""
    if q.get_device() != rope.index or not q.is_cuda:
        raise ValueError("q must be on rope's device, a CUDA device")
    return None if stream is None and _current_device() == rope.index else _elsewhere(rope, stream)


def _heads(Hq, Hkv):
    """The C calls have nothing to do where q has no heads, and k would stay behind."""
    if Hq == 0 and Hkv > 0:
        raise ValueError("q must have at least one head beside k")


def apply_rope(q, k, rope, positions=None, layout=BSHD, inverse=False, q_out=None, k_out=None, stream=None):
    """Q and K (or None) rotated by a Rope in one launch; returns (q, k) of the same shapes and dtype.

    q [B, T, Hq, D] and k [B, T, Hkv, D] (SBHD: [T, B, H, D]), bf16 or fp16, any strides with D contiguous.  positions: None
    (token t is at t), int32 [B] (of each sequence's first token) or [B, T].  inverse=True turns back: gradients of q and k
    from those of the outputs.  q_out and k_out may be q and k themselves."""
    there = _elsewhere_with(rope, q, stream)
    if there is not None:
        with there:
            return apply_rope(q, k, rope, positions, layout, inverse, q_out, k_out)
    D = q.shape[-1]
    dims, qs, dt = _act_dims(q, layout, rope, "q", D)
    B, T, Hq = dims
    q_out, q_os = _out_like(q, q_out, dims, layout, rope, "q_out", dt, D)
    if k is None:
        if k_out is not None:
            raise ValueError("k_out is for k")
        Hkv, ks, k_os, k_ptr, k_out_ptr = 0, (0, 0, 0), (0, 0, 0), 0, 0
    else:
        dims_k, ks, dt_k = _act_dims(k, layout, rope, "k", D)
        Bk, Tk, Hkv = dims_k
        _heads(Hq, Hkv)
        if Bk != B or Tk != T or dt_k != dt:
            raise ValueError("k must have q's batch, tokens and dtype")
        k_out, k_os = _out_like(k, k_out, dims_k, layout, rope, "k_out", dt, D)
        k_ptr, k_out_ptr = k.data_ptr(), k_out.data_ptr()
    p = rope.packed + _pack_rope(q.data_ptr(), k_ptr, q_out.data_ptr(), k_out_ptr, *qs, *ks, *q_os, *k_os,
                                 *_positions(positions, B, T, rope), B, T, Hq, Hkv, D, dt, 1 if inverse else 0)
    _check(_c_rope(p, _raw_stream(rope.index)))
    return q_out, k_out


rope = apply_rope      # the C call's name, by which the documents name it; in the calls `rope` is their Rope


def mxfp8_rope_quantize_qk(q, k, rope, positions=None, layout=BSHD, rule=SCALE_FLOOR, stream=None):
    """Q and K (or None) rotated (as in `rope`) and quantised rowwise to MXFP8 in one launch, from the rotated fp32 values:
    (q_e4m3, q_sc, k_e4m3, k_sc), bytes dense in `layout` and scales [B, H, T, D/32]; D = 128."""
    there = _elsewhere_with(rope, q, stream)
    if there is not None:
        with there:
            return mxfp8_rope_quantize_qk(q, k, rope, positions, layout, rule)
    D = q.shape[-1]
    (B, T, Hq), qs, dt = _act_dims(q, layout, rope, "q", D)
    u8 = dict(dtype=torch.uint8, device=q.device)
    q8, q_sc = torch.empty(q.shape, **u8), torch.empty((B, Hq, T, D // 32), **u8)
    if k is None:
        k8, k_sc, Hkv, ks, k_ptrs = None, None, 0, (0, 0, 0), (0, 0, 0)
    else:
        (Bk, Tk, Hkv), ks, dt_k = _act_dims(k, layout, rope, "k", D)
        _heads(Hq, Hkv)
        if Bk != B or Tk != T or dt_k != dt:
            raise ValueError("k must have q's batch, tokens and dtype")
        k8, k_sc = torch.empty(k.shape, **u8), torch.empty((B, Hkv, T, D // 32), **u8)
        k_ptrs = k.data_ptr(), k8.data_ptr(), k_sc.data_ptr()
    p = rope.packed + _pack_rope_quant(q.data_ptr(), k_ptrs[0], *qs, *ks, q8.data_ptr(), q_sc.data_ptr(), *k_ptrs[1:],
                                       *_positions(positions, B, T, rope), B, T, Hq, Hkv, D, dt, layout, rule)
    _check(_c_rope_quant(p, _raw_stream(rope.index)))
    return q8, q_sc, k8, k_sc


def mx_cache_write_rope(cache, q, k, v, rope, page_table, seq_lens, new_lens=None, layout=BSHD, rule=SCALE_FLOOR, q_out=None,
                        dev_status=None, stream=None):
    """mx_cache_write with K rotated on its way in, and q's rows of the same tokens rotated: returns q_out, shaped and typed
    like q.  Positions are those of the write: token t < new_lens[b] of sequence b is at seq_lens[b] - new_lens[b] + t; rows of
    q_out of other tokens are zeros.  q_out may be q itself."""
    there = _elsewhere(cache, stream)
    if there is not None:
        with there:
            return mx_cache_write_rope(cache, q, k, v, rope, page_table, seq_lens, new_lens, layout, rule, q_out, dev_status)
    if rope.index != cache.index:
        raise ValueError("rope must be on the cache's device")
    dims, qs, dt = _act_dims(q, layout, cache, "q")
    dims_k, ks, dt_k = _act_dims(k, layout, cache, "k")
    dims_v, vs, dt_v = _act_dims(v, layout, cache, "v")
    B, T, Hq = dims
    _heads(Hq, cache.Hkv)
    if dims_k != (B, T, cache.Hkv) or dims_v != dims_k or dt_k != dt or dt_v != dt:
        raise ValueError("k and v must have q's batch, tokens and dtype and the cache's heads")
    q_out, q_os = _out_like(q, q_out, dims, layout, cache, "q_out", dt)
    p = cache.packed + rope.packed + _pack_write_rope(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), *qs, *ks, *vs, *q_os, B, T, Hq, dt, rule,
        *_table(page_table, B, cache), _index(seq_lens, B, cache, "seq_lens"), _index(new_lens, B, cache, "new_lens"),
        _status(dev_status, cache))
    _check(_c_write_rope(p, _raw_stream(cache.index)))
    return q_out


# ----------------------------------------------------------------------------- reading less of a long cache
class MxBounds:
    """Bounds of a cache's pages: codes int8 [num_pages, Hkv, 2, D] (minima, maxima along D) and exps uint8 [num_pages, Hkv],
    the caller's two buffers (mx_cache_bounds_alloc makes new ones).  The handle holds no other state."""

    __slots__ = ("codes", "exps", "of", "packed")

    def __init__(self, cache, codes, exps):
        shape = (cache.num_pages, cache.Hkv)
        for t, n, d, want in ((codes, "codes", torch.int8, shape + (2, cache.D)), (exps, "exps", torch.uint8, shape)):
            if t.dtype != d or tuple(t.shape) != want or t.device != cache.device or not t.is_contiguous():
                raise ValueError("%s must be a contiguous %s tensor %s on the cache's device" % (n, d, want))
        self.codes, self.exps, self.of = codes, exps, shape + (cache.D, cache.index)
        self.packed = struct.pack("@2q", codes.data_ptr(), exps.data_ptr())


def mx_cache_bounds_alloc(cache):
    """MxBounds with new buffers for `cache`.  Pages count as unbounded (exps 0xFF: ahead of every scored page) until
    mx_cache_bounds has made their bounds, which it does for the pages of the tokens that it is told of: all of a prompt's
    behind the prompt, then each step's."""
    shape = (cache.num_pages, cache.Hkv)
    return MxBounds(cache, torch.zeros(shape + (2, cache.D), dtype=torch.int8, device=cache.device),
                    torch.full(shape, 0xFF, dtype=torch.uint8, device=cache.device))


def _bounds_of(bounds, cache):
    if bounds.of != (cache.num_pages, cache.Hkv, cache.D, cache.index):
        raise ValueError("bounds are not this cache's")
    return cache.packed + bounds.packed


def mx_cache_bounds(cache, bounds, page_table, seq_lens, T, new_lens=None, dev_status=None, stream=None):
    """Brings up to date the bounds of the pages that hold the last new_lens[b] (None: T; at most T) tokens of every
    sequence: after a write, with the write's lengths."""
    there = _elsewhere(cache, stream)
    if there is not None:
        with there:
            return mx_cache_bounds(cache, bounds, page_table, seq_lens, T, new_lens, dev_status)
    B = page_table.shape[0]
    p = _bounds_of(bounds, cache) + _pack_bounds(B, T, *_table(page_table, B, cache),
                                    _index(seq_lens, B, cache, "seq_lens"), _index(new_lens, B, cache, "new_lens"),
                                    _status(dev_status, cache))
    _check(_c_bounds(p, _raw_stream(cache.index)))


@functools.lru_cache(maxsize=256)
def mx_cache_sparse_attn_workspace_bytes(B, T, Hq, Hkv, D, page_size, max_pages, top):
    """Bytes of scratch mx_cache_sparse_attn needs at these sizes (the C call of the same name)."""
    return int(lib.mx_cache_sparse_attn_workspace_bytes(B, T, Hq, Hkv, D, page_size, max_pages, top))


def mx_cache_sparse_attn(q, cache, bounds, page_table, seq_lens, top, first=1, last=1, new_lens=None, layout=BSHD,
                         softmax_scale=None, o=None, lse=None, blocks=None, workspace=None, dev_status=None, stream=None):
    """mx_cache_attn over `top` pages for every query and KV head: the first `first`, the last `last` (the query's own among
    them), and those whose bounds score highest against the KV head's queries (bsc.h has the score).  Returns (O shaped and
    typed like q, LSE fp32 [B, Hq, T], blocks int32 [B, T, Hkv, top]: the pages' numbers, ascending, then -1).  Bounds must
    be up to date (mx_cache_bounds).  `workspace`: a device tensor of mx_cache_sparse_attn_workspace_bytes(...) bytes that
    no other running call uses, else one is allocated here."""
    there = _elsewhere(cache, stream)
    if there is not None:
        with there:
            return mx_cache_sparse_attn(q, cache, bounds, page_table, seq_lens, top, first, last, new_lens, layout,
                                        softmax_scale, o, lse, blocks, workspace, dev_status)
    dims, qs, dt = _act_dims(q, layout, cache, "q")
    B, T, Hq = dims
    table = _table(page_table, B, cache)
    device = cache.device
    o, o_s = _out_like(q, o, dims, layout, cache, "o", dt)
    if lse is None:
        lse = torch.empty((B, Hq, T), dtype=torch.float32, device=device)
    elif lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, T) or lse.device != device or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 tensor [B, Hq, T] on the cache's device")
    if blocks is None:
        blocks = torch.empty((B, T, cache.Hkv, max(top, 0)), dtype=torch.int32, device=device)
    elif blocks.dtype != torch.int32 or tuple(blocks.shape) != (B, T, cache.Hkv, top) or blocks.device != device or \
            not blocks.is_contiguous():
        raise ValueError("blocks must be a contiguous int32 tensor [B, T, Hkv, top] on the cache's device")
    if workspace is None:
        need = mx_cache_sparse_attn_workspace_bytes(B, T, Hq, cache.Hkv, cache.D, cache.page_size, table[2], top)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    else:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the cache's device")
        need = workspace.numel() * workspace.element_size()
    p = _bounds_of(bounds, cache) + _pack_sparse(q.data_ptr(), o.data_ptr(), lse.data_ptr(), blocks.data_ptr(),
                                    *qs, *o_s, B, T, Hq, dt, cache.D ** -0.5 if softmax_scale is None else softmax_scale, top,
                                    first, last, *table, _index(seq_lens, B, cache, "seq_lens"),
                                    _index(new_lens, B, cache, "new_lens"), _status(dev_status, cache), workspace.data_ptr(),
                                    need)
    _check(_c_sparse(p, _raw_stream(cache.index)))
    return o, lse, blocks
