"""Argument types of the attention sublayer's entry points (include/moe_decode.h),
bound when the library is loaded; without torch, as the library itself."""

from __future__ import annotations

import ctypes

_vp, _i, _f, _sz, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong


class _Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + [
        (n, ctypes.c_int) for n in ("num_pages", "kv_heads", "page_size", "head_dim")]


def bind(L):
    psz, pc = ctypes.POINTER(_sz), ctypes.POINTER(_Cache)
    L.fp8_quant_rows.argtypes = [_vp, _ll, _i, _i, _i, _vp, _vp, _vp]
    L.fp8_block_gemm_workspace_size.argtypes = [_i, _i, _i, psz]
    L.fp8_block_gemm.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _vp, _sz, _vp]
    L.fp8_linear_workspace_size.argtypes = [_i, _i, _i, psz]
    L.fp8_linear.argtypes = [_vp, _ll, _vp, _vp, _i, _i, _i, _i, _vp, _i, _vp, _sz, _vp]
    L.kv_cache_workspace_size.argtypes = [psz]
    L.kv_cache_append.argtypes = [pc, _vp, _ll, _vp, _ll, _vp, _i, _vp, _vp, _i, _i, _i, _vp, _sz, _vp]
    L.decode_attention_workspace_size.argtypes = [_i, _i, _i, _i, psz]
    L.decode_attention.argtypes = [pc, _vp, _ll, _i, _vp, _i, _vp, _vp, _i, _i, _i, _f, _f, _i, _vp, _vp, _vp, _vp, _sz,
                                   _vp]
    for n in ("fp8_quant_rows", "fp8_block_gemm_workspace_size", "fp8_block_gemm", "fp8_linear_workspace_size",
              "fp8_linear", "kv_cache_workspace_size", "kv_cache_append", "decode_attention_workspace_size",
              "decode_attention"):
        getattr(L, n).restype = ctypes.c_int
