"""The attention sublayer's operators: FP8 block-scaled linear layers, the FP8
paged key/value cache and attention over it (include/moe_decode.h).

The functions carry the C ABI's names.  They check dtypes, shapes, strides and
devices (ValueError); what the library itself refuses raises MoeError.  As
everywhere in this package, work is only enqueued, on the current stream
unless `stream` is given, and outputs and workspaces are the caller's.

AttentionDecode runs them together as a decode step does.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import _check, _ptr, _stream, lib, moe_device_status, moe_workspace_init

_vp, _i, _f, _sz, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong


class _Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + [
        (n, ctypes.c_int) for n in ("num_pages", "kv_heads", "page_size", "head_dim")]


def bind(L):
    """Argument types of this module's entry points (called when the library is loaded)."""
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


def _want(t, name, dtype, shape):
    """t is a dense tensor of this dtype and shape (None: any size)."""
    if t.dtype is not dtype and not (dtype is torch.uint8 and t.dtype is torch.float8_e4m3fn):
        raise ValueError(f"{name}: {dtype} is wanted, got {t.dtype}")
    if len(t.shape) != len(shape) or any(w is not None and w != g for w, g in zip(shape, t.shape)):
        raise ValueError(f"{name}: shape {list(shape)} is wanted, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a dense tensor is wanted, got strides {t.stride()}")


def _same_device(first, *tensors):
    """A GPU's pointers go to the library: all on one CUDA device."""
    if not first.is_cuda:
        raise ValueError("CUDA tensors are wanted")
    d = first.device
    for t in tensors:
        if t is not None and t.device != d:
            raise ValueError(f"tensors on {d} and {t.device}")


def _rows_stride(x, name, shape):
    """Token stride of bf16 rows whose other dimensions are dense."""
    if x.dtype is not torch.bfloat16:
        raise ValueError(f"{name}: torch.bfloat16 is wanted, got {x.dtype}")
    if len(x.shape) != len(shape) or any(w is not None and w != g for w, g in zip(shape, x.shape)):
        raise ValueError(f"{name}: shape {list(shape)} is wanted, got {list(x.shape)}")
    st, n = x.stride(), 1
    for size, stride in zip(reversed(x.shape[1:]), reversed(st[1:])):
        if size != 1 and stride != n:
            raise ValueError(f"{name}: the dimensions after the first must be dense, got strides {st}")
        n *= size
    return st[0] if x.shape[0] > 1 else max(n, (n + 7) // 8 * 8)


def fp8_quant_rows(x, codes, scales, e8m0: bool = False, stream=None):
    """x (bf16 [M, K], any row stride) to E4M3 codes (uint8 [M, K]) and float32
    scales [ceil(K / 128), M rounded up to a multiple of 4]."""
    M, K = x.shape
    ldx = _rows_stride(x, "x", (M, K))
    _want(codes, "codes", torch.uint8, (M, K))
    _want(scales, "scales", torch.float32, (-(-K // 128), -(-M // 4) * 4))
    _same_device(x, codes, scales)
    _check(lib().fp8_quant_rows(x.data_ptr(), ldx, M, K, 1 if e8m0 else 0, codes.data_ptr(), scales.data_ptr(),
                                _stream(stream)), "fp8_quant_rows")


def _size(what, *args) -> int:
    n = _sz(0)
    _check(getattr(lib(), what)(*[int(a) for a in args], ctypes.byref(n)), what)
    return n.value


def fp8_block_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return _size("fp8_block_gemm_workspace_size", M, N, K)


def fp8_linear_workspace_size(M: int, N: int, K: int) -> int:
    return _size("fp8_linear_workspace_size", M, N, K)


def kv_cache_workspace_size() -> int:
    return _size("kv_cache_workspace_size")


def decode_attention_workspace_size(heads: int, kv_heads: int, head_dim: int, max_new: int) -> int:
    return _size("decode_attention_workspace_size", heads, kv_heads, head_dim, max_new)


def _weight(w, w_s, out, M):
    if w.dim() != 2:
        raise ValueError(f"w: [N, K] is wanted, got {list(w.shape)}")
    N, K = w.shape
    _want(w, "w", torch.uint8, (N, K))
    _want(w_s, "w_s", torch.float32, (-(-N // 128), -(-K // 128)))
    if out.dtype is not torch.float32 and out.dtype is not torch.bfloat16:
        raise ValueError(f"out: bfloat16 or float32 is wanted, got {out.dtype}")
    _want(out, "out", out.dtype, (M, N))
    return N, K, 1 if out.dtype is torch.float32 else 0


def fp8_block_gemm(codes, scales, w, w_s, out, workspace, stream=None):
    """out = (codes * scales) . (w * w_s)^T for codes in hand; out bf16 or float32."""
    M = codes.shape[0]
    N, K, f32 = _weight(w, w_s, out, M)
    _want(codes, "codes", torch.uint8, (M, K))
    _want(scales, "scales", torch.float32, (-(-K // 128), -(-M // 4) * 4))
    _same_device(codes, scales, w, w_s, out, workspace)
    _check(lib().fp8_block_gemm(codes.data_ptr(), scales.data_ptr(), w.data_ptr(), w_s.data_ptr(), M, N, K,
                                out.data_ptr(), f32, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                _stream(stream)), "fp8_block_gemm")


def fp8_linear(x, w, w_s, out, workspace, e8m0: bool = False, stream=None):
    """out = x . w^T: x (bf16 [M, K], any row stride) quantised per token per
    128 columns, w (E4M3 [N, K]) with float32 scales w_s for each 128 x 128
    block; out bf16 or float32 [M, N]."""
    M = x.shape[0]
    N, K, f32 = _weight(w, w_s, out, M)
    ldx = _rows_stride(x, "x", (M, K))
    _same_device(x, w, w_s, out, workspace)
    _check(lib().fp8_linear(x.data_ptr(), ldx, w.data_ptr(), w_s.data_ptr(), M, N, K, 1 if e8m0 else 0, out.data_ptr(),
                            f32, workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream)),
           "fp8_linear")


def _batch(k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens):
    if k_cache.dim() != 4:
        raise ValueError(f"k_cache: [pages, kv heads, page size, head dim] is wanted, got {list(k_cache.shape)}")
    shape = k_cache.shape
    pages, hk, page, d = shape
    _want(k_cache, "k_cache", torch.uint8, shape)
    _want(v_cache, "v_cache", torch.uint8, shape)
    _want(k_scale, "k_scale", torch.float32, (pages, hk))
    _want(v_scale, "v_scale", torch.float32, (pages, hk))
    B = lens.shape[0]
    _want(lens, "lens", torch.int32, (B,))
    _want(q_start, "q_start", torch.int32, (B + 1,))
    _want(page_table, "page_table", torch.int32, (B, None))
    c = _Cache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, hk, page, d)
    return c, B, hk, d


def kv_cache_append(k, v, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, max_new: int, workspace,
                    stream=None):
    """Write new tokens' keys and values (bf16 [total, kv heads, head dim], any
    token stride) into the cache; see include/moe_decode.h for the batch."""
    c, B, hk, d = _batch(k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens)
    total = k.shape[0]
    ks = _rows_stride(k, "k", (total, hk, d))
    vs = _rows_stride(v, "v", (total, hk, d))
    _same_device(k, v, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, workspace)
    _check(lib().kv_cache_append(c, k.data_ptr(), ks, v.data_ptr(), vs, page_table.data_ptr(), page_table.shape[1],
                                 q_start.data_ptr(), lens.data_ptr(), B, total, max_new, workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), _stream(stream)), "kv_cache_append")


def decode_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, max_new: int, out, workspace,
                     lse=None, sm_scale: float | None = None, softcap: float = 0.0, window: int = 0, slopes=None,
                     stream=None):
    """Attention of a step's tokens (q bf16 [total, heads, head dim], any token
    stride) over the cache.  out bf16 like q; lse float32 [total, heads] or
    None; sm_scale 1 / sqrt(head dim) by default; slopes float32 [heads]."""
    c, B, hk, d = _batch(k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens)
    if q.dim() != 3:
        raise ValueError(f"q: [tokens, heads, head dim] is wanted, got {list(q.shape)}")
    total, h, _ = q.shape
    qs = _rows_stride(q, "q", (total, h, d))
    _want(out, "out", torch.bfloat16, (total, h, d))
    if lse is not None:
        _want(lse, "lse", torch.float32, (total, h))
    if slopes is not None:
        _want(slopes, "slopes", torch.float32, (h,))
    _same_device(q, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, out, workspace, lse, slopes)
    _check(lib().decode_attention(c, q.data_ptr(), qs, h, page_table.data_ptr(), page_table.shape[1],
                                  q_start.data_ptr(), lens.data_ptr(), B, total, max_new,
                                  1.0 / math.sqrt(d) if sm_scale is None else sm_scale, softcap, window, _ptr(slopes),
                                  out.data_ptr(), _ptr(lse), workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), _stream(stream)), "decode_attention")
