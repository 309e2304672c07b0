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

from . import MOE_OK, MoeError, lib, moe_device_status, moe_workspace_init

_vp, _i, _f, _sz, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
_bf16, _f32, _u8, _e4m3, _i32 = torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn, torch.int32
# the current stream's handle and the current device without the objects around them
_raw_stream, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


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


def _fail(rc: int, what: str):
    raise MoeError(rc, what)


def _handle(stream, dev: int) -> int:
    if stream is None:
        return _raw_stream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


# Every call's checks come twice: as one expression that decides, on the way of
# each step, whether all is well (attribute reads cost about 0.1 us each), and as
# these functions, which find what is not and say so.
def _want(t, name, dtype, shape):
    """t is a dense tensor of this dtype and shape (None: any size)."""
    if t.dtype is not dtype and not (dtype is _u8 and t.dtype is _e4m3):
        raise ValueError(f"{name}: {dtype} is wanted, got {t.dtype}")
    if len(t.shape) != len(shape) or any(w is not None and w != g for w, g in zip(shape, t.shape)):
        raise ValueError(f"{name}: shape {list(shape)} is wanted, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a dense tensor is wanted, got strides {t.stride()}")


def _want_rows(x, name, shape):
    """x holds bf16 rows of this shape whose dimensions after the first are dense."""
    if x.dtype is not _bf16:
        raise ValueError(f"{name}: {_bf16} is wanted, got {x.dtype}")
    if len(x.shape) != len(shape) or any(w is not None and w != g for w, g in zip(shape, x.shape)):
        raise ValueError(f"{name}: shape {list(shape)} is wanted, got {list(x.shape)}")
    n = 1
    for size, stride in zip(reversed(x.shape[1:]), reversed(x.stride()[1:])):
        if size != 1 and stride != n:
            raise ValueError(f"{name}: the dimensions after the first must be dense, got strides {x.stride()}")
        n *= size


def _want_device(*tensors):
    """A GPU's pointers go to the library: all on the current CUDA device."""
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError(f"CUDA tensors are wanted, got one on {t.device}")
    for t in tensors:
        if t is not None and t.get_device() != _device():
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{_device()}")


def _want_workspace(workspace):
    if not workspace.is_contiguous():
        raise ValueError("workspace: a dense tensor is wanted")


def _row_stride(M: int, stride: int, n: int) -> int:
    """Elements between rows of n; where there is only one, its stride says nothing."""
    return stride if M > 1 else n + 7 & -8


def _size(what, *args) -> int:
    n = _sz(0)
    rc = getattr(lib(), what)(*[int(a) for a in args], ctypes.byref(n))
    if rc != MOE_OK:
        _fail(rc, what)
    return n.value


def fp8_block_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return _size("fp8_block_gemm_workspace_size", M, N, K)


def fp8_linear_workspace_size(M: int, N: int, K: int) -> int:
    return _size("fp8_linear_workspace_size", M, N, K)


def kv_cache_workspace_size() -> int:
    return _size("kv_cache_workspace_size")


def decode_attention_workspace_size(heads: int, kv_heads: int, head_dim: int, max_new: int) -> int:
    return _size("decode_attention_workspace_size", heads, kv_heads, head_dim, max_new)


def fp8_quant_rows(x, codes, scales, e8m0: bool = False, stream=None):
    """x (bf16 [M, K], any row stride) to E4M3 codes (uint8 [M, K]) and float32
    scales [ceil(K / 128), M rounded up to a multiple of 4]."""
    _want_rows(x, "x", (None, None))
    M, K = x.shape
    _want(codes, "codes", _u8, (M, K))
    _want(scales, "scales", _f32, (-(-K // 128), M + 3 & -4))
    _want_device(x, codes, scales)
    rc = lib().fp8_quant_rows(x.data_ptr(), _row_stride(M, x.stride(0), K), M, K, 1 if e8m0 else 0, codes.data_ptr(),
                              scales.data_ptr(), _handle(stream, x.get_device()))
    if rc != MOE_OK:
        _fail(rc, "fp8_quant_rows")


def _want_weight(w, w_s, out, M):
    _want(w, "w", _u8, (None, None))
    N, K = w.shape
    _want(w_s, "w_s", _f32, (-(-N // 128), -(-K // 128)))
    if out.dtype is not _f32 and out.dtype is not _bf16:
        raise ValueError(f"out: bfloat16 or float32 is wanted, got {out.dtype}")
    _want(out, "out", out.dtype, (M, N))
    return N, K


def fp8_block_gemm(codes, scales, w, w_s, out, workspace, stream=None):
    """out = (codes * scales) . (w * w_s)^T for codes in hand (fp8_quant_rows);
    out bf16 or float32."""
    M = codes.shape[0]
    N, K = _want_weight(w, w_s, out, M)
    _want(codes, "codes", _u8, (M, K))
    _want(scales, "scales", _f32, (-(-K // 128), M + 3 & -4))
    _want_workspace(workspace)
    _want_device(codes, scales, w, w_s, out, workspace)
    rc = lib().fp8_block_gemm(codes.data_ptr(), scales.data_ptr(), w.data_ptr(), w_s.data_ptr(), M, N, K,
                              out.data_ptr(), 1 if out.dtype is _f32 else 0, workspace.data_ptr(), workspace.nbytes,
                              _handle(stream, codes.get_device()))
    if rc != MOE_OK:
        _fail(rc, "fp8_block_gemm")


def _linear_refused(x, w, w_s, out, workspace):
    _want_rows(x, "x", (None, None))
    N, K = _want_weight(w, w_s, out, x.shape[0])
    _want_rows(x, "x", (None, K))
    _want_workspace(workspace)
    _want_device(x, w, w_s, out, workspace)
    raise ValueError("fp8_linear: arguments refused")


def fp8_linear(x, w, w_s, out, workspace, e8m0: bool = False, stream=None):
    """out = x . w^T: x (bf16 [M, K], any row stride) quantised per token per
    128 columns, w (E4M3 [N, K]) with float32 scales w_s for each 128 x 128
    block; out bf16 or float32 [M, N]."""
    if x.dim() != 2 or w.dim() != 2:
        _linear_refused(x, w, w_s, out, workspace)
    M, K = x.shape
    N = w.shape[0]
    sm, sk = x.stride()
    wt, ot, dev = w.dtype, out.dtype, x.get_device()
    if not (x.dtype is _bf16 and (wt is _u8 or wt is _e4m3) and w_s.dtype is _f32 and (ot is _bf16 or ot is _f32)
            and w.shape == (N, K) and w_s.shape == (N + 127 >> 7, K + 127 >> 7) and out.shape == (M, N)
            and (sk == 1 or K == 1) and w.is_contiguous() and w_s.is_contiguous() and out.is_contiguous()
            and workspace.is_contiguous() and x.get_device() == dev and w.get_device() == dev
            and w_s.get_device() == dev and out.get_device() == dev and workspace.get_device() == dev
            and dev >= 0 and dev == _device()):
        _linear_refused(x, w, w_s, out, workspace)
    rc = lib().fp8_linear(x.data_ptr(), sm if M > 1 else K + 7 & -8, w.data_ptr(), w_s.data_ptr(), M, N, K,
                          1 if e8m0 else 0, out.data_ptr(), 1 if ot is _f32 else 0, workspace.data_ptr(),
                          workspace.nbytes, _handle(stream, dev))
    if rc != MOE_OK:
        _fail(rc, "fp8_linear")


def _batch_ok(k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, workspace, dev):
    """The cache and the batch are as _batch_refused wants them."""
    shape, st = k_cache.shape, (k_cache.shape[0], k_cache.shape[1])
    B = lens.shape[0]
    kt, vt = k_cache.dtype, v_cache.dtype
    return ((kt is _u8 or kt is _e4m3) and (vt is _u8 or vt is _e4m3) and v_cache.shape == shape
            and k_scale.dtype is _f32 and v_scale.dtype is _f32 and k_scale.shape == st and v_scale.shape == st
            and page_table.dtype is _i32 and q_start.dtype is _i32 and lens.dtype is _i32
            and page_table.dim() == 2 and page_table.shape[0] == B and q_start.shape == (B + 1,) and lens.dim() == 1
            and k_cache.is_contiguous() and v_cache.is_contiguous() and k_scale.is_contiguous()
            and v_scale.is_contiguous() and page_table.is_contiguous() and q_start.is_contiguous()
            and lens.is_contiguous() and workspace.is_contiguous() and k_cache.get_device() == dev
            and v_cache.get_device() == dev and k_scale.get_device() == dev and v_scale.get_device() == dev
            and page_table.get_device() == dev and q_start.get_device() == dev and lens.get_device() == dev
            and workspace.get_device() == dev)


def _batch_refused(k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, workspace):
    _want(k_cache, "k_cache", _u8, (None, None, None, None))
    shape = tuple(k_cache.shape)
    _want(v_cache, "v_cache", _u8, shape)
    _want(k_scale, "k_scale", _f32, shape[:2])
    _want(v_scale, "v_scale", _f32, shape[:2])
    _want(lens, "lens", _i32, (None,))
    _want(q_start, "q_start", _i32, (lens.shape[0] + 1,))
    _want(page_table, "page_table", _i32, (lens.shape[0], None))
    _want_workspace(workspace)


def kv_cache_append(k, v, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, max_new: int, workspace,
                    stream=None):
    """Write new tokens' keys and values (bf16 [total, kv heads, head dim], any
    token stride) into the cache; see include/moe_decode.h for the batch."""
    dev = k.get_device()
    if k_cache.dim() != 4 or k.dim() != 3 or v.dim() != 3:
        _append_refused(k, v, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, workspace)
    pages, hk, page, d = k_cache.shape
    total = k.shape[0]
    k0, k1, k2 = k.stride()
    v0, v1, v2 = v.stride()
    if not (_batch_ok(k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, workspace, dev)
            and k.dtype is _bf16 and v.dtype is _bf16 and k.shape == (total, hk, d) and v.shape == (total, hk, d)
            and k2 == 1 and v2 == 1 and (hk == 1 or (k1 == d and v1 == d))
            and v.get_device() == dev and dev >= 0 and dev == _device()):
        _append_refused(k, v, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, workspace)
    if total <= 1:
        k0 = v0 = hk * d
    rc = lib().kv_cache_append(
        _Cache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, hk, page, d),
        k.data_ptr(), k0, v.data_ptr(), v0, page_table.data_ptr(), page_table.shape[1], q_start.data_ptr(),
        lens.data_ptr(), lens.shape[0], total, max_new, workspace.data_ptr(), workspace.nbytes, _handle(stream, dev))
    if rc != MOE_OK:
        _fail(rc, "kv_cache_append")


def _append_refused(k, v, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, workspace):
    _batch_refused(k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, workspace)
    row = (k_cache.shape[1], k_cache.shape[3])
    _want_rows(k, "k", (None, *row))
    _want_rows(v, "v", (k.shape[0], *row))
    _want_device(k, v, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, workspace)
    raise ValueError("kv_cache_append: arguments refused")


def decode_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, max_new: int, out, workspace,
                     lse=None, sm_scale: float | None = None, softcap: float = 0.0, window: int = 0, slopes=None,
                     stream=None):
    """Attention of a step's tokens (q bf16 [total, heads, head dim], any token
    stride) over the cache.  out bf16 like q; lse float32 [total, heads] or
    None; sm_scale 1 / sqrt(head dim) by default; slopes float32 [heads]."""
    dev = q.get_device()
    if k_cache.dim() != 4 or q.dim() != 3:
        _attention_refused(q, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, out, workspace, lse, slopes)
    pages, hk, page, d = k_cache.shape
    shape = q.shape
    total, h, dq = shape
    q0, q1, q2 = q.stride()
    if not (_batch_ok(k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, workspace, dev)
            and q.dtype is _bf16 and out.dtype is _bf16 and dq == d and out.shape == shape
            and q2 == 1 and (h == 1 or q1 == d) and out.is_contiguous()
            and out.get_device() == dev and dev >= 0 and dev == _device()
            and (lse is None or (lse.dtype is _f32 and lse.shape == (total, h) and lse.is_contiguous()
                                 and lse.get_device() == dev))
            and (slopes is None or (slopes.dtype is _f32 and slopes.shape == (h,) and slopes.is_contiguous()
                                    and slopes.get_device() == dev))):
        _attention_refused(q, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, out, workspace, lse, slopes)
    rc = lib().decode_attention(
        _Cache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, hk, page, d),
        q.data_ptr(), q0 if total > 1 else h * d, h, page_table.data_ptr(), page_table.shape[1], q_start.data_ptr(),
        lens.data_ptr(), lens.shape[0], total, max_new, 1.0 / math.sqrt(d) if sm_scale is None else sm_scale, softcap,
        window, None if slopes is None else slopes.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
        workspace.data_ptr(), workspace.nbytes, _handle(stream, dev))
    if rc != MOE_OK:
        _fail(rc, "decode_attention")


def _attention_refused(q, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, out, workspace, lse, slopes):
    _batch_refused(k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, workspace)
    _want_rows(q, "q", (None, None, k_cache.shape[3]))
    total, h, d = q.shape
    _want(out, "out", _bf16, (total, h, d))
    if lse is not None:
        _want(lse, "lse", _f32, (total, h))
    if slopes is not None:
        _want(slopes, "slopes", _f32, (h,))
    _want_device(q, out, lse, slopes, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, workspace)
    raise ValueError("decode_attention: arguments refused")


class Fp8KvCache:
    """The tensors of an FP8 paged cache (nothing needs to be initialised)."""

    def __init__(self, num_pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device="cuda"):
        shape = (num_pages, kv_heads, page_size, head_dim)
        self.k, self.v = (torch.empty(shape, dtype=_u8, device=device) for _ in range(2))
        self.k_scale, self.v_scale = (torch.empty(shape[:2], dtype=_f32, device=device) for _ in range(2))


class AttentionDecode:
    """The attention sublayer of a decode step: the fused query, key and value
    projection, the new tokens' keys and values into the cache, attention over it,
    the output projection.  Its output is what rmsnorm_residual adds to the
    residual before MoeDecodeLayer.

    weights: qkv (E4M3 [(heads + 2 kv_heads) * head_dim, hidden]), o (E4M3
    [hidden, heads * head_dim]) and their float32 block scales qkv_s, o_s.
    `rotate(q, k)`, if given, changes the step's queries and keys in place
    (position encodings) before they are used.  softcap, window, slopes and
    sm_scale as decode_attention's."""

    def __init__(self, hidden: int, heads: int, kv_heads: int, head_dim: int, weights: dict, cache: Fp8KvCache,
                 max_tokens: int, max_new: int = 1, e8m0: bool = False, rotate=None, **options):
        self.hidden, self.heads, self.kv_heads, self.head_dim = hidden, heads, kv_heads, head_dim
        self.weights, self.cache, self.max_new, self.e8m0 = weights, cache, max_new, e8m0
        self.rotate, self.options = rotate, options
        self.max_tokens = max_tokens
        rows = (heads + 2 * kv_heads) * head_dim
        device = cache.k.device
        n = max(fp8_linear_workspace_size(max_tokens, rows, hidden),
                fp8_linear_workspace_size(max_tokens, hidden, heads * head_dim),
                decode_attention_workspace_size(heads, kv_heads, head_dim, max_new), kv_cache_workspace_size())
        self.workspace = torch.empty(n, dtype=_u8, device=device)
        moe_workspace_init(self.workspace)
        self.qkv = torch.empty((max_tokens, heads + 2 * kv_heads, head_dim), dtype=_bf16, device=device)
        self.mixed = torch.empty((max_tokens, heads, head_dim), dtype=_bf16, device=device)

    def __call__(self, x, page_table, q_start, lens, out=None, stream=None):
        """x bf16 [tokens, hidden] -> bf16 [tokens, hidden]; page_table, q_start
        and lens as kv_cache_append's (lens with the step's tokens included)."""
        n, h, hk, c, w = x.shape[0], self.heads, self.kv_heads, self.cache, self.weights
        if n > self.max_tokens:
            raise ValueError(f"{n} tokens: at most {self.max_tokens}")
        if out is None:
            out = torch.empty((n, self.hidden), dtype=_bf16, device=x.device)
        qkv, mixed = self.qkv[:n], self.mixed[:n]
        fp8_linear(x, w["qkv"], w["qkv_s"], qkv.view(n, -1), self.workspace, e8m0=self.e8m0, stream=stream)
        q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        if self.rotate is not None:
            self.rotate(q, k)
        kv_cache_append(k, v, c.k, c.v, c.k_scale, c.v_scale, page_table, q_start, lens, self.max_new, self.workspace,
                        stream=stream)
        decode_attention(q, c.k, c.v, c.k_scale, c.v_scale, page_table, q_start, lens, self.max_new, mixed,
                         self.workspace, stream=stream, **self.options)
        fp8_linear(mixed.view(n, -1), w["o"], w["o_s"], out, self.workspace, e8m0=self.e8m0, stream=stream)
        return out

    def status(self) -> int:
        return moe_device_status(self.workspace)
