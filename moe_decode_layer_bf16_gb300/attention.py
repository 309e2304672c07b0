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

import torch

from . import MOE_OK, MoeError, _stream, lib, moe_device_status, moe_workspace_init
from .attention_abi import _Cache, bind  # noqa: F401

_sz = ctypes.c_size_t
_bf16, _f32, _u8, _e4m3, _i32 = torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn, torch.int32


_native = None


def _calls():
    """The extension module that checks the tensors and calls the library; loaded
    with it, and as indispensable."""
    global _native
    if _native is None:
        lib()
        try:
            from . import _calls as native
        except ImportError as e:
            raise RuntimeError(f"_calls.so is not built (python -m moe_decode_layer_bf16_gb300.build): {e}") from e
        _native = native
    return _native


def _fail(rc: int, what: str):
    raise MoeError(rc, what)


def _handle(stream):
    """The stream's handle, or None for the current one."""
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def _torch_stream(stream, device):
    """torch's stream of a stream or a handle (0 is the default stream's)."""
    if isinstance(stream, torch.Stream):
        return stream
    handle = _handle(stream)
    return torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)


# The extension module refuses what is not as an operator wants it without a
# word; these functions find out what it was and say so.
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
        if t is not None and t.get_device() != torch.cuda.current_device():
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")


def _want_workspace(workspace):
    if not workspace.is_contiguous():
        raise ValueError("workspace: a dense tensor is wanted")


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
    # (where there is only one row, its stride says nothing)
    rc = lib().fp8_quant_rows(x.data_ptr(), x.stride(0) if M > 1 else K + 7 & -8, M, K, 1 if e8m0 else 0,
                              codes.data_ptr(), scales.data_ptr(), _stream(stream))
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
                              _stream(stream))
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
    rc = _calls().fp8_linear(x, w, w_s, out, workspace, e8m0, _handle(stream))
    if rc:
        _linear_refused(x, w, w_s, out, workspace) if rc < 0 else _fail(rc, "fp8_linear")


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
    rc = _calls().kv_cache_append(k, v, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, max_new, workspace,
                                  _handle(stream))
    if rc < 0:
        _append_refused(k, v, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, workspace)
    elif rc:
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
    rc = _calls().decode_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, max_new, out,
                                   workspace, lse, sm_scale, softcap, window, slopes, _handle(stream))
    if rc < 0:
        _attention_refused(q, k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens, out, workspace, lse, slopes)
    elif rc:
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
    (position encodings) before they are used; the step's stream is then torch's
    current one.  softcap, window, slopes and sm_scale as decode_attention's."""

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
        if stream is not None:  # (rotate and a new output's memory belong to it as well)
            with torch.cuda.stream(_torch_stream(stream, x.device)):
                return self(x, page_table, q_start, lens, out)
        n, h, hk, c, w = x.shape[0], self.heads, self.kv_heads, self.cache, self.weights
        if n > self.max_tokens:
            raise ValueError(f"{n} tokens: at most {self.max_tokens}")
        if out is None:
            out = torch.empty((n, self.hidden), dtype=_bf16, device=x.device)
        qkv, mixed = self.qkv[:n], self.mixed[:n]
        fp8_linear(x, w["qkv"], w["qkv_s"], qkv.flatten(1), self.workspace, e8m0=self.e8m0)
        q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        if self.rotate is not None:
            self.rotate(q, k)
        kv_cache_append(k, v, c.k, c.v, c.k_scale, c.v_scale, page_table, q_start, lens, self.max_new, self.workspace)
        decode_attention(q, c.k, c.v, c.k_scale, c.v_scale, page_table, q_start, lens, self.max_new, mixed,
                         self.workspace, **self.options)
        fp8_linear(mixed.flatten(1), w["o"], w["o_s"], out, self.workspace, e8m0=self.e8m0)
        return out

    def status(self) -> int:
        return moe_device_status(self.workspace)
