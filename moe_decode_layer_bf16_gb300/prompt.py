"""A prompt's way through the attention sublayer: the layer boundary with FP8
output, pages of the cache given and taken back on the GPU, and attention of
whole prompts over themselves (include/moe_decode.h).

The functions carry the C ABI's names and check and refuse as the attention
module's do.  KvPages keeps the pages of a batch; AttentionPrompt runs the
sublayer over new prompts, as AttentionDecode does over a step's tokens.
"""

from __future__ import annotations

import torch

from . import moe_device_status, moe_workspace_init
from .attention import (AttentionDecode, _bf16, _calls, _f32, _fail, _handle, _i32, _size, _torch_stream, _u8, _want,
                        _want_device, _want_rows, _want_workspace, fp8_block_gemm, fp8_linear, fp8_linear_workspace_size,
                        kv_cache_append, kv_cache_workspace_size)

_i64 = torch.int64


def prompt_attention_workspace_size() -> int:
    return _size("prompt_attention_workspace_size")


def rmsnorm_residual_fp8(residual, gain, codes, scales, residual_out, eps: float, x=None, out=None, e8m0: bool = False,
                         stream=None):
    """residual_out = x + residual (bf16 [M, H], any row stride; x may be None);
    its RMSNorm as E4M3 codes (uint8 [M, H]) and float32 scales
    [ceil(H / 128), M rounded up to a multiple of 4], and in bf16 if out is given."""
    rc = _calls().rmsnorm_residual_fp8(residual, gain, codes, scales, residual_out, eps, x, out, e8m0, _handle(stream))
    if rc < 0:
        _norm_refused(residual, gain, codes, scales, residual_out, x, out)
    elif rc:
        _fail(rc, "rmsnorm_residual_fp8")


def _norm_refused(residual, gain, codes, scales, residual_out, x, out):
    _want_rows(residual, "residual", (None, None))
    M, H = residual.shape
    _want(gain, "gain", _bf16, (H,))
    _want(codes, "codes", _u8, (M, H))
    _want(scales, "scales", _f32, (-(-H // 128), M + 3 & -4))
    _want(residual_out, "residual_out", _bf16, (M, H))
    if x is not None:
        _want_rows(x, "x", (M, H))
    if out is not None:
        _want(out, "out", _bf16, (M, H))
    _want_device(residual, gain, codes, scales, residual_out, x, out)
    raise ValueError("rmsnorm_residual_fp8: arguments refused")


def _pages_refused(page_table, lens, free_pages, free_state, lens_out, free_out, workspace):
    _want(page_table, "page_table", _i32, (None, None))
    B = page_table.shape[0]
    _want(lens, "lens", _i32, (B,))
    _want(free_pages, "free_pages", _i32, (None,))
    _want(free_state, "free_state", _i32, (2,))
    _want(lens_out, "lens_out", _i32, (B,))
    _want(free_out, "free_out", _i32, (2,))
    _want_workspace(workspace)


def kv_pages_extend(page_table, lens, new, free_pages, free_state, page_size: int, num_pages: int, q_start, lens_out, free_out,
                    positions, slots, workspace, stream=None):
    """Pages for the step's new tokens (int32 [B]) of each sequence, from the stack
    free_pages[:free_state[0]] into page_table; the step's row starts, lengths,
    positions (int32 [rows]) and slots (int64 [rows]).  lens_out may be lens and
    free_out free_state; see include/moe_decode.h for who is served."""
    rc = _calls().kv_pages_extend(page_table, lens, new, free_pages, free_state, page_size, num_pages, q_start, lens_out,
                                  free_out, positions, slots, workspace, _handle(stream))
    if rc < 0:
        _extend_refused(page_table, lens, new, free_pages, free_state, q_start, lens_out, free_out, positions, slots, workspace)
    elif rc:
        _fail(rc, "kv_pages_extend")


def _extend_refused(page_table, lens, new, free_pages, free_state, q_start, lens_out, free_out, positions, slots, workspace):
    _pages_refused(page_table, lens, free_pages, free_state, lens_out, free_out, workspace)
    _want(new, "new", _i32, (lens.shape[0],))
    _want(q_start, "q_start", _i32, (lens.shape[0] + 1,))
    _want(positions, "positions", _i32, (None,))
    _want(slots, "slots", _i64, tuple(positions.shape))
    _want_device(page_table, lens, new, free_pages, free_state, q_start, lens_out, free_out, positions, slots, workspace)
    raise ValueError("kv_pages_extend: arguments refused")


def kv_pages_release(page_table, lens, done, free_pages, free_state, page_size: int, num_pages: int, lens_out, free_out,
                     workspace, stream=None):
    """The pages of the sequences with done (bool or uint8 [B]) back onto the stack;
    their lengths become 0."""
    rc = _calls().kv_pages_release(page_table, lens, done, free_pages, free_state, page_size, num_pages, lens_out, free_out,
                                   workspace, _handle(stream))
    if rc < 0:
        _release_refused(page_table, lens, done, free_pages, free_state, lens_out, free_out, workspace)
    elif rc:
        _fail(rc, "kv_pages_release")


def _release_refused(page_table, lens, done, free_pages, free_state, lens_out, free_out, workspace):
    _pages_refused(page_table, lens, free_pages, free_state, lens_out, free_out, workspace)
    _want(done, "done", _u8 if done.dtype is _u8 else torch.bool, (lens.shape[0],))
    _want_device(page_table, lens, done, free_pages, free_state, lens_out, free_out, workspace)
    raise ValueError("kv_pages_release: arguments refused")


def prompt_attention(q, k, v, q_start, out, workspace, lse=None, sm_scale: float | None = None, softcap: float = 0.0,
                     window: int = 0, slopes=None, stream=None, lens=None):
    """Causal attention of packed prompts over themselves: q bf16 [total, heads,
    head dim], k and v bf16 [total, kv heads, head dim], any row stride; rows
    [q_start[b], q_start[b + 1]) are a prompt.  out bf16 like q; lse float32
    [total, heads] or None; sm_scale 1 / sqrt(head dim) by default; slopes
    float32 [heads].  With lens (int32, a value for each prompt: the tokens that its
    sequence holds) a prompt whose rows are not all of them is left out, and the
    workspace's status says so."""
    rc = _calls().prompt_attention(q, k, v, q_start, out, workspace, lse, sm_scale, softcap, window, slopes, _handle(stream),
                                   lens)
    if rc < 0:
        _prompt_refused(q, k, v, q_start, out, workspace, lse, slopes, lens)
    elif rc:
        _fail(rc, "prompt_attention")


def _prompt_refused(q, k, v, q_start, out, workspace, lse, slopes, lens):
    _want_rows(q, "q", (None, None, None))
    total, h, d = q.shape
    _want_rows(k, "k", (total, None, d))
    _want_rows(v, "v", tuple(k.shape))
    _want(q_start, "q_start", _i32, (None,))
    if q_start.shape[0] < 1:
        raise ValueError("q_start: one value more than prompts is wanted")
    _want(out, "out", _bf16, (total, h, d))
    if lse is not None:
        _want(lse, "lse", _f32, (total, h))
    if slopes is not None:
        _want(slopes, "slopes", _f32, (h,))
    if lens is not None:
        _want(lens, "lens", _i32, (q_start.shape[0] - 1,))
    _want_workspace(workspace)
    _want_device(q, k, v, q_start, out, lse, slopes, lens, workspace)
    raise ValueError("prompt_attention: arguments refused")


class KvPages:
    """The pages of a batch's sequences in an Fp8KvCache: page table, lengths and the
    stack of free pages, kept on the GPU and changed by steps that may be captured.

    After extend: page_table, q_start and lens are what kv_cache_append and
    decode_attention take, positions and slots [max_rows] describe the step's rows
    (-1 behind the last), free[0] counts the pages left and free[1] those that were
    asked for and not given.  A sequence can also stay as it was because it outgrew its
    table or the step max_rows: status() says so."""

    def __init__(self, cache, batch: int, width: int, max_rows: int):
        n, _, self.page_size, _ = cache.k.shape
        device = cache.k.device
        self.num_pages = n

        def ints(*shape):
            return torch.zeros(shape, dtype=_i32, device=device)

        self.page_table, self.lens, self.q_start = ints(batch, width).fill_(-1), ints(batch), ints(batch + 1)
        self.free_pages = torch.arange(n - 1, -1, -1, dtype=_i32, device=device)  # (page 0 on top)
        self.free = torch.tensor([n, 0], dtype=_i32, device=device)
        self.positions = ints(max_rows).fill_(-1)
        self.slots = torch.full((max_rows,), -1, dtype=_i64, device=device)
        self.workspace = torch.empty(kv_cache_workspace_size(), dtype=_u8, device=device)
        moe_workspace_init(self.workspace)

    def extend(self, new, stream=None):
        """Room for new (int32 [batch]) tokens of each sequence."""
        kv_pages_extend(self.page_table, self.lens, new, self.free_pages, self.free, self.page_size, self.num_pages,
                        self.q_start, self.lens, self.free, self.positions, self.slots, self.workspace, stream=stream)

    def release(self, done, stream=None):
        """The pages of the sequences with done (bool [batch]) are free again."""
        kv_pages_release(self.page_table, self.lens, done, self.free_pages, self.free, self.page_size, self.num_pages,
                         self.lens, self.free, self.workspace, stream=stream)

    def status(self) -> int:
        return moe_device_status(self.workspace)


class AttentionPrompt:
    """The attention sublayer over whole new prompts, with an AttentionDecode's weights,
    cache and options: the fused projection, keys and values into the cache (for the
    steps that follow), attention of the prompts over themselves, the output
    projection."""

    def __init__(self, decode: AttentionDecode, max_tokens: int):
        self.decode, self.max_tokens = decode, max_tokens
        d = decode
        h, hk, dim, device = d.heads, d.kv_heads, d.head_dim, d.cache.k.device
        n = max(fp8_linear_workspace_size(max_tokens, (h + 2 * hk) * dim, d.hidden),
                fp8_linear_workspace_size(max_tokens, d.hidden, h * dim), prompt_attention_workspace_size(),
                kv_cache_workspace_size())
        self.workspace = torch.empty(n, dtype=_u8, device=device)
        moe_workspace_init(self.workspace)
        self.qkv = torch.empty((max_tokens, h + 2 * hk, dim), dtype=_bf16, device=device)
        self.mixed = torch.empty((max_tokens, h, dim), dtype=_bf16, device=device)

    def __call__(self, x, page_table, q_start, lens, max_new: int, out=None, stream=None):
        """x: bf16 [tokens, hidden], or the (codes, scales) of rmsnorm_residual_fp8;
        page_table, q_start and lens as kv_cache_append's; max_new a bound of a
        sequence's rows.  A sequence with rows is new: all its tokens are in the step
        (lens[b] = q_start[b + 1] - q_start[b]).  One that goes on is decode_attention's:
        its keys and values go into the cache, but its rows are not attended, and
        status() says MOE_ERR_INVALID_ARG.  Sequences without rows are left alone.
        Rows of no sequence, or of one that goes on, come out as something.  Returns
        bf16 [tokens, hidden]."""
        quantised = isinstance(x, (tuple, list))
        rows = x[0] if quantised else x
        if stream is not None:  # (rotate and a new output's memory belong to it as well)
            with torch.cuda.stream(_torch_stream(stream, rows.device)):
                return self(x, page_table, q_start, lens, max_new, out)
        d, n = self.decode, rows.shape[0]
        h, hk, c, w = d.heads, d.kv_heads, d.cache, d.weights
        if n > self.max_tokens:
            raise ValueError(f"{n} tokens: at most {self.max_tokens}")
        if out is None:
            out = torch.empty((n, d.hidden), dtype=_bf16, device=rows.device)
        qkv, mixed = self.qkv[:n], self.mixed[:n]
        if quantised:
            fp8_block_gemm(x[0], x[1], w["qkv"], w["qkv_s"], qkv.flatten(1), self.workspace)
        else:
            fp8_linear(x, w["qkv"], w["qkv_s"], qkv.flatten(1), self.workspace, e8m0=d.e8m0)
        q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        if d.rotate is not None:
            d.rotate(q, k)
        kv_cache_append(k, v, c.k, c.v, c.k_scale, c.v_scale, page_table, q_start, lens, max_new, self.workspace)
        prompt_attention(q, k, v, q_start, mixed, self.workspace, lens=lens, **d.options)
        fp8_linear(mixed.flatten(1), w["o"], w["o_s"], out, self.workspace, e8m0=d.e8m0)
        return out

    def status(self) -> int:
        return moe_device_status(self.workspace)
