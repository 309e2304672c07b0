/*
 * moe_decode.h -- C ABI of the GB300 (sm_103a) MoE decode-layer library
 * (libmoe_decode.so).
 *
 * One low-batch decode step of a DeepSeek/GLM-style MoE layer, as the vLLM
 * specialized-decode executor pages describe it:
 *   [decode page] vllm.models.glm5next.nvidia.specialized_decode.runtime.decode
 *   [draft page]  vllm.models.glm5next.nvidia.specialized_decode.runtime.draft
 *
 * Conventions shared by every entry point
 *   - All tensor arguments are DEVICE pointers to dense row-major arrays that
 *     the caller allocated on the current CUDA device.  The library never
 *     allocates, frees or synchronises (moe_device_status excepted), and keeps
 *     no pointer past return.  Weights are read, never written (the decode
 *     executor leaves the model's own weights untouched: [decode page] class
 *     SpecializedDecode).
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Work is only enqueued; every call is stream-ordered.
 *   - Return value: MOE_OK or an error code below.  Argument errors are found
 *     on the host before anything is enqueued.  There is no CPU fallback:
 *     an unsupported shape returns MOE_ERR_UNSUPPORTED and the caller decides
 *     (the pages' executors likewise refuse unsupported configurations and
 *     leave the step to the stock forward).
 *   - bf16 = IEEE bfloat16 stored as uint16; fp8 = E4M3 (OCP "E4M3FN") codes
 *     stored as uint8; fp32 = IEEE float.
 */
#ifndef MOE_DECODE_H
#define MOE_DECODE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,          /* null pointer, negative size, bad value  */
  MOE_ERR_UNSUPPORTED = 2,          /* shape outside the supported range        */
  MOE_ERR_WORKSPACE_TOO_SMALL = 3,  /* ws_bytes below the *_workspace_size     */
  MOE_ERR_CUDA = 4,                 /* a CUDA runtime call or launch failed     */
  MOE_ERR_DEVICE_TIMEOUT = 5,       /* a bounded device-side wait gave up       */
  MOE_ERR_SCRATCH_LIMIT = 6         /* the problem needs more than the library's
                                       static scratch (splitk_gemm_bf16_noalloc) */
};

/*
 * Layer dimensions and switches ([decode page] LayerStages._build_mega: the
 * routed-expert kernel is built from num_experts_per_tok, swiglu_limit,
 * routed_scaling_factor and the e8m0 switch; only sigmoid scoring with
 * n_group == 1 and norm_topk_prob is accepted, which is the only routing this
 * library implements).
 *   hidden        H, multiple of 128, <= 16384
 *   inter         I (moe_intermediate_size), multiple of 128, <= 8192
 *   shared_inter  I_s of the shared expert, multiple of 128 (0 = none)
 *   num_experts   E routed experts, 1 <= E <= 512
 *   top_k         k, 1 <= k <= min(E, 16)
 *   routed_scaling  multiplies the normalised top-k weights
 *   swiglu_limit  L in h = silu(min(g, L)) * clamp(u, -L, L); +inf disables it
 *   rms_eps       epsilon inside the RMSNorm square root
 *   e8m0          nonzero: activation block scales are rounded up to powers of
 *                 two (the weights' scales are then expected to be powers of
 *                 two as well; they are used as given either way)
 */
typedef struct moe_layer_dims {
  int hidden;
  int inter;
  int shared_inter;
  int num_experts;
  int top_k;
  float routed_scaling;
  float swiglu_limit;
  float rms_eps;
  int e8m0;
} moe_layer_dims;

/*
 * Weights of one MoE layer ([decode page] LayerStages._build_mega:
 * w13_weight, w13_weight_scale_inv, w2_weight, w2_weight_scale_inv, the
 * shared expert's gate_up_proj / down_proj with their weight_scale_inv, the
 * gate's bf16 weight and e_score_correction_bias).
 *   router_w  bf16 [E, H]
 *   sel_bias  fp32 [E] or NULL: added to the sigmoid scores for selection only
 *   w13       fp8 [E, 2I, H]: rows [0, I) gate, rows [I, 2I) up
 *   w13_s     fp32 [E, 2I/128, H/128]: scale of each 128x128 block (w = code * s)
 *   w2        fp8 [E, H, I];  w2_s fp32 [E, H/128, I/128]
 *   sw13, sw13_s, sw2, sw2_s: the shared expert alike, without the E dimension
 *             (NULL when shared_inter == 0)
 *   norm_gain bf16 [H]: gain of the RMSNorm at the layer boundary
 * All weight pointers must be 16-byte aligned.
 */
typedef struct moe_layer_weights {
  const void *router_w;
  const float *sel_bias;
  const uint8_t *w13;
  const float *w13_s;
  const uint8_t *w2;
  const float *w2_s;
  const uint8_t *sw13;
  const float *sw13_s;
  const uint8_t *sw2;
  const float *sw2_s;
  const void *norm_gain;
} moe_layer_weights;

/* Bytes of device workspace moe_decode_layer needs for up to max_tokens
 * tokens (1 <= max_tokens <= 4096, max_tokens * top_k <= 4096). */
int moe_decode_workspace_size(const moe_layer_dims *dims, int max_tokens, size_t *bytes);

/* Zero a workspace (moe_decode_layer's or splitk_gemm_bf16's) once before its
 * first use.  Calls leave their counters at zero for the next call, so this
 * is needed only once per buffer, and again after a call returned an error
 * (a launch that failed part-way can leave a counter set). */
int moe_workspace_init(void *ws, size_t ws_bytes, void *stream);

/*
 * One decode step of the MoE layer plus the layer boundary, for M tokens:
 *   logits = x . router_w^T (fp32); s = sigmoid(logits); sel = s + sel_bias;
 *   ids = top-k of sel (descending; ties to the lower id);
 *   w = s[ids] / sum(s[ids]) * routed_scaling;
 *   route order: stable counting sort of r = t*k + j by expert;
 *   per routed expert and for the shared expert (weight 1), on FP8 activations
 *   quantised per token per 128-column group (scale = amax/448):
 *     [g; u] = x . w13^T, h = silu(min(g, L)) * clamp(u, -L, L),
 *     h quantised likewise, y = h . w2^T;
 *   m = sum_j w_j * y_(t,j) + y_shared;  r' = m + residual;
 *   residual_out = bf16(r');  out = bf16(r' * rsqrt(mean(r'^2) + eps) * gain).
 * ([decode page] LayerStages._mega_moe / _router; [draft page]
 * SpecializedDraft.reduced_norm: the boundary returns the normalised sum and
 * the updated residual.)
 *
 *   x, residual      bf16 [M, H] inputs (may not alias the outputs)
 *   out, residual_out  bf16 [M, H] outputs
 *   topk_ids         int32 [M, k] or NULL; topk_w fp32 [M, k] or NULL
 *   sorted_routes    int32 [M*k] or NULL: expanded route indices grouped by
 *                    expert (ascending), ascending within an expert
 *   expert_offsets   int32 [E+1] or NULL: start of each expert's routes
 *   workspace        from moe_decode_workspace_size(dims, max_tokens >= M),
 *                    zeroed once by moe_workspace_init; one workspace must not
 *                    be used by two calls that may run concurrently
 * M == 0 is a no-op.  Launches three kernels (router + top-k + route order;
 * the expert kernel; finalize + residual + RMSNorm), four when the
 * tensor-core expert kernel serves an MoE layer (the routed tokens' x codes
 * are first gathered in route order); moe_decode_layer_plan reports which.
 * The expert kernel is the warp-MMA kernel for narrow steps and the tcgen05
 * kernel where an expert's tokens can make a real contraction (a dense layer
 * from 4 tokens, an MoE layer from 16 tokens); both compute the same results
 * up to fp32 summation order and the SwiGLU's exponential.
 *
 * Dense layers ([decode page] LayerStages._build_dense: a dense FP8 MLP run as
 * GEMVs): num_experts = 0, top_k = 0, inter = 0 and the MLP's weights in the
 * shared-expert slot (sw13 [2 I_s, H], sw2 [H, I_s], I_s <= 32768); router_w,
 * w13 and w2 are not read and may be NULL.  Then m = y_shared and the same
 * boundary follows; topk_ids / topk_w / sorted_routes are empty and
 * expert_offsets[0] = 0.
 */
int moe_decode_layer(const moe_layer_dims *dims, const moe_layer_weights *w, int M,
                     const void *x, const void *residual, void *out, void *residual_out,
                     int32_t *topk_ids, float *topk_w, int32_t *sorted_routes,
                     int32_t *expert_offsets, void *workspace, size_t ws_bytes,
                     void *stream);

/* moe_decode_layer that also records four CUDA events (cudaEvent_t passed as
 * void*) on `stream`: events[0] before the router kernel, [1] before the
 * expert phase (the gather of routed rows, when it runs, and the expert
 * kernel), [2] before the boundary kernel, [3] after it, so that a caller can
 * time each phase.  The events are created by the caller. */
int moe_decode_layer_traced(const moe_layer_dims *dims, const moe_layer_weights *w, int M,
                            const void *x, const void *residual, void *out, void *residual_out,
                            int32_t *topk_ids, float *topk_w, int32_t *sorted_routes,
                            int32_t *expert_offsets, void *workspace, size_t ws_bytes,
                            void *stream, void *const *events);

/*
 * Tensor parallelism over each expert's intermediate dimension ([decode page]
 * LayerStages leaves the MoE sublayer "TP-partial"; [draft page] module
 * docstring: the boundaries fuse the all-reduce with the residual add and the
 * RMSNorm).  Rank g of G holds, of every routed expert and of the shared
 * expert, the gate rows [g I/G, (g+1) I/G) and the same up rows of w13, and the
 * same columns of w2, with their block scales (I/G and I_s/G multiples of 128,
 * so that no 128 x 128 scale block and no h quantisation group straddles two
 * ranks).  A rank's shard is therefore an MoE layer with inter = I/G and
 * shared_inter = I_s/G (router weight and bias replicated), and:
 *
 * moe_decode_layer_partial: moe_decode_layer on a rank's shard up to the
 *   weighted finalize: m_out (fp32 [M, H]) = sum_j w_j * y_(t,j) + y_shared,
 *   this rank's share of m; the ranks' m_out sum to the whole layer's m.  No
 *   residual, gain or bf16 outputs (norm_gain may be NULL).  Same workspace
 *   and routing outputs as moe_decode_layer; launches its kernels alike (the
 *   boundary kernel writes m_out instead of normalising).
 *
 * moe_tp_boundary: the layer boundary over G partial sums in this GPU's
 *   memory (gathered by the caller, e.g. an all-gather or peer copies):
 *   m = sum_{g < G} partials[g] (in rank order, fp32), r' = m + residual,
 *   residual_out = bf16(r'), out = bf16(bf16(r') * rsqrt(mean(bf16(r')^2) +
 *   eps) * gain).  partials fp32 [G, M, H]; the rest as rmsnorm_residual.
 */
int moe_decode_layer_partial(const moe_layer_dims *dims, const moe_layer_weights *w, int M,
                             const void *x, float *m_out, int32_t *topk_ids, float *topk_w,
                             int32_t *sorted_routes, int32_t *expert_offsets, void *workspace,
                             size_t ws_bytes, void *stream);
int moe_tp_boundary(const float *partials, int G, const void *residual, const void *gain, int M, int H,
                    float eps, void *out, void *residual_out, void *stream);

/* Bytes of workspace splitk_gemm_bf16 needs for this shape and split_k. */
int splitk_gemm_workspace_size(int M, int N, int K, int split_k, size_t *bytes);

/*
 * Split-K BF16 projection ([draft page] module docstring: the draft's BF16
 * projections such as eh_proj run a split-K GEMM above two tokens;
 * SpecializedDraft.run.  [decode page] LayerStages._router passes its split
 * count to the router's split-K GEMM explicitly):
 *   C[M, N] = alpha * A[M, K] . W[N, K]^T, fp32 accumulation.
 *   A bf16 [M, K]; W bf16 [N, K]; C bf16 [M, N] (c_fp32 == 0) or fp32 [M, N].
 *   1 <= M <= 256, N % 16 == 0, K % 128 == 0; A, W 16-byte aligned.
 *   split_k  0: the library divides the K dimension over the whole GPU
 *            (stream-K: every SM streams an equal share of W);
 *            S > 0: every (token chunk, 64-row tile) of C is cut into exactly
 *            S K-segments of K/(128 S) k-blocks each (rounded), one CTA a
 *            segment; 1 <= S <= K/128 (MOE_ERR_UNSUPPORTED above, a negative
 *            value is MOE_ERR_INVALID_ARG).
 * Partial sums are reduced in segment order, so results are deterministic for
 * a given split; different splits may differ in the last bits.
 */
int splitk_gemm_bf16(const void *A, const void *W, void *C, int c_fp32, int M, int N, int K,
                     int split_k, float alpha, void *ws, size_t ws_bytes, void *stream);

/*
 * splitk_gemm_bf16 without a caller-provided workspace, for callers that
 * cannot allocate device memory at the point where they run the projection
 * (for example a plugin whose enqueue function must not call cudaMalloc, or a
 * runtime that hands out only a fixed pool it owns).  No counterpart on the
 * source pages: this is an interface convenience of this library.
 *
 * Same arguments and result as splitk_gemm_bf16 (the same plan, hence the
 * same bits), minus ws / ws_bytes.  The
 * partial sums and tile counters live in one static device array of
 * MOE_NOALLOC_SCRATCH_BYTES (8 MiB) in the library, which every GPU that
 * loads the library holds until the process exits.  Nothing is allocated or
 * freed.  The first call on a device looks up that array's device address
 * (cudaGetSymbolAddress) and caches it; make that first call before any work
 * whose ordering depends on it.  Every call shares the array: calls that may
 * overlap on the GPU (different streams, or different host threads without
 * ordering) race and corrupt each other's results; serialise them on one
 * stream.  A shape whose split needs more scratch than the limit returns
 * MOE_ERR_SCRATCH_LIMIT before anything is enqueued.  The tile counters are
 * cleared (cudaMemsetAsync on the array, no allocation) at every call.
 */
#define MOE_NOALLOC_SCRATCH_BYTES (8u << 20)
int splitk_gemm_bf16_noalloc(const void *A, const void *W, void *C, int c_fp32, int M, int N, int K,
                             int split_k, float alpha, void *stream);

/* Test hook: fill the whole static scratch of splitk_gemm_bf16_noalloc on the
 * current device with `byte` (stream-ordered), so that a test can check that
 * a call clears the counters it uses whatever an earlier call left there. */
int moe_debug_fill_noalloc_scratch(int byte, void *stream);

/*
 * Layer boundary: optional weighted top-k finalize, residual add, RMSNorm
 * ([draft page] SpecializedDraft.reduced_norm; [decode page] _mega_moe hands
 * the routed rows over unfinalized, in expanded order, for this step):
 *   m[t] = (x ? x[t] : 0) + (rows ? sum_j route_w[t, j] * rows[t*k + j] : 0)
 *          + (shared ? shared[t] : 0)
 *   r' = m + residual;  residual_out = bf16(r');
 *   out = bf16(bf16(r') * rsqrt(mean(bf16(r')^2) + eps) * gain)
 *   x bf16 [M, H] or NULL; residual, gain bf16; rows fp32 [M*k, H] or NULL;
 *   route_w fp32 [M, k] (needed with rows); shared fp32 [M, H] or NULL;
 *   out, residual_out bf16 [M, H].  H % 128 == 0, H <= 16384.
 */
int rmsnorm_residual(const void *x, const void *residual, const void *gain, int M, int H,
                     float eps, const float *rows, const float *route_w, int k,
                     const float *shared, void *out, void *residual_out, void *stream);

/* The MTP layer's input projection ([draft page] vllm.models.glm5next.nvidia
 * .specialized_decode.runtime.draft, SpecializedDraft.run: the input tokens'
 * embeddings and the previous hidden state, each RMS-normalised with its own
 * gain, concatenated, then eh_proj):
 *   A[t] = [ bf16(e * rsqrt(mean(e^2) + eps) * enorm) | bf16(h * rsqrt(mean(h^2) + eps) * hnorm) ],
 *          e = embed[input_ids[t]], h = hidden[t]   (the embedding half first);
 *   out = A . eh_proj_w^T   (split-K BF16 GEMM, fp32 sums rounded once to bf16).
 *
 *   input_ids   int32 [M] device; ids outside [0, vocab) give a zero embedding
 *               half and MOE_ERR_INVALID_ARG in the workspace status word
 *               (moe_device_status), never a read outside the table
 *   embed       bf16 [vocab, H];  hidden bf16 [M, H];  enorm, hnorm bf16 [H]
 *   eh_proj_w   bf16 [H, 2H] row-major;  out bf16 [M, H]
 *   workspace   mtp_eh_front_workspace_size(M, H) bytes, zeroed once by
 *               moe_workspace_init; holds A (readable by the caller after the
 *               call, at byte offset 256, bf16 [M, 2H]) and the split-K sums
 * Limits: 1 <= M <= 256, H % 128 == 0, H <= 16384, vocab >= 1; 16-byte aligned
 * pointers.  Argument errors return before anything is enqueued.  Calls that
 * share a workspace must be stream-ordered.
 * Two kernels: the norm kernel, then the projection, launched with
 * programmatic dependent launch so that it prefetches its first weight tiles
 * into L2 while the norm kernel runs (eh_proj_w must not be written by the
 * kernel enqueued just before the call). */
int mtp_eh_front_workspace_size(int M, int H, size_t *bytes);
int mtp_eh_front(const int32_t *input_ids, const void *embed, int vocab, const void *hidden,
                 const void *enorm, const void *hnorm, float eps, const void *eh_proj_w, int M, int H,
                 void *out, void *ws, size_t ws_bytes, void *stream);

/*
 * ---------------------------------------------------------------------------
 * The attention sublayer of a decode step: FP8 block-scaled projections, an FP8
 * paged key/value cache, and attention of the step's tokens over it.  No
 * counterpart on the source pages, whose executors leave attention to the
 * stock forward; the weight and activation formats are those of the expert
 * layers above.
 *
 * Workspaces.  Each call takes a workspace of its *_workspace_size, zeroed once
 * by moe_workspace_init.  It starts with the status word (moe_device_status)
 * and the counters of split work; every call leaves the counters at zero, so
 * one workspace of the largest size may serve all of these calls in stream
 * order.  After a call returned an error, or moe_device_status reported
 * MOE_ERR_DEVICE_TIMEOUT, it has to be zeroed again.
 * ---------------------------------------------------------------------------
 */

/*
 * Activation quantisation: per row and per group of 128 columns (the last may
 * be shorter), s = amax / 448 in fp32 (rounded up to a power of two when e8m0;
 * 1 for an all-zero group) and codes = E4M3(x / s), the quotient in fp32,
 * rounded to nearest even and saturating.
 *   x       bf16 [M, K], rows x_stride elements apart (x_stride >= K, % 8 == 0)
 *   codes   fp8 [M, K]
 *   scales  fp32 [ceil(K / 128), M4], M4 = M rounded up to a multiple of 4
 *           (k-blocks first: the product reads a block's scales as one run;
 *           columns from M on are not written)
 * K % 16 == 0, K <= 131072, M <= 2^20; x, codes and scales 16-byte aligned.  M == 0 is
 * a no-op.  One kernel.
 */
int fp8_quant_rows(const void *x, long long x_stride, int M, int K, int e8m0, uint8_t *codes, float *scales,
                   void *stream);

/*
 * out[m, n] = sum_kb scales[kb, m] * w_s[n / 128, kb] *
 *             sum_{k in block kb} codes[m, k] * w[n, k]      (fp32 sums)
 *   codes, scales  as fp8_quant_rows writes them
 *   w     fp8 [N, K];  w_s fp32 [ceil(N / 128), ceil(K / 128)]
 *   out   bf16 [M, N], rounded once (out_fp32 == 0), or fp32 [M, N]
 * K % 16 == 0, K <= 131072, any N <= 2^20, M <= 2^20; codes, scales, w, out and the
 * workspace 16-byte aligned.  M == 0 is a no-op.  One kernel; results do not
 * depend on the order in which CTAs finish.
 */
int fp8_block_gemm_workspace_size(int M, int N, int K, size_t *bytes);
int fp8_block_gemm(const uint8_t *codes, const float *scales, const uint8_t *w, const float *w_s, int M, int N, int K,
                   void *out, int out_fp32, void *ws, size_t ws_bytes, void *stream);

/*
 * The linear layer out = x . w^T: fp8_quant_rows into the workspace, then
 * fp8_block_gemm, launched so that it streams its first weights while the
 * quantisation still runs; for a few tokens (up to 8, or 16 of a small layer)
 * one kernel, the product quantising x itself.  The results are those of the
 * two calls.  Arguments and limits as theirs.
 */
int fp8_linear_workspace_size(int M, int N, int K, size_t *bytes);
int fp8_linear(const void *x, long long x_stride, const uint8_t *w, const float *w_s, int M, int N, int K, int e8m0,
               void *out, int out_fp32, void *ws, size_t ws_bytes, void *stream);

/*
 * A paged key/value cache in FP8.  A block is a page of one key/value head:
 * page_size tokens whose codes share one fp32 scale (value = code * scale).
 *   k, v              fp8 [num_pages, kv_heads, page_size, head_dim]
 *   k_scale, v_scale  fp32 [num_pages, kv_heads], finite and at most 2^126 (as the
 *                     append writes them)
 * page_size 16, 32, 64 or 128; head_dim 64 or 128; kv_heads <= 1024; k and v
 * 16-byte aligned.  Nothing needs to be initialised: what a block held before
 * its first slot is written does not matter.
 *
 * The batch of a step, shared by the two calls below (device arrays):
 *   page_table  int32 [B, width]: page of each page_size tokens of a sequence;
 *               entries past a sequence's length are not read
 *   q_start     int32 [B + 1]: rows [q_start[b], q_start[b + 1]) of the step's
 *               `total` tokens are sequence b's newest ones (a sequence may
 *               have none)
 *   lens        int32 [B]: tokens of each sequence, the new ones included
 *   max_new     host bound of the new tokens of any sequence
 * Values that do not fit (a page outside [0, num_pages), rows outside
 * [0, total], a length above width * page_size) set the status word to
 * MOE_ERR_INVALID_ARG; nothing outside the arrays is read or written.
 * width * page_size <= 2^30, B <= 2^20, total <= 2^24.  B == 0 or total == 0 is a
 * no-op, whatever the arrays' pointers.  Rows that no sequence holds are left as
 * they are.
 */
typedef struct moe_kv_cache {
  uint8_t *k;
  uint8_t *v;
  float *k_scale;
  float *v_scale;
  int num_pages;
  int kv_heads;
  int page_size;
  int head_dim;
} moe_kv_cache;

/*
 * Write the new tokens' keys and values (bf16 [total, kv_heads, head_dim],
 * tokens k_stride / v_stride elements apart, multiples of 8, so slices of a
 * fused projection do; 16-byte aligned) at their positions lens[b] - n_b + i.
 * A block's scale is the power of two at or above amax / 448 over the tokens
 * written to it, at least 2^-126, and never shrinks while the block fills:
 * when it grows, the codes that the block holds are rewritten in the new scale
 * (exact except where a code becomes subnormal: nearest even).  A call that
 * writes a block's first slot starts its scale anew.  Infinities do not set
 * a scale (they saturate), NaN stays NaN.  A sequence with bad values is left
 * out; where only a page is out of range, that block is.  A page may belong to
 * two sequences only where neither writes it.  One kernel.
 */
int kv_cache_workspace_size(size_t *bytes);
int kv_cache_append(const moe_kv_cache *cache, const void *k, long long k_stride, const void *v, long long v_stride,
                    const int32_t *page_table, int width, const int32_t *q_start, const int32_t *lens, int B, int total,
                    int max_new, void *ws, size_t ws_bytes, void *stream);

/*
 * Attention of the step's tokens over the cache (their own keys and values
 * written before): for token i of sequence b, at position
 * pos = lens[b] - n_b + i, and query head h with kv head h / (heads / kv_heads):
 *   s_j = sm_scale * q . k_j;  if softcap > 0: s_j = softcap * tanh(s_j / softcap);
 *   if slopes: s_j += slopes[h] * (j - pos)
 *   over j <= pos, j < lens[b] and, if window > 0, j > pos - window:
 *   out = sum_j exp(s_j) v_j / sum_j exp(s_j);  lse = log sum_j exp(s_j).
 * A row that sees no token gives zeros and lse = -inf.  Tokens of a page
 * outside [0, num_pages) are masked.
 *   q      bf16 [total, heads, head_dim], tokens q_stride elements apart
 *          (% 8 == 0), 16-byte aligned; heads % kv_heads == 0, heads <= 4096,
 *          total * heads < 2^31,
 *          min(B, total) * kv_heads + total * heads / 8 <= 7 * 10^8
 *   out    bf16 [total, heads, head_dim];  lse fp32 [total, heads] or NULL
 *   slopes fp32 [heads] or NULL
 * Scores, statistics and sums are fp32 (a capped score is within 2^-22 of caps up
 * to 256, within 2^-20 of itself above); the weights are rounded to 11 bits for
 * their product with V.  V scales of one sequence and head may differ by up to
 * 2^29 before weights lose bits.  An infinity or a NaN in a row of q makes the
 * row NaN; a NaN in a token's k or v reaches the rows that see the token, and no
 * other.
 * One kernel; results do not depend on the order in which CTAs finish.
 */
int decode_attention_workspace_size(int heads, int kv_heads, int head_dim, int max_new, size_t *bytes);
int decode_attention(const moe_kv_cache *cache, const void *q, long long q_stride, int heads,
                     const int32_t *page_table, int width, const int32_t *q_start, const int32_t *lens, int B, int total,
                     int max_new, float sm_scale, float softcap, int window, const float *slopes, void *out, float *lse,
                     void *ws, size_t ws_bytes, void *stream);

/*
 * ---------------------------------------------------------------------------
 * A prompt's way through the attention sublayer: the layer boundary with FP8
 * output, pages of the cache given to the step's tokens and taken back, and
 * attention of whole prompts over themselves.  No counterpart on the source
 * pages; formats, batches and workspaces are those of the calls above.
 * ---------------------------------------------------------------------------
 */

/*
 * rmsnorm_residual whose output is what fp8_block_gemm reads:
 *   r' = x + residual (fp32; x NULL: the residual);  residual_out = bf16(r');
 *   y = residual_out * rsqrt(mean(residual_out^2) + eps) * gain   (fp32);
 *   codes, scales = the quantisation of fp8_quant_rows, of y unrounded (y / s to an
 *   fp32 step);
 *   out = bf16(y), where out is not NULL.
 *   x, residual   bf16 [M, H], rows x_stride / residual_stride elements apart
 *                 (>= H, % 8 == 0)
 *   gain          bf16 [H]
 *   residual_out  bf16 [M, H]; may be the residual itself where that is dense
 *   codes         fp8 [M, H];  scales fp32 [ceil(H / 128), M rounded up to a
 *                 multiple of 4] (columns from M on are not written)
 * H % 16 == 0, H <= 16384, M <= 2^20; every pointer 16-byte aligned; apart from
 * residual_out no output may overlap an input.  M == 0 is a no-op.  One kernel;
 * a row's result does not depend on the other rows, but for the last bits of
 * its mean on whether there are few or many (fp32 sums in another order).
 */
int rmsnorm_residual_fp8(const void *x, long long x_stride, const void *residual, long long residual_stride,
                         const void *gain, int M, int H, float eps, int e8m0, uint8_t *codes, float *scales, void *out,
                         void *residual_out, void *stream);

/*
 * Pages of the cache on the GPU.  The free pages are a stack: the first
 * free_state[0] entries of free_pages, the last of them on top.  Sequence b
 * holds lens[b] tokens in its first ceil(lens[b] / page_size) table entries.
 *
 * kv_pages_extend makes room for a step's new_tokens[b] >= 0 tokens of each
 * sequence and describes the step's rows:
 *   need_b = ceil((lens[b] + new_b) / page_size) - ceil(lens[b] / page_size);
 *   a sequence is served if it needs no page or the needs up to and with it, of
 *   all sequences before it, are at most free_state[0]; n_b = new_b if it is, else
 *   0 (its table, length and rows are then as if it had asked for nothing);
 *   the pages go from the top of the stack down to the served sequences in
 *   turn, to each sequence's table entries in turn;
 *   lens_out[b] = lens[b] + n_b;  q_start[b] = sum of n before b (B + 1 values);
 *   row q_start[b] + i:  positions = lens[b] + i, slots = page * page_size +
 *   position % page_size with the position's page; rows from q_start[B] to
 *   `rows`: -1;
 *   free_out[0] = pages left;  free_out[1] = pages that were asked for and not
 *   given (0: everyone was served).
 *
 * kv_pages_release takes back the pages of the sequences with done[b] != 0:
 * they are pushed sequence by sequence, entry by entry; lens_out[b] = 0 for
 * these and lens[b] for the others, free_out = {free_state[0] + pages, 0}.
 * Table entries stay as they are.  A page that several sequences hold may be
 * released by the last of them only.
 *
 *   page_table  int32 [B, width];  lens, lens_out, new_tokens int32 [B]; done one byte [B]
 *   free_pages  int32 [capacity];  free_state, free_out int32 [2]
 *   q_start     int32 [B + 1];  positions int32 [rows];  slots int64 [rows]
 *   workspace   kv_cache_workspace_size
 * lens_out may be lens, and free_out free_state (a step in place); no other
 * arrays may overlap.  page_size 16, 32, 64 or 128; width * page_size <= 2^30;
 * B <= 2^20; rows <= 2^24.  B == 0 only fills rows and the state.
 * Values that do not fit set the status word to MOE_ERR_INVALID_ARG: a sequence
 * with a negative length or more tokens than its table has room for is left as
 * it is, as is one whose rows (counted over all that is asked for) pass `rows`;
 * a page outside [0, num_pages) is handed on, with slots of -1; a state outside
 * [0, capacity] counts as an empty stack and is left as it is; pages that do not
 * fit on the stack are not released, none of the call's.  One kernel each.
 */
int kv_pages_extend(int32_t *page_table, int width, const int32_t *lens, const int32_t *new_tokens, int B,
                    const int32_t *free_pages, int capacity, const int32_t *free_state, int page_size, int num_pages,
                    int32_t *q_start, int32_t *lens_out, int32_t *free_out, int32_t *positions, int64_t *slots, int rows,
                    void *ws, size_t ws_bytes, void *stream);
int kv_pages_release(const int32_t *page_table, int width, const int32_t *lens, const uint8_t *done, int B,
                     int32_t *free_pages, int capacity, const int32_t *free_state, int page_size, int num_pages,
                     int32_t *lens_out, int32_t *free_out, void *ws, size_t ws_bytes, void *stream);

/*
 * Attention of whole prompts over themselves, from the projection's bf16 keys
 * and values (decode_attention serves tokens whose sequence holds more than the
 * step's).  Rows [q_start[b], q_start[b + 1]) of `total` are prompt b; for its
 * row i and query head h with kv head h / (heads / kv_heads):
 *   s_j = sm_scale * q_i . k_j;  if softcap > 0: s_j = softcap * tanh(s_j / softcap);
 *   if slopes: s_j += slopes[h] * (j - i)
 *   over the prompt's rows j <= i and, if window > 0, j > i - window:
 *   out = sum_j exp(s_j) v_j / sum_j exp(s_j);  lse = log sum_j exp(s_j).
 *   q     bf16 [total, heads, head_dim], k, v bf16 [total, kv_heads, head_dim],
 *         rows q_stride / k_stride / v_stride elements apart (% 8 == 0; slices of
 *         a fused projection do), 16-byte aligned
 *   out   bf16 [total, heads, head_dim], 16-byte aligned;  lse fp32 [total, heads] or NULL
 *   slopes fp32 [heads] or NULL
 * head_dim 64 or 128; heads % kv_heads == 0, heads <= 4096, kv_heads <= 1024;
 * B <= 2^20, total <= 2^24, total * heads < 2^31 - 1024.  B == 0 or total == 0 is a no-op.
 * Rows that no prompt holds are left as they are.  A prompt whose rows do not lie
 * in [0, total), or that starts before an earlier one ends, is left out and sets
 * the status word to MOE_ERR_INVALID_ARG.
 * Scores, statistics and sums are fp32 (a capped score is within 2^-20 of itself);
 * the weights are rounded to bf16 for their product with V, and are up to 2^8 before
 * the division by their sum: finite values of v above about 2^120 / n (n tokens seen)
 * may overflow.  A NaN in a row of q makes the row NaN, and so does an infinity
 * where softcap is 0 (with a cap its scores are plus or minus the cap, as the
 * formula says); a NaN in a row's k or v reaches the rows that see it, and no
 * other; what rows outside the prompts hold does not matter.
 * One kernel; results do not depend on the order in which CTAs finish, and a
 * row's, to the last bit, on no other head or row than those that it sees.
 *
 * prompt_attention_checked is the same, told how many tokens the sequences hold:
 * lens int32 [B], as kv_cache_append takes it (NULL: nothing is checked).  A
 * prompt with rows that are not all of its tokens (lens[b] is not q_start[b + 1]
 * - q_start[b]: one that goes on from what the cache holds, which only
 * decode_attention attends) is left out and sets the status word as well.
 */
int prompt_attention_workspace_size(size_t *bytes);
int prompt_attention(const void *q, long long q_stride, const void *k, long long k_stride, const void *v,
                     long long v_stride, int heads, int kv_heads, int head_dim, const int32_t *q_start, int B, int total,
                     float sm_scale, float softcap, int window, const float *slopes, void *out, float *lse, void *ws,
                     size_t ws_bytes, void *stream);
int prompt_attention_checked(const void *q, long long q_stride, const void *k, long long k_stride, const void *v,
                             long long v_stride, int heads, int kv_heads, int head_dim, const int32_t *q_start,
                             const int32_t *lens, int B, int total, float sm_scale, float softcap, int window,
                             const float *slopes, void *out, float *lse, void *ws, size_t ws_bytes, void *stream);

/* Expert kernels (moe_decode_layer_plan, moe_set_expert_path). */
enum moe_expert_path {
  MOE_PATH_AUTO = 0,      /* the library's choice by layer kind and token count */
  MOE_PATH_WARP_MMA = 1,  /* warp-level FP8 MMAs on 8/16/32-token passes       */
  MOE_PATH_TCGEN05 = 2    /* tcgen05 FP8 MMAs, tensor-memory accumulators,
                             passes of up to 64 tokens                          */
};

/* The expert kernel a moe_decode_layer call of M tokens runs (*path, never
 * MOE_PATH_AUTO for M > 0) and the number of kernels it launches
 * (*launches).  Host only. */
int moe_decode_layer_plan(const moe_layer_dims *dims, int M, int *path, int *launches);

/* Tuning and test hook: force the expert kernel of every later
 * moe_decode_layer call in the process (MOE_PATH_AUTO restores the library's
 * choice).  Process-wide; not meant to change while calls are being made
 * from other host threads. */
int moe_set_expert_path(int path);

/* Read and clear the device status word of a workspace: MOE_OK,
 * MOE_ERR_DEVICE_TIMEOUT when a bounded wait inside a kernel gave up, or
 * MOE_ERR_INVALID_ARG when a kernel met a token id, page or length out of range.  Synchronises `stream`; meant for tests and diagnostics. */
int moe_device_status(void *ws, void *stream);

/* Test hook: nonzero `fault` makes the next moe_decode_layer calls on this
 * workspace withhold one expert's ready signal, so that the waits on it run
 * out (about 0.2 s) and report MOE_ERR_DEVICE_TIMEOUT.  Nothing faults. */
int moe_debug_set_fault(void *ws, int fault, void *stream);

/* Text of a status code. */
const char *moe_status_str(int status);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DECODE_H */
