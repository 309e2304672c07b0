// Internal launch interfaces between the C ABI (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "per_device.h"

namespace moe {

constexpr int kBlock = 128;  // weight scale block side / activation group length

// Header words at the start of a moe_decode_layer workspace (int32 each).
enum HdrWord {
  kHdrStatus = 0,        // 0 or MOE_ERR_DEVICE_TIMEOUT (sticky until read)
  kHdrFault = 1,         // test hook: withhold the first slot's ready signal
  kHdrRouterTicket = 2,  // router CTAs whose logits are complete
  kHdrQueue = 3,         // expert-kernel work queue head
  kHdrActive = 4,        // number of routed experts with at least one route
  kHdrDoneA = 5,         // w13 items finished (h stored and, when due, its group quantised)
  kHdrXReady = 6,        // router CTAs that have quantised their share of x (and, CTA 0, reset
                         // the expert kernel's counters); the expert kernel's last CTA clears it
  kHdrExit = 7,          // expert-kernel CTAs finished
  kHdrRouterFin = 8,     // router CTAs that have routed their share of the tokens
  kHdrWords = 64
};
constexpr int kMaxRouterTickets = 1024;
constexpr int kMaxMk = 4096;       // M * top_k per call
constexpr int kMaxTokens = 4096;   // M per call (the bound for a dense layer, whose top_k is 0)
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 16;

// Stream-K split of a skinny GEMM Y[M, N] = A[M, K] . W[N, K]^T over G CTAs.
// Work cells are (token chunk, 64-row tile, 128-column k-block), k fastest;
// CTA c owns cells [c*T/G, (c+1)*T/G).
// With dyn_tiles > 0 the last dyn_tiles (chunk, tile)s are left out of the
// static split: they are cut into units of dyn_unit k-blocks (dyn_nu a tile,
// fixed boundaries) that the CTAs take from a counter once their static share
// is done, so that the CTAs that stream faster take the tail.
struct GemvPlan {
  int M, N, K;
  int chunk_tokens;  // 8, 16 or 32
  int n_chunks, n_tiles, nkb;
  long long total;   // statically split cells
  int G;             // CTAs
  int max_segs;      // most static runs that cover one (chunk, tile)
  int dyn_tiles = 0, dyn_unit = 0, dyn_nu = 0;
};
void plan_gemv(GemvPlan& p, int M, int N, int K, int G, int dyn_tiles = 0);
// (chunk, tile)s of the dynamic tail of an automatic split-K plan over n_ct
// of them, and its unit length in k-blocks
inline long long splitk_dyn_tiles(long long n_ct) { return n_ct >= 32 ? n_ct / 8 : 0; }
constexpr int kDynUnit = 4;
constexpr int kDynMinRun = 64;  // static cells a CTA streams at least for the tail to be used
// resident CTAs per SM of the split-K (router == false) or router kernel on
// the current device (cached per device)
int gemv_blocks_per_sm(int chunk_tokens, bool router);
size_t gemv_partials_bytes(const GemvPlan& p);
// token chunk of a skinny GEMM of M tokens: 8, 16 or 32 columns per CTA pass
inline int gemv_chunk_tokens(int M) { return M <= 8 ? 8 : (M <= 16 ? 16 : 32); }

// SM count of the current device (cached per device): MOE_OK or MOE_ERR_CUDA.
int current_device_sms(int* sms);
// The plan of one split-K projection, shared by every entry point that runs
// it.  split_k == 0: stream-K over all SMs (every CTA streams an equal share
// of W); split_k = S > 0: every (token chunk, 64-row tile) is cut into exactly
// S K-segments, one CTA each.  Returns MOE_OK, MOE_ERR_INVALID_ARG or
// MOE_ERR_UNSUPPORTED (shape or split out of range) or MOE_ERR_CUDA.
int plan_splitk(GemvPlan& p, int M, int N, int K, int split_k);
// Bytes of the plan's counters (one per (chunk, tile), then the dynamic
// tail's unit counter and exit counter; rounded up to 256) and of its partial
// sums (0 when no tile is split).
size_t splitk_ticket_bytes(const GemvPlan& p);
size_t splitk_partial_bytes(const GemvPlan& p);

struct SplitKArgs {
  const void* A;
  const void* W;
  void* C;
  int c_fp32;
  float alpha;
  float* partials;
  unsigned* tickets;
  // programmatic dependent launch: the kernel starts while the preceding one
  // (which writes A, never W) ends, prefetches its first weights into L2 and
  // waits for that kernel before it reads A
  bool pdl = false;
};
cudaError_t launch_splitk(const GemvPlan& p, const SplitKArgs& a, cudaStream_t s);

struct RouterArgs {
  const void* x;       // bf16 [M, H]
  const void* W;       // bf16 [E, H]
  const float* bias;   // [E] or null
  int E, k, e8m0;
  float scaling;
  float* partials;
  unsigned* tickets;
  float* logits;       // [M, E]
  uint8_t* xq;         // [M, H]
  float* xs;           // [M, H/128]
  int* hdr;
  int* ids;            // [M*k]
  float* tw;           // [M*k]
  int* sorted;         // [M*k]
  int* off;            // [E+1]
  int* act;            // [E]
  int* gcount;         // expert-kernel counters reset here
  int n_gcount;
  int* ready;
  int n_ready;
  int32_t* user_ids;
  float* user_w;
  int32_t* user_sorted;
  int32_t* user_off;
};
cudaError_t launch_router(const GemvPlan& p, const RouterArgs& a, cudaStream_t s);

struct ExpertArgs {
  int H, I, Is, E, k, M, Mk, Imax, gI;
  int hsS;  // row stride (floats) of the h scales: gI rounded up to 32 (one 128-byte line per row)
  float limit;
  int e8m0;
  const uint8_t* w13; const float* w13_s;
  const uint8_t* w2;  const float* w2_s;
  const uint8_t* sw13; const float* sw13_s;
  const uint8_t* sw2;  const float* sw2_s;
  const uint8_t* xq; const float* xs;
  const int* sorted; const int* off; const int* act;
  int* hdr; int* gcount; int* ready;
  float* h; uint8_t* hq; float* hs;
  float* rows; float* shared_out;
  int router_ctas;  // CTAs of the router launch that precedes this kernel
  int bq;           // w2 item size in 32-row quarters of a 128-row block: 4, 2 or 1
};
// An expert-kernel launch prepared on the host (tensor maps encoded, the
// pass width and ring depth chosen, the shared-memory limit set) before the
// router is enqueued, so that no host work falls between the router's and the
// expert kernel's launches.
// Extra arguments of the tensor-core (tcgen05) form of the expert kernel:
//   xg       the routed tokens' x codes in route order (launch_gather_rows)
//   sh_segs  K segments of the shared slot's w2 items (tc_shared_segments),
//            whose partial rows follow one another in shared_out
//   a_segs   K segments of the shared slot's w13 items (tc_w13_segments),
//            partial [g; u] rows in gu_part (tc_w13_partial_bytes), counted
//            per group in pcount (zeroed by the router with the counters)
struct TcExtra {
  const uint8_t* xg;
  int sh_segs;
  int a_segs;
  float* gu_part;
  int* pcount;
};
struct ExpertsLaunch {
  ExpertArgs a;
  CUtensorMap maps[7];
  bool tc;               // the tcgen05 kernel (else the warp-MMA kernel)
  int tt;                // warp-MMA kernel: 8-token columns per pass
  int nst;               // warp-MMA kernel: ring stages
  size_t smem;           // dynamic shared memory
  TcExtra tcx;           // tcgen05 kernel
};
cudaError_t prepare_experts(const ExpertArgs& a, ExpertsLaunch& L);
cudaError_t prepare_experts_tc(const ExpertArgs& a, const TcExtra& x, ExpertsLaunch& L);
cudaError_t launch_experts(const ExpertsLaunch& L, int num_sms, cudaStream_t s);
cudaError_t launch_gather_rows(const uint8_t* xq, const int* sorted, int k, int Mk, int H, uint8_t* xg, int num_sms,
                               cudaStream_t s);
constexpr int kMaxSharedSegs = 16;  // K segments of a dense layer's w2 items at most
int tc_shared_segments(int E, int H, int Is, int M, int num_sms);
int tc_w13_segments(int E, int H, int Is, int M);
size_t tc_w13_partial_bytes(int E, int Is);

struct NormArgs {
  const void* x; const void* residual; const void* gain;
  const float* rows; const float* route_w; const float* shared;
  void* out; void* residual_out;
  int M, H, k;
  int shared_parts;  // partial rows [parts][M][H] in `shared`, added in order (>= 1)
  float* m_out;      // non-null: write m (fp32 [M, H]) there and stop (no residual, no norm)
  float eps;
  int early;  // residual and gain come from before the preceding kernels (the layer call)
};
cudaError_t launch_rmsnorm(const NormArgs& a, cudaStream_t s);

struct EhNormArgs {
  const int32_t* ids; const void* embed; int vocab;
  const void* hidden; const void* enorm; const void* hnorm;
  float eps;
  void* out;  // bf16 [M, 2H]
  int M, H;
  int* status;
};
cudaError_t launch_eh_norm(const EhNormArgs& a, cudaStream_t s);

// FP8 block-scaled linear layer (fp8_linear.cu).
struct QuantArgs {
  const void* x;  // bf16 [M, K], row stride ldx elements
  long long ldx;
  int M, K, nkb, e8m0;
  uint8_t* codes;  // [M, K]
  float* scales;   // [nkb][mp]
  int mp;          // linear_scale_stride(M)
};
// tokens of a row of activation scales: M rounded up so that runs start on 16 bytes
inline int linear_scale_stride(int M) { return (M + 3) & ~3; }
cudaError_t launch_quant_rows(const QuantArgs& a, int sms, cudaStream_t s);

constexpr int kLinMaxCtas = 160;  // CTAs of the product at most (one per SM)
struct LinPlan {
  int M, N, K, nkb;
  bool tok_rows;      // the tokens are the MMA's rows (else its columns)
  int nt;             // the kernel's columns: 16, 32, 64, 128 (tokens) or 256 (weight rows)
  int chunk;          // tokens of a CTA's token tile
  int n_tt, n_wt;     // token tiles (tok_rows: of both CTAs of a pair), weight tiles
  int G;              // CTAs (tok_rows: pairs of CTAs)
  int waves;          // whole (row tile, column tile) pairs of each CTA
  int rest;           // pairs after those,
  int pieces;         // each cut along K into so many
};
// Whether the product quantises x itself: it saves the quantisation's launch, but every
// CTA quantises the tokens of all its cells, eight at a time.  Up to 8 tokens it always
// pays, up to 16 where a CTA has few cells.  Measured, us itself / by a kernel of its
// own: 7168 -> 9216 (28 cells a CTA) 1 token 14.6 / 16.1, 8 16.2 / 16.6, 16 18.8 / 17.2;
// 2048 -> 1536 (4 cells a CTA) 1 token 5.2 / 6.1, 8 5.5 / 6.5, 16 6.5 / 6.9.
inline bool linear_fused(const LinPlan& p) {
  const int cells = p.waves * p.nkb + (p.rest > 0 ? (p.nkb + p.pieces - 1) / p.pieces : 0);
  return p.M <= 8 || (p.M <= 16 && cells <= 8);
}
struct LinArgs {
  // the caller's: x (to be quantised: linear_fused) or codes and scales
  const void* x = nullptr;     // bf16 [M, K], row stride ldx elements
  long long ldx = 0;
  int e8m0 = 0;
  const float* xs = nullptr;   // [nkb][mp]
  const float* w_s = nullptr;  // [n_wblk][nkb]
  void* out = nullptr;
  int out_fp32 = 0;
  int* status = nullptr;
  int* tickets = nullptr;      // one a CTA, zero between calls
  float* partials = nullptr;   // [CTA][nt][128]
  bool after_quant = false;    // the kernel just enqueued is the launch_quant_rows that writes the
                               // codes and scales, and no other input
  // the plan's
  int mp, M, N, K, nkb, chunk, n_wt, n_wblk, G, waves, pieces;
  // each CTA's piece of the remaining pairs: weight tile, token tile, k-blocks
  // (none: k0 == k1), and the CTA with the pair's first piece
  struct Piece { uint16_t w, t, k0, k1, first; } piece[kLinMaxCtas];
  bool tok_rows;
};
void plan_linear(LinPlan& p, int M, int N, int K, int sms);
cudaError_t launch_linear(const LinPlan& p, LinArgs a, const uint8_t* xq, const uint8_t* w, cudaStream_t s);

// The FP8 paged cache: writing new tokens (kv_append.cu) and attention over it
// (attention.cu).  Caches [num_pages][kv_heads][page_size][head_dim] codes,
// scales [num_pages][kv_heads], page_table [B][width], q_start [B + 1], lens [B].
struct AppendArgs {
  const void* k; const void* v;  // bf16 [total][kv_heads][head_dim], token strides in elements
  long long k_stride, v_stride;
  uint8_t* k_cache; uint8_t* v_cache;
  float* k_scale; float* v_scale;
  const int32_t* page_table; const int32_t* q_start; const int32_t* lens;
  int num_pages, kv_heads, page_size, head_dim, width, B, total, max_new;
  int blocks;  // blocks a sequence's new tokens can touch
  int* status;
};
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t s);

constexpr int kAttMaxCtas = 160;  // CTAs of the attention kernel at most (one per SM)
// Items (a sequence's and kv head's groups of rows) of a call at most.
constexpr int kAttMaxItems = 700000000;
struct AttArgs {
  const void* q;  // bf16 [total][G * kv_heads][head_dim], token stride in elements
  long long q_stride;
  const uint8_t* k_cache; const uint8_t* v_cache;
  const float* k_scale; const float* v_scale;
  const int32_t* page_table; const int32_t* q_start; const int32_t* lens;
  const float* slopes;  // [G * kv_heads] or null
  void* out; float* lse;
  int num_pages, kv_heads, page_size, head_dim, width, B, total, max_new;
  int G;       // query heads per kv head
  int window;  // tokens a row sees at most, 0 = all
  float sm_scale, softcap;
  int* status;
  int* tickets;     // [kAttMaxCtas], zero between calls
  float* partials;  // attention_partial_bytes
};
int attention_row_tiles(int G, int max_new);
size_t attention_partial_bytes(int D, int G, int max_new);
cudaError_t launch_attention(const AttArgs& a, int sms, cudaStream_t s);

// Residual addition and RMSNorm with FP8 output (rmsnorm_fp8.cu).
struct NormFp8Args {
  const void* x;  // bf16 [M, H] or null, row strides in elements
  const void* residual;
  const void* gain;
  long long ldx, ldr;
  void* residual_out;  // bf16 [M, H]; may be the residual
  void* out;           // bf16 [M, H] or null
  uint8_t* codes;      // [M, H]
  float* scales;       // [groups][mp]
  int M, H, mp, e8m0;
  float eps;
};
cudaError_t launch_rmsnorm_fp8(const NormFp8Args& a, int sms, cudaStream_t s);

// Pages of the cache given to a step's tokens and taken back (kv_pages.cu).
struct PagesArgs {
  int32_t* page_table;       // [B][width]
  const int32_t* lens;       // [B]
  const int32_t* fresh;      // extend: new tokens [B]
  const uint8_t* done;       // release: [B]
  int32_t* free_pages;       // [capacity], read by extend, written by release
  const int32_t* free_state; // {pages on the stack, ...}
  int32_t* q_start;          // extend: [B + 1]
  int32_t* lens_out;         // [B]
  int32_t* free_out;         // {pages on the stack, pages that were missing}
  int32_t* positions;        // extend: [rows]
  int64_t* slots;            // extend: [rows]
  int width, shift, num_pages, capacity, B, rows;  // shift: log2 of the page's tokens
  int* status;
  int* ticket;  // zero between calls
};
cudaError_t launch_kv_pages_extend(const PagesArgs& a, int sms, cudaStream_t s);
cudaError_t launch_kv_pages_release(const PagesArgs& a, int sms, cudaStream_t s);

// Causal attention over packed prompts (prompt_attention.cu).
struct PromptArgs {
  const void* q;  // bf16 [total][G * kv_heads][D], token strides in elements
  const void* k;  // bf16 [total][kv_heads][D]
  const void* v;
  long long q_stride, k_stride, v_stride;
  const int32_t* q_start;  // [B + 1]
  const int32_t* lens;     // [B]: tokens of the sequences, all of them rows here; or null
  const float* slopes;     // [G * kv_heads] or null
  void* out;
  float* lse;
  int kv_heads, G, D, B, total;
  int window;  // tokens a row sees at most, 0 = all
  float sm_scale, softcap;
  int* status;
  int* tickets;
  // the launch's
  int rows;      // packed rows of a tile
  bool out32;    // out lies on a multiple of 32 bytes
  float cap_in;  // sm_scale / softcap
};
cudaError_t launch_prompt_attention(const PromptArgs& a, int sms, cudaStream_t s);

// Lets launches of `kernel` on the current device take `bytes` of dynamic shared memory.
template <class K>
cudaError_t allow_smem(OncePerDevice& once, K kernel, size_t bytes) {
  int dev = 0;
  if (const cudaError_t rc = cudaGetDevice(&dev); rc != cudaSuccess) return rc;
  return once(dev, [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes); });
}

// Launch configuration that lets a kernel start while its predecessor in the
// stream finishes (it waits with griddepcontrol.wait before using its results).
struct PdlLaunch {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  PdlLaunch(dim3 grid, dim3 block, size_t smem, cudaStream_t s) {
    cfg = cudaLaunchConfig_t{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

}  // namespace moe
