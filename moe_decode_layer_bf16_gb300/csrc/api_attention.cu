// C ABI of the attention sublayer's operators (declared in
// include/moe_decode.h): the FP8 block-scaled linear layer, the FP8 paged
// cache's writer, and attention over the cache.  Argument checks, workspace
// layout and launches; host code only.
#include <algorithm>
#include <climits>
#include <cmath>

#include "../../include/moe_decode.h"
#include "kernels.h"
#include "op_workspace.h"

namespace moe {

namespace {

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
// No sequence is longer, so no window is wider (and its differences fit in 32 bits).
constexpr int kMaxLen = 1 << 30;

int check_linear(int M, int N, int K) {
  if (M < 0 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (K % 16 || K > (1 << 17) || N > (1 << 20) || M > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Partial sums of any split this shape may get, whatever the SM count.
size_t linear_partial_bound(int M, int N, int K) {
  LinPlan p;
  plan_linear(p, std::max(M, 1), N, K, kLinMaxCtas);
  const long long cells = (long long)p.n_tt * p.n_wt * p.nkb;
  const long long ctas = std::min<long long>(kLinMaxCtas, p.tok_rows ? 2 * cells : cells);
  return (size_t)ctas * p.nt * kBlock * sizeof(float);
}

size_t codes_bytes(int M, int K) { return up256((size_t)M * K); }
size_t scales_bytes(int M, int K) { return up256((size_t)linear_scale_stride(M) * ((K + kBlock - 1) / kBlock) * sizeof(float)); }

int plan_here(LinPlan& p, int M, int N, int K) {
  int sms = 0;
  const int rc = current_device_sms(&sms);
  if (rc == MOE_OK) plan_linear(p, M, N, K, sms);
  return rc;
}

int gemm_launch(const LinPlan& p, LinArgs a, const uint8_t* codes, const uint8_t* w, const Ws& ws, uint8_t* partials,
                cudaStream_t s) {
  a.status = ws.status;
  a.tickets = ws.tickets;
  a.partials = reinterpret_cast<float*>(partials);
  return launch_linear(p, a, codes, w, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int check_x(const void* x, long long x_stride, int K) {
  if (!x || !al16(x)) return MOE_ERR_INVALID_ARG;
  if (x_stride < K || x_stride % 8) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int quant_launch(const void* x, long long x_stride, int M, int K, int e8m0, uint8_t* codes, float* scales,
                 cudaStream_t s) {
  int sms = 0;
  const int rc = current_device_sms(&sms);
  if (rc != MOE_OK) return rc;
  QuantArgs a;
  a.x = x; a.ldx = x_stride; a.M = M; a.K = K; a.nkb = (K + kBlock - 1) / kBlock; a.e8m0 = e8m0 ? 1 : 0;
  a.codes = codes; a.scales = scales; a.mp = linear_scale_stride(M);
  return launch_quant_rows(a, sms, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int check_cache_dims(int num_pages, int kv_heads, int page_size, int head_dim) {
  if (num_pages < 1 || kv_heads < 1 || page_size < 1 || head_dim < 1) return MOE_ERR_INVALID_ARG;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return MOE_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return MOE_ERR_UNSUPPORTED;
  if (kv_heads > 1024 || (long long)num_pages * kv_heads > INT_MAX) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_cache(const moe_kv_cache* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  const int rc = check_cache_dims(c->num_pages, c->kv_heads, c->page_size, c->head_dim);
  if (rc != MOE_OK) return rc;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !al16(c->k) || !al16(c->v)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int check_batch(const moe_kv_cache* c, const int32_t* page_table, int width, const int32_t* q_start,
                const int32_t* lens, int B, int total, int max_new) {
  if (B < 0 || total < 0 || width < 0 || max_new < 1) return MOE_ERR_INVALID_ARG;
  if ((long long)width * c->page_size > kMaxLen || B > (1 << 20) || total > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (B == 0 || total == 0) return MOE_OK;  // a no-op: nothing of the batch is read (arrays of no elements may be null)
  if (width < 1 || !page_table || !q_start || !lens) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int check_rows(const void* p, long long stride, long long row) {
  if (!p || !al16(p) || stride < row || stride % 8) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

int fp8_quant_rows(const void* x, long long x_stride, int M, int K, int e8m0, uint8_t* codes, float* scales,
                   void* stream) {
  int rc = check_linear(M, 1, K);
  if (rc != MOE_OK) return rc;
  if (M == 0) return MOE_OK;
  if ((rc = check_x(x, x_stride, K)) != MOE_OK) return rc;
  if (!codes || !scales || !al16(codes) || !al16(scales)) return MOE_ERR_INVALID_ARG;
  return quant_launch(x, x_stride, M, K, e8m0, codes, scales, (cudaStream_t)stream);
}

int fp8_block_gemm_workspace_size(int M, int N, int K, size_t* bytes) {
  const int rc = check_linear(M, N, K);
  if (rc != MOE_OK) return rc;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = kDataAt + linear_partial_bound(M, N, K);
  return MOE_OK;
}

int fp8_block_gemm(const uint8_t* codes, const float* scales, const uint8_t* w, const float* w_s, int M, int N, int K,
                   void* out, int out_fp32, void* ws, size_t ws_bytes, void* stream) {
  size_t need = 0;
  const int rc = fp8_block_gemm_workspace_size(M, N, K, &need);
  if (rc != MOE_OK) return rc;
  if (M == 0) return MOE_OK;
  if (!codes || !scales || !w || !w_s || !out || !ws) return MOE_ERR_INVALID_ARG;
  if (!al16(codes) || !al16(scales) || !al16(w) || !al16(out) || !al16(ws)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const Ws l(ws);
  LinPlan p;
  if (const int bad = plan_here(p, M, N, K); bad != MOE_OK) return bad;
  LinArgs a;
  a.xs = scales; a.w_s = w_s; a.out = out; a.out_fp32 = out_fp32 ? 1 : 0;
  return gemm_launch(p, a, codes, w, l, l.data, (cudaStream_t)stream);
}

int fp8_linear_workspace_size(int M, int N, int K, size_t* bytes) {
  const int rc = check_linear(M, N, K);
  if (rc != MOE_OK) return rc;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = kDataAt + codes_bytes(M, K) + scales_bytes(M, K) + linear_partial_bound(M, N, K);
  return MOE_OK;
}

int fp8_linear(const void* x, long long x_stride, const uint8_t* w, const float* w_s, int M, int N, int K, int e8m0,
               void* out, int out_fp32, void* ws, size_t ws_bytes, void* stream) {
  size_t need = 0;
  int rc = fp8_linear_workspace_size(M, N, K, &need);
  if (rc != MOE_OK) return rc;
  if (M == 0) return MOE_OK;
  if ((rc = check_x(x, x_stride, K)) != MOE_OK) return rc;
  if (!w || !w_s || !out || !ws || !al16(w) || !al16(out) || !al16(ws)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const Ws l(ws);
  uint8_t* codes = l.data;
  float* scales = reinterpret_cast<float*>(codes + codes_bytes(M, K));
  uint8_t* partials = codes + codes_bytes(M, K) + scales_bytes(M, K);
  LinArgs a;
  a.w_s = w_s; a.out = out; a.out_fp32 = out_fp32 ? 1 : 0;
  LinPlan p;
  if ((rc = plan_here(p, M, N, K)) != MOE_OK) return rc;
  if (linear_fused(p)) {
    a.x = x; a.ldx = x_stride; a.e8m0 = e8m0 ? 1 : 0;
    return gemm_launch(p, a, nullptr, w, l, partials, (cudaStream_t)stream);
  }
  if ((rc = quant_launch(x, x_stride, M, K, e8m0, codes, scales, (cudaStream_t)stream)) != MOE_OK) return rc;
  // the product streams its first weights while the quantisation still runs
  a.xs = scales;
  a.after_quant = true;
  return gemm_launch(p, a, codes, w, l, partials, (cudaStream_t)stream);
}

int kv_cache_workspace_size(size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = kDataAt;
  return MOE_OK;
}

int kv_cache_append(const moe_kv_cache* cache, const void* k, long long k_stride, const void* v, long long v_stride,
                    const int32_t* page_table, int width, const int32_t* q_start, const int32_t* lens, int B, int total,
                    int max_new, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_cache(cache);
  if (rc != MOE_OK) return rc;
  if ((rc = check_batch(cache, page_table, width, q_start, lens, B, total, max_new)) != MOE_OK) return rc;
  if (B == 0 || total == 0) return MOE_OK;
  const long long row = (long long)cache->kv_heads * cache->head_dim;
  if ((rc = check_rows(k, k_stride, row)) != MOE_OK || (rc = check_rows(v, v_stride, row)) != MOE_OK) return rc;
  if (!ws || !al16(ws)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < kDataAt) return MOE_ERR_WORKSPACE_TOO_SMALL;
  AppendArgs a;
  a.k = k; a.v = v; a.k_stride = k_stride; a.v_stride = v_stride;
  a.k_cache = cache->k; a.v_cache = cache->v; a.k_scale = cache->k_scale; a.v_scale = cache->v_scale;
  a.page_table = page_table; a.q_start = q_start; a.lens = lens;
  a.num_pages = cache->num_pages; a.kv_heads = cache->kv_heads; a.page_size = cache->page_size;
  a.head_dim = cache->head_dim; a.width = width; a.B = B; a.total = total; a.max_new = max_new;
  const long long n = std::min(max_new, total);
  const long long blocks = (n + cache->page_size - 2) / cache->page_size + 1;
  if (blocks * B > INT_MAX) return MOE_ERR_UNSUPPORTED;
  a.blocks = (int)blocks;
  a.status = Ws(ws).status;
  return launch_kv_append(a, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int decode_attention_workspace_size(int heads, int kv_heads, int head_dim, int max_new, size_t* bytes) {
  if (!bytes || heads < 1 || max_new < 1) return MOE_ERR_INVALID_ARG;
  const int rc = check_cache_dims(1, kv_heads, 16, head_dim);
  if (rc != MOE_OK) return rc;
  if (heads % kv_heads || heads > 4096) return MOE_ERR_UNSUPPORTED;
  *bytes = kDataAt + attention_partial_bytes(head_dim, heads / kv_heads, max_new);
  return MOE_OK;
}

int decode_attention(const moe_kv_cache* cache, const void* q, long long q_stride, int heads,
                     const int32_t* page_table, int width, const int32_t* q_start, const int32_t* lens, int B, int total,
                     int max_new, float sm_scale, float softcap, int window, const float* slopes, void* out, float* lse,
                     void* ws, size_t ws_bytes, void* stream) {
  int rc = check_cache(cache);
  if (rc != MOE_OK) return rc;
  if ((rc = check_batch(cache, page_table, width, q_start, lens, B, total, max_new)) != MOE_OK) return rc;
  size_t need = 0;
  if ((rc = decode_attention_workspace_size(heads, cache->kv_heads, cache->head_dim, max_new, &need)) != MOE_OK) return rc;
  if (!std::isfinite(sm_scale) || !std::isfinite(softcap) || softcap < 0.f || window < 0) return MOE_ERR_INVALID_ARG;
  if ((long long)total * heads > INT_MAX) return MOE_ERR_UNSUPPORTED;
  if ((long long)std::min(B, total) * cache->kv_heads + (long long)total * heads / 8 > kAttMaxItems)
    return MOE_ERR_UNSUPPORTED;
  if (B == 0 || total == 0) return MOE_OK;
  if ((rc = check_rows(q, q_stride, (long long)heads * cache->head_dim)) != MOE_OK) return rc;
  if (!out || !ws || !al16(out) || !al16(ws)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  if ((rc = current_device_sms(&sms)) != MOE_OK) return rc;
  const Ws l(ws);
  AttArgs a;
  a.q = q; a.q_stride = q_stride;
  a.k_cache = cache->k; a.v_cache = cache->v; a.k_scale = cache->k_scale; a.v_scale = cache->v_scale;
  a.page_table = page_table; a.q_start = q_start; a.lens = lens; a.slopes = slopes; a.out = out; a.lse = lse;
  a.num_pages = cache->num_pages; a.kv_heads = cache->kv_heads; a.page_size = cache->page_size;
  a.head_dim = cache->head_dim; a.width = width; a.B = B; a.total = total; a.max_new = max_new;
  a.G = heads / cache->kv_heads; a.window = std::min(window, kMaxLen); a.sm_scale = sm_scale; a.softcap = softcap;
  a.status = l.status; a.tickets = l.tickets; a.partials = reinterpret_cast<float*>(l.data);
  return launch_attention(a, sms, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
