// C ABI of what a prompt meets on its way through the attention sublayer (declared in
// include/moe_decode.h): the residual's addition and RMSNorm with FP8 output, pages of
// the cache given and taken back, attention over packed prompts.  Argument checks and
// launches; host code only.
#include <algorithm>
#include <climits>
#include <cmath>

#include "../../include/moe_decode.h"
#include "kernels.h"
#include "op_workspace.h"

namespace moe {

namespace {

// No sequence is longer, so no window is wider (and its differences fit in 32 bits).
constexpr int kMaxLen = 1 << 30;

int check_rows(const void* p, long long stride, long long row) {
  if (!p || !al16(p) || stride < row || stride % 8) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int shift_of(int page_size) {
  return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : page_size == 128 ? 7 : -1;
}

int check_pages(const int32_t* page_table, int width, const int32_t* lens, int B, const int32_t* free_pages, int capacity,
                const int32_t* free_state, int page_size, int num_pages, const int32_t* lens_out, const int32_t* free_out,
                const void* ws, size_t ws_bytes) {
  if (B < 0 || width < 0 || capacity < 0 || num_pages < 1 || page_size < 1) return MOE_ERR_INVALID_ARG;
  if (shift_of(page_size) < 0) return MOE_ERR_UNSUPPORTED;
  if ((long long)width * page_size > kMaxLen || B > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (!free_state || !free_out || (capacity > 0 && !free_pages)) return MOE_ERR_INVALID_ARG;
  if (B > 0 && (width < 1 || !page_table || !lens || !lens_out)) return MOE_ERR_INVALID_ARG;
  if (!ws || !al16(ws)) return MOE_ERR_INVALID_ARG;
  return ws_bytes < kDataAt ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

int rmsnorm_residual_fp8(const void* x, long long x_stride, const void* residual, long long residual_stride,
                         const void* gain, int M, int H, float eps, int e8m0, uint8_t* codes, float* scales, void* out,
                         void* residual_out, void* stream) {
  if (M < 0 || H < 1 || !(eps >= 0.f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
  if (H % 16 || H > 16384 || M > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  int rc = check_rows(residual, residual_stride, H);
  if (rc != MOE_OK || (x && (rc = check_rows(x, x_stride, H)) != MOE_OK)) return rc;
  if (!gain || !codes || !scales || !residual_out) return MOE_ERR_INVALID_ARG;
  if (!al16(gain) || !al16(codes) || !al16(scales) || !al16(residual_out) || (out && !al16(out)))
    return MOE_ERR_INVALID_ARG;
  if (residual_out == residual && M > 1 && residual_stride != H) return MOE_ERR_INVALID_ARG;  // (rows would meet)
  int sms = 0;
  if ((rc = current_device_sms(&sms)) != MOE_OK) return rc;
  NormFp8Args a;
  a.x = x; a.residual = residual; a.gain = gain; a.ldx = x_stride; a.ldr = residual_stride;
  a.residual_out = residual_out; a.out = out; a.codes = codes; a.scales = scales;
  a.M = M; a.H = H; a.mp = linear_scale_stride(M); a.e8m0 = e8m0 ? 1 : 0; a.eps = eps;
  return launch_rmsnorm_fp8(a, sms, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int kv_pages_extend(int32_t* page_table, int width, const int32_t* lens, const int32_t* new_tokens, int B,
                    const int32_t* free_pages, int capacity, const int32_t* free_state, int page_size, int num_pages,
                    int32_t* q_start, int32_t* lens_out, int32_t* free_out, int32_t* positions, int64_t* slots, int rows,
                    void* ws, size_t ws_bytes, void* stream) {
  int rc = check_pages(page_table, width, lens, B, free_pages, capacity, free_state, page_size, num_pages, lens_out,
                       free_out, ws, ws_bytes);
  if (rc != MOE_OK) return rc;
  if (rows < 0 || (B > 0 && !new_tokens) || !q_start || (rows > 0 && (!positions || !slots))) return MOE_ERR_INVALID_ARG;
  if (rows > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  int sms = 0;
  if ((rc = current_device_sms(&sms)) != MOE_OK) return rc;
  PagesArgs a{};
  a.page_table = page_table; a.lens = lens; a.fresh = new_tokens; a.free_pages = const_cast<int32_t*>(free_pages);
  a.free_state = free_state; a.q_start = q_start; a.lens_out = lens_out; a.free_out = free_out; a.positions = positions;
  a.slots = slots; a.width = width; a.shift = shift_of(page_size); a.num_pages = num_pages; a.capacity = capacity; a.B = B;
  a.rows = rows; a.status = Ws(ws).status; a.ticket = Ws(ws).tickets;
  return launch_kv_pages_extend(a, sms, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int kv_pages_release(const int32_t* page_table, int width, const int32_t* lens, const uint8_t* done, int B,
                     int32_t* free_pages, int capacity, const int32_t* free_state, int page_size, int num_pages,
                     int32_t* lens_out, int32_t* free_out, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_pages(page_table, width, lens, B, free_pages, capacity, free_state, page_size, num_pages, lens_out,
                       free_out, ws, ws_bytes);
  if (rc != MOE_OK) return rc;
  if (B > 0 && !done) return MOE_ERR_INVALID_ARG;
  int sms = 0;
  if ((rc = current_device_sms(&sms)) != MOE_OK) return rc;
  PagesArgs a{};
  a.page_table = const_cast<int32_t*>(page_table); a.lens = lens; a.done = done; a.free_pages = free_pages;
  a.free_state = free_state; a.lens_out = lens_out; a.free_out = free_out; a.width = width; a.shift = shift_of(page_size);
  a.num_pages = num_pages; a.capacity = capacity; a.B = B; a.status = Ws(ws).status;
  a.ticket = Ws(ws).tickets;
  return launch_kv_pages_release(a, sms, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int prompt_attention_workspace_size(size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = kDataAt;
  return MOE_OK;
}

int prompt_attention_checked(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                             long long v_stride, int heads, int kv_heads, int head_dim, const int32_t* q_start,
                             const int32_t* lens, int B, int total, float sm_scale, float softcap, int window,
                             const float* slopes, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (B < 0 || total < 0 || heads < 1 || kv_heads < 1 || head_dim < 1) return MOE_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return MOE_ERR_UNSUPPORTED;
  if (heads % kv_heads || heads > 4096 || kv_heads > 1024) return MOE_ERR_UNSUPPORTED;
  if (B > (1 << 20) || total > (1 << 24) || (long long)total * heads > INT_MAX - 1024) return MOE_ERR_UNSUPPORTED;
  if (!std::isfinite(sm_scale) || !std::isfinite(softcap) || softcap < 0.f || window < 0) return MOE_ERR_INVALID_ARG;
  if (B == 0 || total == 0) return MOE_OK;
  int rc;
  if ((rc = check_rows(q, q_stride, (long long)heads * head_dim)) != MOE_OK ||
      (rc = check_rows(k, k_stride, (long long)kv_heads * head_dim)) != MOE_OK ||
      (rc = check_rows(v, v_stride, (long long)kv_heads * head_dim)) != MOE_OK)
    return rc;
  if (!q_start || !out || !ws || !al16(out) || !al16(ws)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < kDataAt) return MOE_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  if ((rc = current_device_sms(&sms)) != MOE_OK) return rc;
  const Ws l(ws);
  PromptArgs a;
  a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.q_start = q_start; a.lens = lens; a.slopes = slopes; a.out = out; a.lse = lse;
  a.kv_heads = kv_heads; a.G = heads / kv_heads; a.D = head_dim; a.B = B; a.total = total;
  a.window = std::min(window, kMaxLen); a.sm_scale = sm_scale; a.softcap = softcap;
  a.status = l.status; a.tickets = l.tickets;
  return launch_prompt_attention(a, sms, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int prompt_attention(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                     long long v_stride, int heads, int kv_heads, int head_dim, const int32_t* q_start, int B, int total,
                     float sm_scale, float softcap, int window, const float* slopes, void* out, float* lse, void* ws,
                     size_t ws_bytes, void* stream) {
  return prompt_attention_checked(q, q_stride, k, k_stride, v, v_stride, heads, kv_heads, head_dim, q_start, nullptr, B,
                                  total, sm_scale, softcap, window, slopes, out, lse, ws, ws_bytes, stream);
}

}  // extern "C"
