// Causal attention of packed prompts over themselves, grouped heads, bf16:
//   s_j = sm_scale q . k_j (capped, biased by distance), j <= i, j > i - window;
//   out = sum_j exp(s_j) v_j / sum_j exp(s_j);  lse = log sum_j exp(s_j).
//
// A warp for each row and head, one pass over its keys with the running maximum and sum.
#include "common.cuh"
#include "kernels.h"
#include "step_rows.h"
#include "../../include/moe_decode.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

template <int D>
__global__ void __launch_bounds__(kThreads) prompt_attention_kernel(PromptArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y, heads = a.G * a.kv_heads, hk = h / a.G;
  grid_dep_launch();
  grid_dep_wait();
  const int row = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= a.total) return;
  int start = -1;
  for (int b = 0; b < a.B; ++b) {
    const int s = a.q_start[b], e = a.q_start[b + 1];
    if (!step_rows_ok(s, e, a.total)) {
      if (lane == 0) atomicExch(a.status, MOE_ERR_INVALID_ARG);
      continue;
    }
    if (s <= row && row < e) start = s;
  }
  if (start < 0) return;
  const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + row * a.q_stride + (size_t)h * D;
  float qf[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    qf[i] = __bfloat162float(q[lane + 32 * i]);
    acc[i] = 0.f;
  }
  const int first = a.window > 0 ? max(start, row - a.window + 1) : start;
  const float slope = a.slopes ? a.slopes[h] : 0.f;
  for (int j = first; j <= row; ++j) {
    const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(a.k) + j * a.k_stride + (size_t)hk * D;
    const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(a.v) + j * a.v_stride + (size_t)hk * D;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s += qf[i] * __bfloat162float(k[lane + 32 * i]);
    s = warp_sum(s) * a.sm_scale;
    if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
    if (a.slopes) s += slope * (float)(j - row);
    const float top = fmaxf(m, s), keep = expf(m - top), p = expf(s - top);
    m = top;
    l = l * keep + p;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = acc[i] * keep + p * __bfloat162float(v[lane + 32 * i]);
  }
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + ((size_t)row * heads + h) * D;
#pragma unroll
  for (int i = 0; i < E; ++i) out[lane + 32 * i] = __float2bfloat16(acc[i] / l);
  if (a.lse && lane == 0) a.lse[(size_t)row * heads + h] = m + logf(l);
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs& a, int sms, cudaStream_t s) {
  PdlLaunch L(dim3((a.total + kThreads / 32 - 1) / (kThreads / 32), a.G * a.kv_heads), dim3(kThreads), 0, s);
  if (a.D == 64) return cudaLaunchKernelEx(&L.cfg, prompt_attention_kernel<64>, a);
  return cudaLaunchKernelEx(&L.cfg, prompt_attention_kernel<128>, a);
}

}  // namespace moe
