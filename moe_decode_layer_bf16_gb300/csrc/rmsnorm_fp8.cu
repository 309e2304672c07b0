// Residual addition, RMSNorm and quantisation to E4M3 in one pass:
//   r' = bf16(x + residual);  y = r' * rsqrt(mean(r'^2) + eps) * gain;
//   s = amax of |y| over 128 columns / 448;  codes = E4M3(y / s).
// y is not rounded before it is quantised.
//
// One CTA a row, a thread for each V times 8 columns, which stay in registers from the
// one read to the write: the row's sum is a reduction over the CTA, a group's maximum
// one over 16 lanes.  Bound by bytes for many rows; for a few by latency.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

// 8 bf16 values as floats
MOE_DEV void unpack8(const uint4& v, float* f) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
MOE_DEV uint4 pack8(const float* f) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// (No read-only loads: this kernel starts while others may still write its inputs.)
template <int V, int T>
__global__ void __launch_bounds__(T) rmsnorm_fp8_kernel(NormFp8Args a) {
  __shared__ float s_sum[T / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const int t = blockIdx.x, nv = a.H / 8;  // 16-byte pieces of a row
  const uint4* res = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.residual) + t * a.ldr);
  const uint4* xx = a.x ? reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.x) + t * a.ldx) : nullptr;
  const uint4* gain = reinterpret_cast<const uint4*>(a.gain);
  grid_dep_launch();
  grid_dep_wait();
  uint4 r[V], g[V], xv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = tid + i * threads;
    r[i] = g[i] = xv[i] = make_uint4(0, 0, 0, 0);
    if (j < nv) {
      r[i] = res[j];
      if (xx) xv[i] = xx[j];
      g[i] = gain[j];
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float f[8];
    unpack8(r[i], f);
    if (xx) {
      float e[8];
      unpack8(xv[i], e);
#pragma unroll
      for (int c = 0; c < 8; ++c) f[c] = e[c] + f[c];
      r[i] = pack8(f);
      unpack8(r[i], f);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) ss += f[c] * f[c];
  }
  ss = warp_sum(ss);
  if (lane == 0) s_sum[warp] = ss;
  __syncthreads();
  ss = warp_sum(lane < threads / 32 ? s_sum[lane] : 0.f);
  const float inv = 1.f / sqrtf(ss / (float)a.H + a.eps);
  const size_t row = (size_t)t * nv;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = tid + i * threads;
    float f[8], w[8], amax = 0.f;
    unpack8(r[i], f);
    unpack8(g[i], w);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      f[c] = f[c] * inv * w[c];
      amax = fmaxf(amax, fabsf(f[c]));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (j >= nv) continue;
    reinterpret_cast<uint4*>(a.residual_out)[row + j] = r[i];
    if (a.out) reinterpret_cast<uint4*>(a.out)[row + j] = pack8(f);
    const float s = group_scale(amax, a.e8m0 != 0);
#pragma unroll
    for (int c = 0; c < 8; ++c) f[c] = __fdiv_rn(f[c], s);
    reinterpret_cast<uint2*>(a.codes)[row + j] =
        make_uint2(f32x4_to_e4m3x4(f[0], f[1], f[2], f[3]), f32x4_to_e4m3x4(f[4], f[5], f[6], f[7]));
    if ((j & 15) == 0) a.scales[(size_t)(j >> 4) * a.mp + t] = s;
  }
}

}  // namespace

cudaError_t launch_rmsnorm_fp8(const NormFp8Args& a, int sms, cudaStream_t s) {
  const int nv = a.H / 8;
  auto threads = [&](int v) { return ((nv + v - 1) / v + 31) / 32 * 32; };
  auto go = [&](auto kernel, int t) {
    PdlLaunch L(dim3(a.M), dim3(t), 0, s);
    return cudaLaunchKernelEx(&L.cfg, kernel, a);
  };
  if (nv <= 1024 && a.M <= 2 * sms) return go(rmsnorm_fp8_kernel<1, 1024>, threads(1));
  if (nv <= 1024) return go(rmsnorm_fp8_kernel<4, 256>, threads(4));
  return go(rmsnorm_fp8_kernel<4, 512>, threads(4));
}

}  // namespace moe
