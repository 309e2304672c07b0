// Residual addition, RMSNorm and quantisation to E4M3 in one pass:
//   r' = bf16(x + residual);  y = r' * rsqrt(mean(r'^2) + eps) * gain;
//   s = amax of |y| over 128 columns / 448;  codes = E4M3(y / s).
// y is not rounded before it is quantised.
//
// One CTA a row (or a warp, for narrow rows), a thread for each V times 8 columns, which
// stay in registers from the one read to the write: the row's sum is a reduction over the
// CTA, a group's maximum one over 16 lanes.  Bound by bytes for many rows (8192 x 7168, 413 MB, 62.7 us,
// 0.97 of the copy rate); for a few by latency (1 x 7168 2.1 us).
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
// V: pieces of a thread; T: threads of a row at most; R: rows of a CTA, a warp each if more than one.
template <int V, int T, int R>
__global__ void __launch_bounds__(T * R) rmsnorm_fp8_kernel(NormFp8Args a) {
  static_assert(R == 1 || T == 32, "several rows: a warp each");
  __shared__ float s_sum[T / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const int t = R * blockIdx.x + threadIdx.y, nv = a.H / 8;  // 16-byte pieces of a row
  if (R > 1 && t >= a.M) return;
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
  if constexpr (R == 1) {
    if (lane == 0) s_sum[warp] = ss;
    __syncthreads();
    ss = warp_sum(lane < threads / 32 ? s_sum[lane] : 0.f);
  }
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
    // y / s as a product with 1 / s, a step of fp32 off at most (y itself is): a division for
    // each value bounded the kernel (8192 rows of 7168 72.8 us)
    float to_normal = 1.f;  // a factor that makes 1 / s a normal number
    if (!(s >= 1e-30f && s <= 1e30f)) {
      to_normal = s < 1.f ? 0x1p64f : 0x1p-64f;
#pragma unroll
      for (int c = 0; c < 8; ++c) f[c] *= to_normal;
    }
    const float by = 1.f / (s * to_normal);
#pragma unroll
    for (int c = 0; c < 8; ++c) f[c] *= by;
    reinterpret_cast<uint2*>(a.codes)[row + j] =
        make_uint2(f32x4_to_e4m3x4(f[0], f[1], f[2], f[3]), f32x4_to_e4m3x4(f[4], f[5], f[6], f[7]));
    if ((j & 15) == 0) a.scales[(size_t)(j >> 4) * a.mp + t] = s;
  }
}

}  // namespace

cudaError_t launch_rmsnorm_fp8(const NormFp8Args& a, int sms, cudaStream_t s) {
  const int nv = a.H / 8;
  auto go = [&](auto kernel, int v, int rows) {
    PdlLaunch L(dim3((a.M + rows - 1) / rows), dim3(rows > 1 ? 32 : ((nv + v - 1) / v + 31) / 32 * 32, rows), 0, s);
    return cudaLaunchKernelEx(&L.cfg, kernel, a);
  };
  // A few rows: as many threads as a row has pieces (1 x 7168 2.1 us; with 4 pieces a thread
  // 0.9 more).  Many: 4 pieces a thread (8192 x 7168 62.7 us, with 2 pieces 65.4, with one half
  // as fast again); narrow rows a warp each (8192 x 512 4.8 us, as CTAs of their own 8.7), and
  // between them 2 pieces (8192 x 1040 11.7, with 4 13.4).
  const bool few = a.M <= 2 * sms;
  if (few && nv <= 1024) return go(rmsnorm_fp8_kernel<1, 1024, 1>, 1, 1);
  if (!few && nv <= 32) return go(rmsnorm_fp8_kernel<1, 32, 8>, 1, 8);
  if (!few && nv <= 64) return go(rmsnorm_fp8_kernel<2, 32, 8>, 2, 8);
  if (!few && nv <= 128) return go(rmsnorm_fp8_kernel<4, 32, 8>, 4, 8);
  if (!few && nv <= 256) return go(rmsnorm_fp8_kernel<2, 128, 1>, 2, 1);
  if (nv <= 1024) return go(rmsnorm_fp8_kernel<4, 256, 1>, 4, 1);
  return go(rmsnorm_fp8_kernel<4, 512, 1>, 4, 1);
}

}  // namespace moe
