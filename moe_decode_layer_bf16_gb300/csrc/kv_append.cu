// Writes a step's new keys and values into the FP8 paged cache.
//
// A block is a page of one key/value head: page_size tokens x head_dim E4M3
// codes with one fp32 scale.  The scale is the power of two at or above
// amax / 448 (at least 2^-126), so that when a louder token arrives and the
// scale grows, the codes the block already holds are divided by a power of
// two: exact, but for those that fall among the subnormal codes, which are
// rounded to nearest even.  A block whose first slot is written by the call
// takes its scale from the new tokens alone.  Infinities do not set the scale
// (they saturate at 448 of it) and NaN stays NaN.
//
// One CTA per (touched block, head, keys or values): it owns the block, so no
// atomics and no order.  The block's new rows are read once into registers (their
// place does not depend on the page, so that read does not wait for the page's
// number), their maximum reduced over the CTA, then converted and stored.  Bound
// by latency for a token each (64 sequences 4.9 us in a graph), and for prompt chunks by
// that chain of steps, of which a CTA has one block's under way at a time (4 x 2048
// tokens 13.0 us, 3.8 TB/s of the copy's 6.8).
#include "common.cuh"
#include "kernels.h"
#include "step_rows.h"
#include "../../include/moe_decode.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

// power of two at or above v (v >= 0, finite), at least 2^-126
MOE_DEV float pow2_ceil(float v) {
  const uint32_t bits = (__float_as_uint(fmaxf(v, 1.17549435e-38f)) + 0x7fffffu) & 0x7f800000u;
  return __uint_as_float(bits);
}

// |x| for the block's maximum: infinities and NaN do not count
MOE_DEV float finite_abs(float v) {
  const float a = fabsf(v);
  return a <= 3.4028235e38f ? a : 0.f;
}

MOE_DEV float e4m3_to_f32(uint32_t code) {
  uint32_t h;
  asm("{ .reg .b16 c; cvt.u16.u32 c, %1; cvt.rn.f16x2.e4m3x2 %0, c; }" : "=r"(h) : "r"(code));
  float f;
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.f32.f16 %0, lo; }" : "=f"(f) : "r"(h));
  return f;
}

// (out of line: the way of scales that are no powers of two)
__device__ __noinline__ float quotient(float x, float s) { return __fdiv_rn(x, s); }

// Four codes in the scale `from` rewritten in the scale `to`.
MOE_DEV uint32_t rescale4(uint32_t c, float from, float to) {
  const float k = __fdiv_rn(from, to);  // a power of two
  return f32x4_to_e4m3x4(e4m3_to_f32(c & 0xff) * k, e4m3_to_f32((c >> 8) & 0xff) * k,
                         e4m3_to_f32((c >> 16) & 0xff) * k, e4m3_to_f32(c >> 24) * k);
}

// (No read-only loads: this kernel starts while others may still write its inputs.)
template <int D, int P>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendArgs a) {
  constexpr int kLanes = D / 8;                       // threads of a token's row, 8 values each
  constexpr int kTok = kThreads / kLanes;             // tokens of a pass
  constexpr int kPass = (P + kTok - 1) / kTok;        // passes over a block
  __shared__ float s_red[kThreads / 32];
  const int tid = threadIdx.x;
  const int b = a.blocks == 1 ? blockIdx.x : blockIdx.x / a.blocks, j = blockIdx.x - b * a.blocks;
  const int head = blockIdx.y;
  const bool kv = blockIdx.z != 0;  // values
  // launched while the kernel before may still run: nothing is read before it is complete
  grid_dep_launch();
  grid_dep_wait();
  const int start = a.q_start[b], stop = a.q_start[b + 1];
  const int len = a.lens[b];
  const bool rows_ok = step_rows_ok(start, stop, a.total);
  const int n = rows_ok ? stop - start : 0;
  if (rows_ok && n == 0) return;
  const long long cap = (long long)a.width * P;
  bool bad = !rows_ok || n > a.max_new || len < n || len > cap;
  const int blk = bad ? 0 : (len - n) / P + j;
  if (!bad && blk > (len - 1) / P) return;  // the call touches fewer blocks of this sequence
  const int lo = max(blk * P, len - n), hi = bad ? lo : min((blk + 1) * P, len);  // new positions in this block
  const int held = lo - blk * P;                                                  // tokens the block holds already
  const int sub = tid % kLanes, row0 = tid / kLanes;
  const uint16_t* src = reinterpret_cast<const uint16_t*>(kv ? a.v : a.k);
  const long long stride = kv ? a.v_stride : a.k_stride;
  const uint16_t* rows = src + (long long)(start + lo - (len - n)) * stride + head * D + sub * 8;
  uint4 r[kPass];
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const int t = p * kTok + row0;
    r[p] = t < hi - lo ? __ldcg(reinterpret_cast<const uint4*>(rows + (long long)t * stride)) : make_uint4(0, 0, 0, 0);
  }
  int page = -1;
  if (!bad) {
    page = a.page_table[(size_t)b * a.width + blk];
    bad = page < 0 || page >= a.num_pages;
  }
  if (bad) {  // nothing is written for this block
    if (tid == 0) atomicExch(a.status, MOE_ERR_INVALID_ARG);
    return;
  }
  const size_t si = (size_t)page * a.kv_heads + head;
  uint8_t* dst = (kv ? a.v_cache : a.k_cache) + si * P * D;
  float* scale = (kv ? a.v_scale : a.k_scale) + si;
  const float old = held > 0 ? *scale : 0.f;
  float amax = 0.f;
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const uint32_t w[4] = {r[p].x, r[p].y, r[p].z, r[p].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fmaxf(finite_abs(bf16_lo(w[i])), finite_abs(bf16_hi(w[i]))));
  }
  amax = warp_max(amax);
  if ((tid & 31) == 0) s_red[tid >> 5] = amax;
  __syncthreads();  // (and every thread has read the old scale)
  amax = s_red[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) amax = fmaxf(amax, s_red[i]);
  float s = pow2_ceil(__fdiv_rn(amax, kFp8Max));
  if (held > 0) s = fmaxf(s, old);
  if (tid == 0) *scale = s;
  if (held > 0 && s != old) {
    for (int i = tid; i < held * D / 16; i += kThreads) {
      uint4* c = reinterpret_cast<uint4*>(dst) + i;
      const uint4 v = *c;
      *c = make_uint4(rescale4(v.x, old, s), rescale4(v.y, old, s), rescale4(v.z, old, s), rescale4(v.w, old, s));
    }
  }
  // x / s: a power of two's reciprocal is exact; a scale that the caller's own
  // cache brought along may be any number
  const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0;
  const float inv = __frcp_rn(s);
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const int t = p * kTok + row0;
    if (t < hi - lo) {
      float f[8] = {bf16_lo(r[p].x), bf16_hi(r[p].x), bf16_lo(r[p].y), bf16_hi(r[p].y),
                    bf16_lo(r[p].z), bf16_hi(r[p].z), bf16_lo(r[p].w), bf16_hi(r[p].w)};
      if (pow2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= inv;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = quotient(f[i], s);
      }
      uint2 q;
      q.x = f32x4_to_e4m3x4(f[0], f[1], f[2], f[3]);
      q.y = f32x4_to_e4m3x4(f[4], f[5], f[6], f[7]);
      *reinterpret_cast<uint2*>(dst + (size_t)(held + t) * D + sub * 8) = q;
    }
  }
}

template <int D>
cudaError_t launch_d(const AppendArgs& a, cudaStream_t s) {
  PdlLaunch L(dim3((unsigned)(a.B * a.blocks), (unsigned)a.kv_heads, 2), dim3(kThreads), 0, s);
  switch (a.page_size) {
    case 16: return cudaLaunchKernelEx(&L.cfg, kv_append_kernel<D, 16>, a);
    case 32: return cudaLaunchKernelEx(&L.cfg, kv_append_kernel<D, 32>, a);
    case 64: return cudaLaunchKernelEx(&L.cfg, kv_append_kernel<D, 64>, a);
    default: return cudaLaunchKernelEx(&L.cfg, kv_append_kernel<D, 128>, a);
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t s) {
  if (a.B == 0 || a.total == 0) return cudaSuccess;
  return a.head_dim == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace moe
