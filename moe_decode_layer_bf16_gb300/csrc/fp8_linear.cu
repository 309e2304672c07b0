// FP8 block-scaled linear layer: out[m, n] = sum_k x[m, k] * w[n, k] with
// x quantised per token per 128 columns (scale xs[m, kb] = amax / 448) and w
// in E4M3 with one fp32 scale for each 128 x 128 block, i.e.
//   out[m, n] = sum_kb xs[m, kb] * ws[n / 128, kb] * sum_{k in kb} xq[m, k] * wq[n, k],
// every sum in fp32, rounded once at the end.  The weight format is the one of
// the expert layers, so the attention projections around them use it too.
//
// Two kernels: the quantisation (a stream over x), and the product on
// tcgen05.mma.kind::f8f6f4 (E4M3 x E4M3, fp32 accumulators in tensor memory).
//
// The product.  The weights are the MMA's 128 rows and the tokens its columns
// (NT = 16 .. 256 of a chunk), so that one token still fills the MMA's rows
// and the weights are streamed once per 256 tokens.  The unit of work is a
// cell: (128 rows of w) x (a chunk of tokens) x (one 128-column k-block), i.e.
// one 16 KB weight tile and one NT x 128 activation tile through TMA (128-byte
// swizzle), four MMAs of K = 32 into one of the accumulator buffers, and an
// epilogue that adds the buffer, times ws * xs, to fp32 registers: the scales
// are fp32 values of their own for each k-block, so they cannot ride in the
// MMA.  Rows past N, tokens past M and columns past K are zeros of the TMA fill.
//
// Work split.  One CTA per SM.  Whole waves of (row tile, chunk) pairs are
// dealt out as they are; the remaining pairs are cut along K into one equal
// share of cells per CTA (stream-K), so that one token's 72 row tiles keep all
// 152 SMs streaming.  A CTA that holds a piece of a pair writes its fp32 sums to
// the workspace; the last to arrive adds the pieces in k order (the result does
// not depend on who is last).
//
// Roles (12 warps): TMA producer, MMA issuer, two warps that prepare the
// ws * xs products of each cell, eight epilogue warps (four lane quadrants x
// two column halves).  Every wait is bounded.
#include <cuda.h>

#include <algorithm>

#include "async.cuh"
#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"
#include "tmap.h"
#include "../../include/moe_decode.h"

namespace moe {

namespace {

// ------------------------------------------------------------- quantisation
// One 16-lane half-warp per (token, 128-column group), 8 columns a lane: one
// 16-byte load, a shuffle maximum, one 8-byte store.  K % 16 == 0, so a lane's
// 8 columns lie inside a row or outside of it as a whole.
constexpr int kQuantThreads = 256;

__global__ void __launch_bounds__(kQuantThreads) quant_rows_kernel(QuantArgs a) {
  grid_dep_launch();  // the product may start streaming its weights now
  const int lane16 = threadIdx.x & 15;
  const long long n_groups = (long long)a.M * a.nkb;
  const long long step = (long long)gridDim.x * (kQuantThreads / 16);
  for (long long gi = (long long)blockIdx.x * (kQuantThreads / 16) + (threadIdx.x >> 4); gi < n_groups; gi += step) {
    const long long m = gi / a.nkb;
    const int kb = (int)(gi - m * a.nkb);
    const int col = kb * kBlock + lane16 * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (col < a.K) v = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.x) + m * a.ldx + col));
    const float f[8] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y),
                        bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
    // the half-warps of a warp may hold different numbers of groups
    const unsigned mask = 0xffffu << (threadIdx.x & 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, o));
    const float s = group_scale(amax, a.e8m0 != 0);
    if (col < a.K) {
      uint2 q;
      q.x = f32x4_to_e4m3x4(__fdiv_rn(f[0], s), __fdiv_rn(f[1], s), __fdiv_rn(f[2], s), __fdiv_rn(f[3], s));
      q.y = f32x4_to_e4m3x4(__fdiv_rn(f[4], s), __fdiv_rn(f[5], s), __fdiv_rn(f[6], s), __fdiv_rn(f[7], s));
      *reinterpret_cast<uint2*>(a.codes + m * a.K + col) = q;
    }
    if (lane16 == 0) a.scales[gi] = s;
  }
}

// ------------------------------------------------------------- product
constexpr int kRows = 128;              // weight rows of a tile: the MMA's M
constexpr int kWTile = kRows * 128;     // 16 KB
constexpr int kNEpi = 8;                // epilogue warps
constexpr int kThreads = 12 * 32;
constexpr int kPW = 0, kMW = 1, kSW = 2, kEW0 = 4;

template <int NT>
struct Cfg {
  static constexpr int kXBox = NT < 32 ? NT : 32;             // token rows of one activation copy
  static constexpr int kStage = kWTile + NT * 128;            // ring stage: a weight and an activation tile
  static constexpr int kNST = std::min(12, 204 * 1024 / kStage);
  static constexpr int kTST = NT <= 128 ? 4 : 2;              // accumulator buffers in tensor memory
  static constexpr int kTCols = NT * kTST;                    // 64 .. 512, a power of two
  static constexpr int kHalf = NT / 2;                        // columns of an epilogue warp
  static constexpr int kSWarps = NT <= 32 ? 1 : 2;            // warps that prepare scale products
  static constexpr size_t kBars = (size_t)kNST * kStage;
  static constexpr int kNBars = 2 * kNST + 3 * kTST + 3;
  static constexpr size_t kScale = (kBars + kNBars * 8 + 15) / 16 * 16;  // [kTST][NT] fp32
  static constexpr size_t kMisc = kScale + (size_t)kTST * NT * 4;
  static constexpr size_t kSmem = 1024 + kMisc + 16;
};

struct LinMaps {
  CUtensorMap w, x;
};

// The pieces of work of CTA c: whole (tile, chunk) pairs c, c + G, ..., then
// its share of the cells of the remaining pairs, one pair after the other.
struct Pieces {
  const LinArgs& p;
  int c;
  int i;               // next whole pair of this CTA
  long long at, end;   // remaining cells [at, end) of the split pairs
  int pair, k0, k1;    // the current piece
  MOE_DEV Pieces(const LinArgs& a, int cta) : p(a), c(cta), i(0) {
    at = p.split_cells * c / p.G_split;
    end = p.split_cells * (c + 1) / p.G_split;
    if (c >= p.G_split) at = end = 0;
  }
  MOE_DEV bool next() {
    if (i < p.waves) {
      pair = i++ * p.G + c;
      k0 = 0;
      k1 = p.nkb;
      return true;
    }
    if (at >= end) return false;
    const long long t = at / p.nkb;
    pair = p.waves * p.G + (int)t;
    k0 = (int)(at - t * p.nkb);
    k1 = (int)min((long long)p.nkb, end - t * p.nkb);
    at = t * p.nkb + k1;
    return true;
  }
  // CTA that holds cell x of the split pairs
  MOE_DEV int owner(long long x) const { return (int)(((x + 1) * p.G_split - 1) / p.split_cells); }
};

MOE_DEV void store_out(const LinArgs& p, long long m, int n, float v) {
  if (p.out_fp32)
    reinterpret_cast<float*>(p.out)[m * p.N + n] = v;
  else
    reinterpret_cast<__nv_bfloat16*>(p.out)[m * p.N + n] = __float2bfloat16_rn(v);
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(LinArgs p, const __grid_constant__ LinMaps maps) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (su32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* ring = smem;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);
  uint64_t* empty = full + C::kNST;
  uint64_t* tfull = empty + C::kNST;
  uint64_t* tempty = tfull + C::kTST;
  uint64_t* sready = tempty + C::kTST;
  uint64_t* mma_done = sready + C::kTST;
  uint64_t* pdone = mma_done + 1;  // the eight epilogue warps wrote their part of a piece
  uint64_t* pdec = pdone + 1;      // whether this CTA is the last of the pair to arrive
  float* cstage = reinterpret_cast<float*>(smem + C::kScale);
  volatile int* s_misc = reinterpret_cast<volatile int*>(smem + C::kMisc);  // [0] tensor memory, [1] last to arrive
  int* status = p.status;

  if (tid == 0) {
    for (int i = 0; i < C::kNST; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < C::kTST; ++i) {
      mbar_init(tfull + i, 1);
      mbar_init(tempty + i, kNEpi);
      mbar_init(sready + i, C::kSWarps);
    }
    mbar_init(mma_done, 1);
    mbar_init(pdone, kNEpi);
    mbar_init(pdec, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMW) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32((const void*)s_misc)),
                 "r"(C::kTCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)s_misc[0];
  Pieces pc(p, blockIdx.x);

  if (warp == kPW) {
    // ================================================================ producer
    // Weights do not depend on the kernel before this one (the quantisation):
    // the ring's first tiles of them are in flight before it is waited for.
    uint32_t gs = 0;
    if (lane == 0) {
      {
        Pieces ahead(p, blockIdx.x);
        int n = 0;
        while (n < C::kNST && ahead.next()) {
          const int tile = ahead.pair % p.n_tiles;
          for (int kb = ahead.k0; kb < ahead.k1 && n < C::kNST; ++kb, ++n) {
            const int chunk = ahead.pair / p.n_tiles;
            const int ntok = min(p.chunk, p.M - chunk * p.chunk);
            const int nbox = (ntok + C::kXBox - 1) / C::kXBox;
            mbar_expect_tx(full + n, (uint32_t)(kWTile + nbox * C::kXBox * 128));
            tma_load_2d(ring + (size_t)n * C::kStage, &maps.w, kb * kBlock, tile * kRows, full + n);
          }
        }
      }
      grid_dep_wait();
      asm volatile("fence.proxy.async.global;" ::: "memory");  // codes of the kernel before are read with TMA
      int si = 0;
      uint32_t ph = 0;
      bool alive = true;
      while (alive && pc.next()) {
        const int tile = pc.pair % p.n_tiles, chunk = pc.pair / p.n_tiles;
        const int t0 = chunk * p.chunk;
        const int ntok = min(p.chunk, p.M - t0);
        const int nbox = (ntok + C::kXBox - 1) / C::kXBox;
        for (int kb = pc.k0; kb < pc.k1; ++kb) {
          uint8_t* st = ring + (size_t)si * C::kStage;
          if (gs >= (uint32_t)C::kNST) {
            if (!mbar_wait_landed(empty + si, ph ^ 1u, status)) { alive = false; break; }
            mbar_expect_tx(full + si, (uint32_t)(kWTile + nbox * C::kXBox * 128));
            tma_load_2d(st, &maps.w, kb * kBlock, tile * kRows, full + si);
          }
          for (int b = 0; b < nbox; ++b)
            tma_load_2d(st + kWTile + b * C::kXBox * 128, &maps.x, kb * kBlock, t0 + b * C::kXBox, full + si);
          ++gs;
          if (++si == C::kNST) { si = 0; ph ^= 1u; }
        }
      }
      // every copy this CTA issued lands before it ends
      for (uint32_t j = (gs > (uint32_t)C::kNST ? gs - C::kNST : 0); j < gs; ++j)
        mbar_wait_landed(full + (j % C::kNST), (j / C::kNST) & 1u, status);
    }
    __syncwarp();
  } else if (warp == kMW) {
    // ================================================================ MMA issue
    if (lane == 0) {
      int si = 0, ti = 0;
      uint32_t ph = 0, tp = 0;
      bool alive = true;
      while (alive && pc.next()) {
        const int chunk = pc.pair / p.n_tiles;
        const int ntok = min(p.chunk, p.M - chunk * p.chunk);
        const uint32_t idesc = instr_desc(kRows, (ntok + 15) & ~15);
        for (int kb = pc.k0; kb < pc.k1; ++kb) {
          if (!mbar_wait_landed(tempty + ti, tp ^ 1u, status) || !mbar_wait_landed(full + si, ph, status)) {
            alive = false;
            break;
          }
          tc_fence_after();
          const uint32_t sb = su32(ring + (size_t)si * C::kStage);
          const uint64_t da = smem_desc(sb), db = smem_desc(sb + kWTile);
          const uint32_t dt = tmem + (uint32_t)(ti * NT);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) tc_mma(dt, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1 : 0);
          tc_commit(empty + si);
          tc_commit(tfull + ti);
          if (++si == C::kNST) { si = 0; ph ^= 1u; }
          if (++ti == C::kTST) { ti = 0; tp ^= 1u; }
        }
      }
      // every MMA this thread issued is complete before the memory is freed
      tc_commit(mma_done);
      mbar_wait_landed(mma_done, 0, status);
    }
    __syncwarp();
  } else if (warp >= kSW && warp < kSW + C::kSWarps) {
    // ================================================================ scale products
    grid_dep_wait();
    constexpr int kCols = NT / C::kSWarps;           // columns of this warp
    constexpr int kPer = (kCols + 31) / 32;
    const int c0 = (warp - kSW) * kCols;
    int ti = 0;
    uint32_t tp = 0;
    bool alive = true;
    while (alive && pc.next()) {
      const int tile = pc.pair % p.n_tiles, chunk = pc.pair / p.n_tiles;
      const int t0 = chunk * p.chunk;
      const int ntok = min(p.chunk, p.M - t0);
      const float* wr = p.w_s + (size_t)tile * p.nkb;
      for (int kb = pc.k0; kb < pc.k1; ++kb) {
        const float ws = ld_ca(wr + kb);
        float v[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int col = c0 + 32 * j + lane;
          v[j] = 32 * j + lane < kCols && col < ntok ? ws * ld_ca(p.xs + (size_t)(t0 + col) * p.nkb + kb) : 0.f;
        }
        if (!mbar_wait_landed(tempty + ti, tp ^ 1u, status)) { alive = false; break; }
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (32 * j + lane < kCols) cstage[ti * NT + c0 + 32 * j + lane] = v[j];
        __syncwarp();
        if (lane == 0) mbar_arrive(sready + ti);
        if (++ti == C::kTST) { ti = 0; tp ^= 1u; }
      }
    }
  } else if (warp >= kEW0) {
    // ================================================================ epilogue
    const int qd = warp & 3, hf = (warp - kEW0) >> 2;
    const int r = 32 * qd + lane;                 // row of the 128-row tile
    const int col0 = hf * C::kHalf;
    constexpr int kStep = C::kHalf < 16 ? C::kHalf : 16;
    float acc[C::kHalf];
    int ti = 0;
    uint32_t tp = 0, np = 0;  // np: split pieces so far (phases of pdone and pdec)
    bool alive = true;
    while (alive && pc.next()) {
      const int tile = pc.pair % p.n_tiles, chunk = pc.pair / p.n_tiles;
      const int t0 = chunk * p.chunk;
      const int ntok = min(p.chunk, p.M - t0);
#pragma unroll
      for (int j = 0; j < C::kHalf; ++j) acc[j] = 0.f;
      for (int kb = pc.k0; kb < pc.k1; ++kb) {
        if (!mbar_wait_landed(tfull + ti, tp, status) || !mbar_wait_landed(sready + ti, tp, status)) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint32_t ta = tmem + ((uint32_t)(32 * qd) << 16) + (uint32_t)(ti * NT + col0);
        const float* cs = cstage + ti * NT + col0;
#pragma unroll
        for (int j0 = 0; j0 < C::kHalf; j0 += kStep) {
          if (col0 + j0 < ntok) {
            float d[kStep];
            if constexpr (kStep == 16) tc_ld16(ta + j0, d); else tc_ld8(ta + j0, d);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < kStep; j += 4) {
              const float4 f = *reinterpret_cast<const float4*>(cs + j0 + j);
              acc[j0 + j] += d[j] * f.x;
              acc[j0 + j + 1] += d[j + 1] * f.y;
              acc[j0 + j + 2] += d[j + 2] * f.z;
              acc[j0 + j + 3] += d[j + 3] * f.w;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty + ti);
        if (++ti == C::kTST) { ti = 0; tp ^= 1u; }
      }
      if (!alive) break;
      const int n = tile * kRows + r;
      const bool whole = pc.k0 == 0 && pc.k1 == p.nkb;
      int c_first = 0, c_last = 0;
      if (!whole) {
        // this piece's sums go to the workspace; the last CTA of the pair to
        // arrive adds all pieces in k order
        const long long x0 = (long long)(pc.pair - p.waves * p.G) * p.nkb;
        c_first = pc.owner(x0);
        c_last = pc.owner(x0 + p.nkb - 1);
        // a CTA's pieces: slot 0 continues a pair of the CTA before it, slot 1 starts one
        float* part = p.partials + ((size_t)blockIdx.x * 2 + (pc.k0 == 0 ? 1 : 0)) * NT * kRows;
#pragma unroll
        for (int j = 0; j < C::kHalf; ++j)
          if (col0 + j < ntok) __stcg(part + (size_t)(col0 + j) * kRows + r, acc[j]);
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(pdone);
        if (!mbar_wait_landed(pdone, np & 1u, status)) break;
        if (tid == kEW0 * 32) {
          __threadfence();
          const int got = atom_add_acq_rel(p.tickets + c_first, 1);
          const bool last = got == c_last - c_first;
          if (last) p.tickets[c_first] = 0;  // ready for the next call
          s_misc[1] = last;
          mbar_arrive(pdec);
        }
        if (!mbar_wait_landed(pdec, np & 1u, status)) break;
        ++np;
        if (!s_misc[1]) continue;
        __threadfence();
#pragma unroll
        for (int j = 0; j < C::kHalf; ++j) acc[j] = 0.f;
        for (int c = c_first; c <= c_last; ++c) {
          const float* ps = p.partials + ((size_t)c * 2 + (c == c_first ? 1 : 0)) * NT * kRows;
#pragma unroll
          for (int j = 0; j < C::kHalf; ++j)
            if (col0 + j < ntok) acc[j] += __ldcg(ps + (size_t)(col0 + j) * kRows + r);
        }
      }
      if (n < p.N) {
#pragma unroll
        for (int j = 0; j < C::kHalf; ++j)
          if (col0 + j < ntok) store_out(p, t0 + col0 + j, n, acc[j]);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kMW) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTCols) : "memory");
  }
}

template <int NT>
cudaError_t launch_nt(const LinPlan& p, const LinArgs& a, const LinMaps& maps, bool pdl, cudaStream_t s) {
  using C = Cfg<NT>;
  // a process-wide attribute of the kernel, set once (an atomic static)
  static const cudaError_t rc =
      cudaFuncSetAttribute(linear_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (rc != cudaSuccess) return rc;
  if (pdl) {
    PdlLaunch L(dim3(p.G), dim3(kThreads), C::kSmem, s);
    return cudaLaunchKernelEx(&L.cfg, linear_kernel<NT>, a, maps);
  }
  linear_kernel<NT><<<p.G, kThreads, C::kSmem, s>>>(a, maps);
  return cudaGetLastError();
}

}  // namespace

// Token columns of a chunk: the smallest MMA width that holds all tokens, up
// to 256; above, equal chunks of at most 256 (a multiple of 16).
void plan_linear(LinPlan& p, int M, int N, int K, int sms) {
  p.M = M; p.N = N; p.K = K;
  p.nkb = (K + kBlock - 1) / kBlock;
  p.nt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
  p.n_chunks = (M + p.nt - 1) / p.nt;
  p.chunk = ((M + p.n_chunks - 1) / p.n_chunks + 15) & ~15;
  p.n_chunks = (M + p.chunk - 1) / p.chunk;
  p.n_tiles = (N + kRows - 1) / kRows;
  const long long pairs = (long long)p.n_chunks * p.n_tiles;
  const long long cells = pairs * p.nkb;
  p.G = (int)std::min<long long>({cells, (long long)sms, (long long)kLinMaxCtas});
  p.waves = (int)(pairs / p.G);
  p.split_cells = (pairs - (long long)p.waves * p.G) * p.nkb;
  // at least kLinMinRun cells a CTA: shorter pieces cost more to add than they save
  const long long rest = pairs - (long long)p.waves * p.G;
  p.G_split = (int)std::max<long long>(1, std::min<long long>(p.G, std::max(p.split_cells / kLinMinRun, rest)));
}

size_t linear_partial_bytes(const LinPlan& p) {
  return p.split_cells > 0 && p.G_split > 1 ? (size_t)p.G_split * 2 * p.nt * kRows * sizeof(float) : 0;
}

cudaError_t launch_quant_rows(const QuantArgs& a, int sms, cudaStream_t s) {
  if (a.M == 0) return cudaSuccess;
  const long long groups = (long long)a.M * a.nkb;
  const long long ctas = (groups + kQuantThreads / 16 - 1) / (kQuantThreads / 16);
  quant_rows_kernel<<<(unsigned)std::min<long long>(ctas, (long long)sms * 8), kQuantThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_linear(const LinPlan& p, const uint8_t* xq, const float* xs, const uint8_t* w, const float* w_s,
                          void* out, int out_fp32, int* status, int* tickets, float* partials, bool pdl,
                          cudaStream_t s) {
  LinMaps maps;
  if (!tmap_2d(&maps.w, w, p.K, p.N, 128, kRows) || !tmap_2d(&maps.x, xq, p.K, p.M, 128, p.nt < 32 ? p.nt : 32))
    return cudaErrorInvalidValue;
  LinArgs a;
  a.xs = xs; a.w_s = w_s; a.out = out; a.out_fp32 = out_fp32;
  a.M = p.M; a.N = p.N; a.nkb = p.nkb; a.chunk = p.chunk; a.n_tiles = p.n_tiles;
  a.G = p.G; a.waves = p.waves; a.G_split = p.G_split; a.split_cells = p.split_cells;
  a.status = status; a.tickets = tickets; a.partials = partials;
  switch (p.nt) {
    case 16: return launch_nt<16>(p, a, maps, pdl, s);
    case 32: return launch_nt<32>(p, a, maps, pdl, s);
    case 64: return launch_nt<64>(p, a, maps, pdl, s);
    case 128: return launch_nt<128>(p, a, maps, pdl, s);
    default: return launch_nt<256>(p, a, maps, pdl, s);
  }
}

}  // namespace moe
