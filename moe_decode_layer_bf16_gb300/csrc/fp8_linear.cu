// FP8 block-scaled linear layer: out[m, n] = sum_k x[m, k] * w[n, k] with
// x quantised per token per 128 columns (scale xs[m, kb] = amax / 448) and w
// in E4M3 with one fp32 scale for each 128 x 128 block, i.e.
//   out[m, n] = sum_kb xs[m, kb] * ws[n / 128, kb] * sum_{k in kb} xq[m, k] * wq[n, k],
// every sum in fp32, rounded once at the end.  The weight format is the one of
// the expert layers, so the attention projections around them use it too.
//
// What bounds it.  One token of 7168 -> 9216 is 66 MB of weights: 14.4 us, 4.6 TB/s (0.68
// of the copy rate; start and exchange of sums are about 5 us of it).  4096 tokens are
// 541 GFLOP: 221 us back to back, 2450 TFLOP/s, of which the quantisation takes 15 and
// the MMAs alone 160; between MMAs of a cell the accumulator buffer goes to the epilogue
// and back, and with two buffers of 256 columns (all of tensor memory) that round trip
// shows.
//
// Two kernels: the quantisation (a stream over x), and the product on
// tcgen05.mma.kind::f8f6f4 (E4M3 x E4M3, fp32 accumulators in tensor memory);
// for a few tokens one, the product quantising what it needs as it goes.
//
// The product, in two arrangements of one kernel.  Up to 128 tokens the weights are
// the MMA's 128 rows and the tokens its columns (NT = 16 .. 128), so that one
// token still fills the MMA's rows and the weights are streamed once.  Above,
// 256 tokens are the rows and 256 weight rows the columns of a pair of CTAs
// (cta_group::2): each holds 128 of the tokens with their accumulators and 128
// of the weight rows, so a cell of 256 x 256 takes 32 KB of copies in each CTA
// where a CTA alone needs 48 KB for half of it.  A thread of the epilogue then
// owns one token and one weight block, and needs one scale for its 128 columns.
//
// The unit of work is a cell: a pair of a row tile and a column tile in one
// 128-column k-block, i.e. one tile of each operand through TMA (128-byte
// swizzle), four MMAs of K = 32 into one of the accumulator buffers, and an
// epilogue that adds the buffer, times ws * xs, to fp32 registers: the scales
// are fp32 values of their own for each k-block, so they cannot ride in the
// MMA.  Rows past N, tokens past M and columns past K are zeros of the TMA fill.
//
// Work split.  One CTA per SM (a pair of CTAs counts as one here).  Whole waves of
// pairs of tiles are dealt out as they are; the remaining ones are cut along K
// into pieces of equal length where that is worth the exchange of their sums, one
// a CTA, so that one token's 72 row tiles keep 144 SMs streaming.  A
// CTA that holds a piece of a pair writes its fp32 sums to the workspace; the
// last to arrive adds the pieces in k order (the result does not depend on who
// is last).
//
// Roles (12 warps): TMA producer, MMA issuer, a warp that copies each cell's
// token scales and an idle one (or two of the six that quantise), eight epilogue
// warps (four lane quadrants x two column halves).  Every wait is bounded.
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
// A warp takes eight 128-column groups of a token: a 16-lane half-warp for a group
// at a time, 8 columns a lane, four groups of each in flight; one 16-byte load, a
// shuffle maximum, one 8-byte store a group.  K % 16 == 0, so a lane's 8 columns
// lie inside a row or outside of it as a whole.
//
// A code is E4M3(fl32(x / s)).  The quotient comes from one reciprocal a group and
// Markstein's correction (IBM J. Res. Dev. 34, 1990): q = fl(x y) with
// y = fl(1 / s), then fl(q + fl(x - q s) y) is fl(x / s).  x and amax are bf16, so
// there are 128 x 128 pairs of significands, and the two agree for all of them.
constexpr int kQuantThreads = 256;

struct Quotient {
  float s, y;
  bool far;  // 1 / s or the products may be no normal numbers
  MOE_DEV explicit Quotient(float scale) {
    s = scale;
    y = __frcp_rn(scale);
    far = !(scale >= 1e-30f && scale <= 1e30f);
  }
  MOE_DEV float operator()(float x) const {
    const float q = x * y;
    return fmaf(fmaf(-q, s, x), y, q);
  }
};
// the same by division, for scales where the reciprocal will not do (kept out of line)
__device__ __noinline__ uint32_t codes4_far(float s, uint32_t a, uint32_t b) {
  return f32x4_to_e4m3x4(__fdiv_rn(bf16_lo(a), s), __fdiv_rn(bf16_hi(a), s), __fdiv_rn(bf16_lo(b), s),
                         __fdiv_rn(bf16_hi(b), s));
}
MOE_DEV uint32_t codes4(const Quotient& q, uint32_t a, uint32_t b) {  // of four bf16 values
  return f32x4_to_e4m3x4(q(bf16_lo(a)), q(bf16_hi(a)), q(bf16_lo(b)), q(bf16_hi(b)));
}
MOE_DEV uint2 codes8(const Quotient& q, const uint4& v) {
  uint2 c = make_uint2(codes4(q, v.x, v.y), codes4(q, v.z, v.w));
  if (q.far) c = make_uint2(codes4_far(q.s, v.x, v.y), codes4_far(q.s, v.z, v.w));
  return c;
}
MOE_DEV float amax8(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
  return m;
}

// (No read-only loads: the kernels here start while others may still write their inputs.)
__global__ void __launch_bounds__(kQuantThreads) quant_rows_kernel(QuantArgs a) {
  grid_dep_wait();    // (launched while the kernel before may still run)
  grid_dep_launch();  // the product may start streaming its weights now
  const int lane = threadIdx.x & 31, lane16 = lane & 15;
  const int n_runs = (a.nkb + 7) / 8, n_units = a.M * n_runs;
  for (int u = blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5); u < n_units; u += gridDim.x * (kQuantThreads / 32)) {
    const int m = u / n_runs, kb0 = (u - m * n_runs) * 8 + (lane >> 4);  // this half-warp: groups kb0, kb0 + 2, ...
    const uint16_t* x = reinterpret_cast<const uint16_t*>(a.x) + m * a.ldx + lane16 * 8;
    uint8_t* codes = a.codes + (size_t)m * a.K + lane16 * 8;
    uint4 v[4];
    float amax[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = (kb0 + 2 * i) * kBlock;
      v[i] = col + lane16 * 8 < a.K ? __ldcg(reinterpret_cast<const uint4*>(x + col)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) amax[i] = amax8(v[i]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], o));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int kb = kb0 + 2 * i;
      const float s = group_scale(amax[i], a.e8m0 != 0);
      const uint2 c = codes8(Quotient(s), v[i]);
      if (kb * kBlock + lane16 * 8 < a.K) *reinterpret_cast<uint2*>(codes + kb * kBlock) = c;
      // k-blocks first: the product reads a block's scales as one run
      if (lane16 == 0 && kb < a.nkb) a.scales[(size_t)kb * a.mp + m] = s;
    }
  }
}

// ------------------------------------------------------------- product
constexpr int kRows = 128;              // rows of a row tile: the MMA's M
constexpr int kRTile = kRows * 128;     // 16 KB
constexpr int kNEpi = 8;                // epilogue warps
constexpr int kPW = 0, kMW = 1, kSW = 2, kEW0 = 4, kEW1 = kEW0 + kNEpi;

// NT columns; TR: the tokens are the rows; XQ: the kernel quantises x itself
constexpr int kTurnRow = 80;  // 64 bytes of a row; 16-byte accesses of 8 rows meet no bank twice

template <int NT, bool TR, bool XQ>
struct Cfg {
  static_assert(!XQ || (!TR && NT <= 16), "a warp quantises a cell's tokens, eight at a time");
  // warps that quantise: 2, 3 and four behind the epilogue (a cell takes one of
  // them 1650 clocks, and a cell's weights arrive every 760: with two warps one
  // token 20.0 us)
  static constexpr int kQW = XQ ? 6 : 0;
  static constexpr int kThreads = (kEW1 + (XQ ? kQW - 2 : 0)) * 32;
  static constexpr bool kPair = TR;                           // two CTAs work on a cell
  static constexpr int kCRows = kPair ? NT / 2 : NT;          // rows of this CTA's column tile
  static constexpr int kCBox = TR ? kCRows : std::min(NT, 32);  // of them in one copy (tokens: no more than there are)
  static constexpr int kStage = kRTile + kCRows * 128;        // ring stage: a row tile and a column tile
  static constexpr int kRaw = XQ ? 2 : 1;                     // cells of a quantising warp whose rows of x are on their way
  static constexpr size_t kRawBytes = (size_t)kQW * kRaw * NT * 256;
  static constexpr int kNST = std::min(12, (int)((212 * 1024 - kRawBytes) / kStage));
  // weight tiles in flight before the codes are waited for: the copies complete
  // in order, so more of them delay the first cell's codes (11 of 11: one
  // token 23.1 us, first cell 4.7 us after the start).  XQ: all (holding the
  // others back until the first rows of x are here: 18.4 -> 19.1 us)
  static constexpr int kAhead = XQ ? kNST : std::min(kNST, 4);
  // weight tiles brought into L2 before the kernel before is complete (one token, 7168 ->
  // 9216, and 8 tokens, 7168 -> 7168, us in a graph: 6 14.4 14.5, 12 14.6 14.5, 20 14.6
  // 14.7, 32 15.5 15.3; other sizes alike)
  static constexpr int kPrefetch = 6;
  static constexpr int kTST = NT <= 128 ? 4 : 2;              // accumulator buffers in tensor memory
  static constexpr int kTCols = NT * kTST;                    // 64 .. 512, a power of two
  static constexpr int kHalf = NT / 2;                        // columns of an epilogue warp
  static constexpr int kToks = TR ? kRows : NT;               // tokens of a cell
  static constexpr int kXST = 8;                              // cells whose token scales are in flight
  static constexpr size_t kBars = (size_t)kNST * kStage;
  static constexpr int kNBars = 2 * kNST + 2 * kTST + 2 * kXST + 3;
  static constexpr size_t kScale = (kBars + kNBars * 8 + 15) / 16 * 16;  // [kXST][kToks] fp32
  static constexpr size_t kMisc = kScale + (size_t)kXST * kToks * 4;
  static constexpr size_t kRawAt = kMisc + 16;
  // TR: where an epilogue warp turns 64 bytes of each of its 32 output rows
  static constexpr size_t kTurnAt = (kRawAt + kRawBytes + 15) / 16 * 16;
  static constexpr size_t kSmem = 1024 + kTurnAt + (TR ? (size_t)kNEpi * 32 * kTurnRow : 0);
  // registers: 12 warps start with 168 a thread; with 128 accumulators the
  // epilogue takes 232 of them (it spills with 216) and the other four warps keep 40
  // (256 x 232 + 128 x 40 = 384 x 168)
  static constexpr bool kSplitRegs = TR;
};

struct LinMaps {
  CUtensorMap w, x;
};

// The pieces of work of CTA c: whole pairs c, c + G, ..., then at most one piece of
// a remaining pair, from a table (no division is left for the kernel's first steps).
struct Pieces {
  const LinArgs& p;
  int i;             // next whole pair of this CTA
  int k0, k1;        // the current piece: k-blocks
  int cw, ct;        // its weight tile and token tile (of both CTAs)
  int row, col;      // this CTA's row tile, and the column tile
  MOE_DEV explicit Pieces(const LinArgs& a) : p(a), i(0) {}
  MOE_DEV int cta() const { return p.tok_rows ? blockIdx.x >> 1 : blockIdx.x; }
  MOE_DEV bool next() {
    if (i < p.waves) {
      // weight tiles follow one another within a token tile
      const int pair = i * p.G + cta();
      ct = pair / p.n_wt;
      cw = pair - ct * p.n_wt;
      k0 = 0;
      k1 = p.nkb;
    } else {
      const LinArgs::Piece& q = p.piece[cta()];
      if (i > p.waves || q.k0 == q.k1) return false;
      cw = q.w;
      ct = q.t;
      k0 = q.k0;
      k1 = q.k1;
    }
    ++i;
    row = p.tok_rows ? 2 * ct + (blockIdx.x & 1) : cw;
    col = p.tok_rows ? cw : ct;
    return true;
  }
};

// (a0, a1) += (d0, d1) * (f0, f1), one packed instruction
MOE_DEV void fma2(float& a0, float& a1, float d0, float d1, float f0, float f1) {
  asm("{ .reg .b64 a, d, f;\n mov.b64 a, {%0, %1};\n mov.b64 d, {%2, %3};\n mov.b64 f, {%4, %5};\n"
      " fma.rn.f32x2 a, d, f, a;\n mov.b64 {%0, %1}, a; }"
      : "+f"(a0), "+f"(a1) : "f"(d0), "f"(d1), "f"(f0), "f"(f1));
}

MOE_DEV void store_out(const LinArgs& p, long long m, int n, float v) {
  if (p.out_fp32)
    reinterpret_cast<float*>(p.out)[m * p.N + n] = v;
  else
    reinterpret_cast<__nv_bfloat16*>(p.out)[m * p.N + n] = __float2bfloat16_rn(v);
}

// A warp's 32 rows (lane: row) of kCols values, of which `ncol` are live, written
// to out[m0 + row][n0 ...] as E-byte values.
template <int W>  // bytes of a store
MOE_DEV void store_rows(uint8_t* out, size_t row_bytes, const uint8_t* turn, int lane, int rows, int bytes) {
  constexpr int kLanes = 64 / W < 32 ? 64 / W : 32;  // of a row
  const int at = lane % kLanes * W;
#pragma unroll 4
  for (int r = lane / kLanes; r < rows; r += 32 / kLanes) {
    if (at < bytes) {
      const uint8_t* src = turn + r * kTurnRow + at;
      uint8_t* dst = out + r * row_bytes + at;
      if constexpr (W == 16) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
      if constexpr (W == 4) *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(src);
      if constexpr (W == 2) *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(src);
    }
  }
}
template <int E, int kCols>
MOE_DEV void store_turned(const LinArgs& p, uint8_t* turn, const float* acc, int lane, int m0, int n0, int rows, int ncol) {
  constexpr int kStep = 64 / E;  // columns at a time
  const size_t row_bytes = (size_t)p.N * E;
  uint8_t* out = reinterpret_cast<uint8_t*>(p.out) + m0 * row_bytes + (size_t)n0 * E;
#pragma unroll
  for (int j0 = 0; j0 < kCols; j0 += kStep) {
    if (j0 >= ncol) break;
    __syncwarp();  // the bytes before have been read
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* v = acc + j0 + i * (16 / E);
      uint4 w;
      if constexpr (E == 4)
        w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      else
        w = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
      *reinterpret_cast<uint4*>(turn + lane * kTurnRow + 16 * i) = w;
    }
    __syncwarp();
    const int bytes = min(kStep, ncol - j0) * E;
    if (row_bytes % 16 == 0)  // (then ncol * E is a multiple of 16 too)
      store_rows<16>(out + j0 * E, row_bytes, turn, lane, rows, bytes);
    else if (row_bytes % 4 == 0)
      store_rows<4>(out + j0 * E, row_bytes, turn, lane, rows, bytes);
    else if constexpr (E == 2) {
      store_rows<2>(out + j0 * E, row_bytes, turn, lane, rows, bytes);
    }
  }
}

template <int NT, bool TR, bool XQ>
__global__ void __launch_bounds__((Cfg<NT, TR, XQ>::kThreads), 1) linear_kernel(LinArgs p, const __grid_constant__ LinMaps maps) {
  using C = Cfg<NT, TR, XQ>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (su32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (known to be the same in a warp)
  uint8_t* ring = smem;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);
  uint64_t* empty = full + C::kNST;
  uint64_t* tfull = empty + C::kNST;
  uint64_t* tempty = tfull + C::kTST;
  uint64_t* sfull = tempty + C::kTST;
  uint64_t* sempty = sfull + C::kXST;
  uint64_t* mma_done = sempty + C::kXST;
  uint64_t* pdone = mma_done + 1;  // the eight epilogue warps wrote their part of a piece
  uint64_t* pdec = pdone + 1;      // whether this CTA is the last of the pair to arrive
  float* xring = reinterpret_cast<float*>(smem + C::kScale);
  volatile int* s_misc = reinterpret_cast<volatile int*>(smem + C::kMisc);  // [0] tensor memory, [1] last to arrive
  int* status = p.status;

  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.w) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.x) : "memory");
    for (int i = 0; i < C::kNST; ++i) {
      mbar_init(full + i, XQ || C::kPair ? 2 : 1);  // the copies (of both CTAs), and a quantising warp
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < C::kTST; ++i) {
      mbar_init(tfull + i, 1);
      mbar_init(tempty + i, C::kPair ? 2 * kNEpi : kNEpi);  // (a pair's MMAs wait for both CTAs' epilogues)
    }
    for (int i = 0; i < C::kXST; ++i) {
      mbar_init(sfull + i, 1);
      mbar_init(sempty + i, kNEpi);
    }
    mbar_init(mma_done, 1);
    mbar_init(pdone, kNEpi);
    mbar_init(pdec, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMW) {
    if constexpr (C::kPair) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32((const void*)s_misc)),
                   "r"(C::kTCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32((const void*)s_misc)),
                   "r"(C::kTCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  // launched while the kernel before may still run: each role waits for it before
  // it reads or writes.  Only where that kernel is this call's quantisation do the
  // weights' copies not wait for it; else their first tiles are brought into L2
  // meanwhile.
  grid_dep_launch();
  tc_fence_before();
  if constexpr (C::kPair) cluster_sync(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)s_misc[0];
  const int rank = C::kPair ? blockIdx.x & 1 : 0;  // CTA of the pair; CTA 0 issues the MMAs
  Pieces pc(p);
  // tokens of a token tile, live columns of a column tile
  auto toks = [&](int t) { return min(p.chunk, p.M - t * p.chunk); };
  auto cols = [&](int c) { return TR ? min(NT, p.N - c * NT) : toks(c); };

  if (warp < kEW0 || (XQ && warp >= kEW1)) {
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == kPW) {
      // ================================================================ producer
      // Weights do not depend on the kernel before this one (the quantisation):
      // the first tiles of them are in flight before it is waited for.
      if (elect_one()) {
        uint32_t gs = 0, ahead = 0;
        auto load_w = [&](const Pieces& q, int kb, int si) {
          uint8_t* st = ring + (size_t)si * C::kStage;
          const int nbox = XQ ? 0 : (cols(q.col) + C::kCBox - 1) / C::kCBox;
          if constexpr (C::kPair) {
            // both CTAs' copies count on CTA 0's barrier
            const uint32_t bar = mapa(su32(full + si), 0);
            mbar_expect_tx_at(bar, (uint32_t)(kRTile + C::kCRows * 128));
            tma_load_2d_pair(st + kRTile, &maps.w, kb * kBlock, q.col * NT + rank * C::kCRows, bar);
          } else {
            mbar_expect_tx(full + si, (uint32_t)(kRTile + nbox * C::kCBox * 128));
            tma_load_2d(st, &maps.w, kb * kBlock, q.row * kRows, full + si);
          }
        };
        if (!p.after_quant) {
          Pieces q(p);
          int n = 0;
          while (n < C::kPrefetch && q.next())
            for (int kb = q.k0; kb < q.k1 && n < C::kPrefetch; ++kb, ++n)
              tma_prefetch_2d(&maps.w, kb * kBlock, TR ? q.col * NT + rank * C::kCRows : q.row * kRows);
          grid_dep_wait();
        }
        {
          Pieces q(p);
          while (ahead < (uint32_t)C::kAhead && q.next())
            for (int kb = q.k0; kb < q.k1 && ahead < (uint32_t)C::kAhead; ++kb) load_w(q, kb, (int)ahead++);
        }
        if (!XQ) {
          if (p.after_quant) grid_dep_wait();
          asm volatile("fence.proxy.async.global;" ::: "memory");  // codes of the kernel before are read with TMA
        }
        int si = 0;
        uint32_t ph = 0;
        bool alive = true;
        while (alive && pc.next()) {
          const int t0 = (TR ? pc.row : pc.col) * p.chunk;
          const int nbox = TR ? 1 : XQ ? 0 : (toks(pc.col) + C::kCBox - 1) / C::kCBox;
          for (int kb = pc.k0; kb < pc.k1; ++kb) {
            if (gs >= ahead) {
              if (gs >= (uint32_t)C::kNST && !mbar_wait_landed(empty + si, ph ^ 1u, status)) { alive = false; break; }
              load_w(pc, kb, si);
            }
            uint8_t* xt = ring + (size_t)si * C::kStage + (TR ? 0 : kRTile);
            if constexpr (C::kPair)
              tma_load_2d_pair(xt, &maps.x, kb * kBlock, t0, mapa(su32(full + si), 0));
            else
              for (int b = 0; b < nbox; ++b)
                tma_load_2d(xt + b * C::kCBox * 128, &maps.x, kb * kBlock, t0 + b * C::kCBox, full + si);
            ++gs;
            if (++si == C::kNST) { si = 0; ph ^= 1u; }
          }
        }
        // every copy this CTA issued lands before it ends (a pair's, before both end)
        for (uint32_t j = (gs > (uint32_t)C::kNST ? gs - C::kNST : 0); j < gs && rank == 0; ++j)
          mbar_wait_landed(full + (j % C::kNST), (j / C::kNST) & 1u, status);
      }
      __syncwarp();
    } else if (warp == kMW) {
      // ================================================================ MMA issue
      if (rank == 0 && elect_one()) {
        int si = 0, ti = 0;
        uint32_t ph = 0, tp = 0;
        bool alive = true;
        while (alive && pc.next()) {
          // (a pair's columns are always 256: those past N are zeros)
          const uint32_t idesc = C::kPair ? instr_desc(2 * kRows, NT) : instr_desc(kRows, (cols(pc.col) + 15) & ~15);
          for (int kb = pc.k0; kb < pc.k1; ++kb) {
            if (!mbar_wait_landed(tempty + ti, tp ^ 1u, status) || !mbar_wait_landed(full + si, ph, status)) {
              alive = false;
              break;
            }
            tc_fence_after();
            const uint32_t sb = su32(ring + (size_t)si * C::kStage);
            const uint64_t da = smem_desc(sb), db = smem_desc(sb + kRTile);
            const uint32_t dt = tmem + (uint32_t)(ti * NT);
            if constexpr (C::kPair) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) tc_mma_pair(dt, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1 : 0);
              tc_commit_pair(empty + si);
              tc_commit_pair(tfull + ti);
            } else {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) tc_mma(dt, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1 : 0);
              tc_commit(empty + si);
              tc_commit(tfull + ti);
            }
            if (++si == C::kNST) { si = 0; ph ^= 1u; }
            if (++ti == C::kTST) { ti = 0; tp ^= 1u; }
          }
        }
        // every MMA this thread issued is complete before the memory is freed
        if constexpr (C::kPair) tc_commit_pair(mma_done); else tc_commit(mma_done);
        mbar_wait_landed(mma_done, 0, status);
      }
      __syncwarp();
    } else if (XQ) {
      // ================================================================ quantisation
      // kQW warps take cells in turn and fill their activation tile and scales:
      // four lanes for a token's group, 32 columns each, eight tokens at a time.
      // A warp's rows are copied kRaw of its cells ahead into shared memory, where
      // each thread reads back only what it copied itself.  (Every CTA quantises
      // the groups it needs for itself: at 16 tokens 4 KB of x beside a cell's
      // 16 KB of weights, and no kernel before this one.)
      grid_dep_wait();
      constexpr int kIt = NT / 8;  // passes of eight tokens
      const int me = warp < kEW0 ? warp - kSW : warp - kEW1 + 2, tok = lane >> 2, quarter = lane & 3;
      const uint16_t* x = reinterpret_cast<const uint16_t*>(p.x) + quarter * 32;
      uint8_t* raw = smem + C::kRawAt + me * (C::kRaw * kIt * 2048) + lane * 16;  // [kRaw][kIt][4 chunks][lane]
      // this warp's cells, one after the other
      struct Cells {
        Pieces pc;
        int kb;
        bool more;
        MOE_DEV Cells(const LinArgs& a, int first) : pc(a) {
          more = pc.next();
          kb = pc.k0;
          step(first);
        }
        MOE_DEV void step(int n) {
          kb += n;
          while (more && kb >= pc.k1) {
            const int past = kb - pc.k1;
            more = pc.next();
            kb = pc.k0 + past;
          }
        }
      };
      Cells at(p, me), ahead = at;
      uint32_t an = 0;
      auto copy = [&]() {
        if (ahead.more) {
          const int t0 = ahead.pc.col * p.chunk, ntok = toks(ahead.pc.col);
          uint8_t* to = raw + (an++ % C::kRaw) * (kIt * 2048);
#pragma unroll
          for (int i = 0; i < kIt; ++i) {
            const int t = 8 * i + tok;
            if (8 * i < ntok) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                // past the last token or column: zeros, nothing is read
                const bool ok = t < ntok && ahead.kb * kBlock + quarter * 32 + 8 * j < p.K;
                const uint16_t* from = ok ? x + (long long)(t0 + t) * p.ldx + ahead.kb * kBlock + 8 * j : x;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(su32(to + i * 2048 + j * 512)),
                             "l"(from), "r"(ok ? 16 : 0)
                             : "memory");
              }
            }
          }
          ahead.step(C::kQW);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      for (int i = 0; i < C::kRaw - 1; ++i) copy();
      for (uint32_t n = me, mine = 0; at.more; n += C::kQW, ++mine) {
        const int ntok = toks(at.pc.col);
        copy();
        asm volatile("cp.async.wait_group %0;" ::"n"(C::kRaw - 1) : "memory");
        const uint8_t* from = raw + (mine % C::kRaw) * (kIt * 2048);
        const uint32_t si = n % C::kNST, xi = n % C::kXST;
        uint8_t* xt = ring + (size_t)si * C::kStage + kRTile;
        uint4 code[kIt][2];
        float s[kIt];
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
          if (8 * i < ntok) {  // the same in the warp
            uint4 v[4];
            float amax = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[j] = *reinterpret_cast<const uint4*>(from + i * 2048 + j * 512);
              amax = fmaxf(amax, amax8(v[j]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            s[i] = group_scale(amax, p.e8m0 != 0);
            const Quotient q(s[i]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint2 c0 = codes8(q, v[2 * j]), c1 = codes8(q, v[2 * j + 1]);
              code[i][j] = make_uint4(c0.x, c0.y, c1.x, c1.y);
            }
          }
        }
        if (!mbar_wait_landed(empty + si, ((n / C::kNST) & 1u) ^ 1u, status) ||
            !mbar_wait_landed(sempty + xi, ((n / C::kXST) & 1u) ^ 1u, status))
          break;
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
          const int t = 8 * i + tok;  // (a column past the last token is not read back)
          if (8 * i < ntok) {
#pragma unroll
            for (int j = 0; j < 2; ++j)  // 16-byte chunk 2 quarter + j of row t, swizzled as TMA would
              *reinterpret_cast<uint4*>(xt + t * 128 + (((2 * quarter + j) ^ (t & 7)) << 4)) = code[i][j];
            if (quarter == 0) xring[xi * C::kToks + t] = s[i];
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the tile is read by the MMA
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(full + si);
          mbar_arrive(sfull + xi);
        }
        at.step(C::kQW);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == kSW) {
      // ================================================================ token scales
      // A cell's xs run, copied up to kXST cells ahead of its epilogue (its own
      // ring: it is held until the epilogue is done with the cell).
      if (elect_one()) {
        grid_dep_wait();
        asm volatile("fence.proxy.async.global;" ::: "memory");
        uint32_t n = 0;
        bool alive = true;
        while (alive && pc.next()) {
          const int t = TR ? pc.row : pc.col;
          const int ntok = toks(t);  // (a pair's second CTA may have none)
          const uint32_t bytes = ntok > 0 ? (uint32_t)((ntok + 3) & ~3) * 4u : 0u;
          for (int kb = pc.k0; kb < pc.k1; ++kb, ++n) {
            const uint32_t xi = n % C::kXST;
            if (!mbar_wait_landed(sempty + xi, ((n / C::kXST) & 1u) ^ 1u, status)) { alive = false; break; }
            mbar_expect_tx(sfull + xi, bytes);
            if (bytes) bulk_load(xring + xi * C::kToks, p.xs + (size_t)kb * p.mp + t * p.chunk, bytes, sfull + xi);
          }
        }
        for (uint32_t j = (n > (uint32_t)C::kXST ? n - C::kXST : 0); j < n; ++j)
          mbar_wait_landed(sfull + j % C::kXST, (j / C::kXST) & 1u, status);
      }
      __syncwarp();
    }
  } else {
    // ================================================================ epilogue
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    grid_dep_wait();
    const int qd = warp & 3, hf = (warp - kEW0) >> 2;
    const int r = 32 * qd + lane;                 // row of the row tile
    const int col0 = hf * C::kHalf;
    constexpr int kStep = TR ? 32 : C::kHalf < 16 ? C::kHalf : 16;   // columns of one read of the accumulator
    float acc[C::kHalf];
    int ti = 0;
    uint32_t tp = 0, nc = 0;  // nc: cells so far
    bool alive = true;
    while (alive && pc.next()) {
      const int ncol = cols(pc.col) - col0;       // live columns of this warp (may be none)
      // weight scales: lane i holds k-block i of a run of 32, the next run is
      // read ahead; this warp's columns (TR) or the rows are one weight block
      const int wblk = min(TR ? pc.col * (NT / kBlock) + hf : pc.row, p.n_wblk - 1);
      const float* wr = p.w_s + (size_t)wblk * p.nkb;
      float ws = pc.k0 + lane < pc.k1 ? __ldcg(wr + pc.k0 + lane) : 0.f, wn = 0.f;
      const bool whole = pc.k0 == 0 && pc.k1 == p.nkb;
#pragma unroll
      for (int j = 0; j < C::kHalf; ++j) acc[j] = 0.f;
      for (int kb = pc.k0; kb < pc.k1; ++kb, ++nc) {
        const int off = (kb - pc.k0) & 31;
        if (off == 0) {
          if (kb != pc.k0) ws = wn;
          wn = kb + 32 + lane < pc.k1 ? __ldcg(wr + kb + 32 + lane) : 0.f;
        }
        const float w = __shfl_sync(0xffffffffu, ws, off);
        const uint32_t xi = nc % C::kXST;
        const float* xs = xring + xi * C::kToks;
        if (!mbar_wait_landed(sfull + xi, (nc / C::kXST) & 1u, status)) { alive = false; break; }
        const float s = TR ? w * xs[r] : 0.f;
        if (!mbar_wait_landed(tfull + ti, tp, status)) { alive = false; break; }
        tc_fence_after();
        const uint32_t ta = tmem + ((uint32_t)(32 * qd) << 16) + (uint32_t)(ti * NT + col0);
        if constexpr (TR) {
          // two reads of 32 columns in flight
          float d[2][32];
          tc_ld32(ta, d[0]);
#pragma unroll
          for (int j0 = 0; j0 < C::kHalf; j0 += kStep) {
            const int k = (j0 / kStep) & 1;
            tc_wait_ld();
            if (j0 + kStep < C::kHalf) tc_ld32(ta + j0 + kStep, d[k ^ 1]);
#pragma unroll
            for (int j = 0; j < kStep; j += 2) fma2(acc[j0 + j], acc[j0 + j + 1], d[k][j], d[k][j + 1], s, s);
          }
        } else {
#pragma unroll
          for (int j0 = 0; j0 < C::kHalf; j0 += kStep) {
            if (j0 < ncol) {
              float d[kStep];
              if constexpr (kStep == 16) tc_ld16(ta + j0, d); else tc_ld8(ta + j0, d);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < kStep; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(xs + col0 + j0 + j);
                fma2(acc[j0 + j], acc[j0 + j + 1], d[j], d[j + 1], f.x * w, f.y * w);
                fma2(acc[j0 + j + 2], acc[j0 + j + 3], d[j + 2], d[j + 3], f.z * w, f.w * w);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (C::kPair) mbar_arrive_at(mapa(su32(tempty + ti), 0)); else mbar_arrive(tempty + ti);
          mbar_arrive(sempty + xi);
        }
        if (++ti == C::kTST) { ti = 0; tp ^= 1u; }
      }
      if (!alive) break;
      if (!whole) {
        // this piece's sums go to the workspace; the last CTA of the pair to
        // arrive adds all pieces in k order.  The counter's release and acquire
        // reach the other warps through the barriers.
        const int c_first = p.piece[pc.cta()].first, c_last = c_first + p.pieces - 1;
        float* part = p.partials + (size_t)blockIdx.x * NT * kRows;
#pragma unroll
        for (int j = 0; j < C::kHalf; j += 4)
          if (j < ncol)
            __stcg(reinterpret_cast<float4*>(part) + (size_t)(col0 + j) / 4 * kRows + r,
                   make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]));
        __syncwarp();
        if (lane == 0) mbar_arrive(pdone);
        if (!mbar_wait_landed(pdone, 0, status)) break;
        if (tid == kEW0 * 32) {
          int* ticket = p.tickets + (C::kPair ? 2 * c_first + rank : c_first);
          const int got = atom_add_acq_rel(ticket, 1);
          const bool last = got == c_last - c_first;
          if (last) *ticket = 0;  // ready for the next call
          s_misc[1] = last;
          mbar_arrive(pdec);
        }
        if (!mbar_wait_landed(pdec, 0, status)) break;
        if (!s_misc[1]) continue;
#pragma unroll
        for (int j = 0; j < C::kHalf; ++j) acc[j] = 0.f;
        // up to 16 reads of 16 bytes in flight
        constexpr int kJ = C::kHalf < 64 ? C::kHalf : 64, kC = 64 / kJ;
        for (int c0 = c_first; c0 <= c_last; c0 += kC) {
#pragma unroll
          for (int j0 = 0; j0 < C::kHalf; j0 += kJ) {
            float4 v[kC][kJ / 4];
#pragma unroll
            for (int i = 0; i < kC; ++i) {
              const int c = min(c0 + i, c_last);
              const float4* ps = reinterpret_cast<const float4*>(
                  p.partials + (size_t)(C::kPair ? 2 * c + rank : c) * NT * kRows);
#pragma unroll
              for (int j = 0; j < kJ; j += 4)
                v[i][j / 4] = j0 + j < ncol ? __ldcg(ps + (size_t)(col0 + j0 + j) / 4 * kRows + r)
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < kC; ++i)
              if (c0 + i <= c_last)
#pragma unroll
                for (int j = 0; j < kJ; j += 4) {
                  acc[j0 + j] += v[i][j / 4].x;
                  acc[j0 + j + 1] += v[i][j / 4].y;
                  acc[j0 + j + 2] += v[i][j / 4].z;
                  acc[j0 + j + 3] += v[i][j / 4].w;
                }
          }
        }
      }
      if constexpr (TR) {
        // A lane holds a row: written from there, every store would touch 32
        // rows.  So 64 bytes of each row are turned through shared memory, and a
        // row's bytes written by neighbouring lanes, as wide as the rows' alignment
        // allows (4096 x 7168 -> 9216 248 -> 233 us; 510 x 176 -> 5934, whose rows
        // hold no 16-byte pieces, 46.1 -> 8.5).
        const int m0 = pc.row * kRows + 32 * qd, n0 = pc.col * NT + col0;
        uint8_t* turn = smem + C::kTurnAt + (size_t)(warp - kEW0) * 32 * kTurnRow;
        const int rows = min(32, p.M - m0);
        if (p.out_fp32) {
          store_turned<4, C::kHalf>(p, turn, acc, lane, m0, n0, rows, ncol);
        } else {
          store_turned<2, C::kHalf>(p, turn, acc, lane, m0, n0, rows, ncol);
        }
      } else {
        const int n = pc.row * kRows + r;
        if (n < p.N) {
#pragma unroll
          for (int j = 0; j < C::kHalf; ++j)
            if (j < ncol) store_out(p, pc.col * p.chunk + col0 + j, n, acc[j]);
        }
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  if constexpr (C::kPair) cluster_sync(); else __syncthreads();
  if (warp == kMW) {
    tc_fence_after();
    if constexpr (C::kPair)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTCols) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTCols) : "memory");
  }
}

template <int NT, bool TR, bool XQ>
cudaError_t launch_nt(const LinPlan& p, const LinArgs& a, const LinMaps& maps, cudaStream_t s) {
  using C = Cfg<NT, TR, XQ>;
  static OncePerDevice once;
  if (const cudaError_t rc = allow_smem(once, linear_kernel<NT, TR, XQ>, C::kSmem); rc != cudaSuccess) return rc;
  PdlLaunch L(dim3(C::kPair ? 2 * p.G : p.G), dim3(C::kThreads), C::kSmem, s);
  cudaLaunchAttribute attr[2] = {L.attr[0], {}};
  if (C::kPair) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    L.cfg.attrs = attr;
    L.cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&L.cfg, linear_kernel<NT, TR, XQ>, a, maps);
}

}  // namespace

// Up to 128 tokens: the tokens are the columns, at the smallest width that holds
// them.  Above: token tiles of 256 rows (128 a CTA), weight tiles of 256 columns
// (tiles of 128 tokens as columns instead, us: 4096 x 7168 -> 9216 495 for 230, 256 x
// 7168 -> 9216 36.5 for 30.4, 343 x 1392 -> 4957 12.5 for 12.9, 388 x 336 -> 3465 7.5
// for 9.4: only launches of a few cells lose).
void plan_linear(LinPlan& p, int M, int N, int K, int sms) {
  p.M = M; p.N = N; p.K = K;
  p.nkb = (K + kBlock - 1) / kBlock;
  p.tok_rows = M > 128;
  p.nt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
  p.chunk = std::min(p.nt, kRows);
  p.n_tt = p.tok_rows ? (M + 2 * kRows - 1) / (2 * kRows) : (M + p.chunk - 1) / p.chunk;
  p.n_wt = p.tok_rows ? (N + 255) / 256 : (N + kRows - 1) / kRows;
  const long long pairs = (long long)p.n_tt * p.n_wt;
  const int ctas = std::min(sms, kLinMaxCtas);
  p.G = p.tok_rows ? std::max(1, ctas / 2) : ctas;
  p.waves = (int)(pairs / p.G);
  p.rest = (int)(pairs - (long long)p.waves * p.G);
  // Pieces of each remaining pair: as many as make the last CTA end earliest.  In
  // units of the time a cell takes (0.25 us), / 128: the longest piece's cells,
  // and for the exchange of sums a fixed part, one that grows with a CTA's
  // sums, and (weights as rows) one with the CTAs that exchange at a time.
  // Measured over 1 .. 64 pieces (M x K -> N): us whole / with the best number / as
  // chosen: 1 x 4720 -> 354 11.6 / 5.5 / 5.5, 22 x 1408 -> 2763 7.1 / 7.1 / 7.0,
  // 96 x 6880 -> 844 29.3 / 13.6 / 14.1, 145 x 4032 -> 186 18.9 / 15.0 / 16.3,
  // 1908 x 6320 -> 117 35.8 / 27.6 / 28.3, 482 x 2144 -> 651 14.7 / 14.7 / 15.3.
  // Equal shares of all remaining cells for every CTA, whose pieces cross from one
  // pair into the next, were slower throughout (two pieces to exchange a CTA:
  // 1 x 7168 -> 9216 16.0 us for 14.5, 256 x 7168 -> 9216 32.6 for 27.6).
  p.pieces = 1;
  long long best = 128LL * p.nkb;
  for (int s = 2; p.rest > 0 && s <= p.nkb && (long long)s * p.rest <= p.G; ++s) {
    const long long exchange = p.tok_rows ? 640 + s * (576LL * std::min(N, 256) / 256) : 512 + s * (8LL * p.rest + p.nt);
    const long long cost = 128LL * ((p.nkb + s - 1) / s) + exchange;
    if (cost < best) { best = cost; p.pieces = s; }
  }
  if (p.waves == 0) p.G = p.rest * p.pieces;
}

cudaError_t launch_quant_rows(const QuantArgs& a, int sms, cudaStream_t s) {
  if (a.M == 0) return cudaSuccess;
  const int units = a.M * ((a.nkb + 7) / 8), per = kQuantThreads / 32;
  PdlLaunch L(dim3((unsigned)std::min((units + per - 1) / per, sms * 8)), dim3(kQuantThreads), 0, s);
  return cudaLaunchKernelEx(&L.cfg, quant_rows_kernel, a);
}

cudaError_t launch_linear(const LinPlan& p, LinArgs a, const uint8_t* xq, const uint8_t* w, cudaStream_t s) {
  LinMaps maps;
  const bool fused = a.x != nullptr;
  if (!tmap_2d(&maps.w, w, p.K, p.N, 128, kRows)) return cudaErrorInvalidValue;
  if (fused)
    maps.x = maps.w;  // (not used)
  else if (!tmap_2d(&maps.x, xq, p.K, p.M, 128, p.tok_rows ? kRows : std::min(p.nt, 32)))
    return cudaErrorInvalidValue;
  a.mp = linear_scale_stride(p.M);
  a.M = p.M; a.N = p.N; a.K = p.K; a.nkb = p.nkb; a.chunk = p.chunk; a.n_wt = p.n_wt;
  a.n_wblk = (p.N + kBlock - 1) / kBlock;
  a.tok_rows = p.tok_rows; a.G = p.G; a.waves = p.waves; a.pieces = p.pieces;
  for (int c = 0; c < p.G; ++c) {
    const int r = c / p.pieces, i = c - r * p.pieces;
    const long long pair = (long long)p.waves * p.G + r;
    if (r >= p.rest) { a.piece[c] = {}; continue; }
    a.piece[c] = {(uint16_t)(pair % p.n_wt), (uint16_t)(pair / p.n_wt), (uint16_t)(p.nkb * i / p.pieces),
                  (uint16_t)(p.nkb * (i + 1) / p.pieces), (uint16_t)(r * p.pieces)};
  }
  if (fused) return launch_nt<16, false, true>(p, a, maps, s);
  switch (p.nt) {
    case 16: return launch_nt<16, false, false>(p, a, maps, s);
    case 32: return launch_nt<32, false, false>(p, a, maps, s);
    case 64: return launch_nt<64, false, false>(p, a, maps, s);
    case 128: return launch_nt<128, false, false>(p, a, maps, s);
    default: return launch_nt<256, true, false>(p, a, maps, s);
  }
}

}  // namespace moe
