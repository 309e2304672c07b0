// Attention of a step's tokens over the FP8 paged cache (grouped query heads):
// for row r = (token i of sequence b, query head h) at position
// pos = len_b - n_b + i, over the cached tokens j <= pos (and j > pos - window):
//   s_j = sm_scale * q_r . (k_j * ks_page(j)),  s_j = cap * tanh(s_j / cap),
//   s_j += slope_h * (j - pos);
//   out_r = sum_j exp(s_j) * v_j * vs_page(j) / sum_j exp(s_j),
//   lse_r = log sum_j exp(s_j).
// A row that sees no token gives zeros and -inf.
//
// What bounds it: each cached byte is read once for the 8 or 16 rows that share
// the head, far below the tensor cores' balance, so the cache stream from HBM
// is the floor.  One pass with the running maximum and sum of the softmax.
//
// Work split.  The unit is a tile of 64 tokens of one item (sequence, kv head,
// group of up to 8 RT rows).  Every CTA (one per SM) adds up the sequences' tile
// counts for itself and takes an equal share of all tiles, whatever the
// lengths, so one long sequence fills the GPU like a batch of short ones.  An
// item that spans CTAs is joined through the workspace by the last CTA to
// arrive, in order of position.
//
// Inside a CTA a producer warp copies pages (TMA, 128- or 64-byte swizzle) into a
// ring of tiles and seven consumer warps take tiles in turn, each with its own
// maximum, sum and accumulator; they join at the end of an item.
//
// Arithmetic of a tile.
//   S = Q K^T on mma m16n8k32 (E4M3): K goes to the tensor core as it is
//   stored.  Each row of Q, scaled to a maximum in [128, 256), is the sum of an
//   E4M3 part and a second E4M3 part of 1/16 the size: a bf16 value has 8
//   significant bits and each part carries 4, so the split is exact for values
//   within 2^-14 of the row's largest and off by at most 2^-22 of it below.  The two
//   parts are the upper and lower 8 of the MMA's 16 rows, so no row is wasted
//   and their sum is an addition within a thread.
//   O^T = V^T P^T on mma m16n8k16 (f16): the S accumulator is the B operand as it
//   lies in registers; V's codes are paired over two tokens with byte permutes
//   and converted to f16 (exact).  P is rounded to f16 (11 bits, 2^-12 of its
//   value), scaled by 2^15 and by its page's scale over the largest seen, so
//   that it stays a normal number down to 2^-29 of the largest weight; sums
//   and statistics are fp32, and the sum of the weights takes them unrounded.
// The token order inside a tile's fragments is chosen so that both operands
// come from shared memory in 16-byte loads without bank conflicts (D = 128):
// column n of S's 8-token tile t is token 8 t + 4 (n & 1) + (n >> 1).
#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "async.cuh"
#include "common.cuh"
#include "kernels.h"
#include "tmap.h"
#include "../../include/moe_decode.h"

namespace moe {

namespace {

constexpr int kTile = 64;                 // tokens of a tile
constexpr int kWarps = 7;                 // consumer warps (with the producer two a scheduler: up to 255 registers)
constexpr int kThreads = (kWarps + 1) * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPScale = 32768.f;        // weights are rounded to f16 in units of 2^-15

// Per tile: the scales of its four 16-token groups and which of them were loaded.
struct TileMeta {
  float ks[4], vs[4];
  int mask;
  int pad[3];
};

template <int D, int RT>
struct AttCfg {
  static constexpr int kRowsC = 8 * RT;                    // rows of an item
  static constexpr int kHalfTile = kTile * D;              // bytes of the K (or V) part of a tile
  static constexpr int kStage = 2 * kHalfTile;
  static constexpr int kRed = kWarps * kRowsC * D * 4;     // the warps' accumulators at the end of an item
  static constexpr int kNST = std::min(24, (220 * 1024 - kRed) / kStage);
  static constexpr size_t kRedAt = (size_t)kNST * kStage;
  static constexpr size_t kStatAt = kRedAt + kRed;         // [warp][row] maximum and sum, [warp] largest V scale
  static constexpr size_t kMetaAt = kStatAt + (size_t)kWarps * (2 * kRowsC + 4) * 4;
  static constexpr size_t kBarsAt = kMetaAt + (size_t)kNST * sizeof(TileMeta);
  static constexpr size_t kMiscAt = kBarsAt + (2 * kNST + 2) * 8;
  static constexpr size_t kSmem = 1024 + kMiscAt + 64 + 40;
};

struct AttMaps {
  CUtensorMap k, v;
};

MOE_DEV void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
MOE_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two E4M3 pairs (the lower and the upper half of w) to two f16 pairs
MOE_DEV void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
      : "=r"(lo), "=r"(hi) : "r"(w));
}
MOE_DEV float2 e4m3x2_to_f32x2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
MOE_DEV uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
// 16-byte chunk c of token row t of a tile of D-byte rows, as TMA swizzles it
template <int D>
MOE_DEV uint32_t chunk_at(uint32_t base, int t, int c) {
  if constexpr (D == 128) return base + t * 128 + ((c ^ (t & 7)) << 4);
  return base + t * 64 + ((c ^ ((t >> 1) & 3)) << 4);
}

// What a sequence asks for, from the device-side lengths; the same in every
// CTA.  Lengths out of range count as an empty sequence and are reported.
struct Seq {
  int start, n, len, tile0, tiles, groups;  // groups: row groups
};
template <int RT>
MOE_DEV Seq load_seq(const AttArgs& a, int b, bool report) {
  Seq s;
  s.start = __ldg(a.q_start + b);
  s.n = __ldg(a.q_start + b + 1) - s.start;
  s.len = __ldg(a.lens + b);
  const long long cap = (long long)a.width * a.page_size;
  bool bad = false;
  if (s.start < 0 || s.n < 0 || s.start > a.total || s.n > a.total - s.start) { s.n = 0; s.start = 0; bad = true; }
  if (s.len < 0 || s.len > cap) { s.len = 0; bad = true; }
  if (bad && report) atomicExch(a.status, MOE_ERR_INVALID_ARG);
  // the first token any row sees (the first row's window), then whole tiles
  const int lo = a.window > 0 ? max(0, s.len - s.n + 1 - a.window) : 0;
  s.tile0 = lo / kTile;
  s.tiles = max(1, (s.len + kTile - 1) / kTile - s.tile0);
  s.groups = (int)(((long long)s.n * a.G + 8 * RT - 1) / (8 * RT));
  return s;
}

// The pieces of a CTA: tiles [t0, t1) of an item (b, head, group).
struct Walk {
  long long left;      // tiles this CTA still has to hand out
  int b, head, grp;
  int t0, t1;
  long long item0;     // first tile of the item, counted over all items
  Seq s;
};
template <int RT>
MOE_DEV void walk_start(Walk& w, const AttArgs& a, int b, long long b_first, long long x, long long count) {
  w.left = count;
  w.b = b;
  if (count <= 0) return;
  w.s = load_seq<RT>(a, b, false);
  const long long it = (x - b_first) / w.s.tiles;
  w.head = (int)(it / w.s.groups);
  w.grp = (int)(it % w.s.groups);
  w.item0 = b_first + it * w.s.tiles;
  w.t0 = (int)(x - w.item0);
  w.t1 = (int)min((long long)w.s.tiles, w.t0 + count);
}
template <int RT>
MOE_DEV bool walk_next(Walk& w, const AttArgs& a) {  // to the next piece
  w.left -= w.t1 - w.t0;
  if (w.left <= 0) return false;
  w.item0 += w.s.tiles;
  if (++w.grp == w.s.groups) {
    w.grp = 0;
    if (++w.head == a.kv_heads) {
      w.head = 0;
      do {
        ++w.b;
        w.s = load_seq<RT>(a, w.b, false);
      } while (w.s.groups == 0);  // (a sequence without rows has no tiles; left > 0: one with rows follows)
    }
  }
  w.t0 = 0;
  w.t1 = (int)min((long long)w.s.tiles, w.left);
  return true;
}

// Four columns of a finished row, and (first column) its log-sum-exp.
MOE_DEV void att_store(const AttArgs& a, int start, int row, int head, int D, int d, float4 acc, float M, float L) {
  const size_t tok = (size_t)(start + row / a.G);
  const int hq = head * a.G + row % a.G;
  const float inv = L == 0.f ? 0.f : __fdiv_rn(1.f, L);
  uint2 v;
  v.x = pack_bf16(acc.x * inv, acc.y * inv);
  v.y = pack_bf16(acc.z * inv, acc.w * inv);
  const size_t hi = tok * (size_t)(a.G * a.kv_heads) + hq;
  *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + hi * D + d) = v;
  if (a.lse && d == 0) a.lse[hi] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

template <int D, int RT, bool MODS>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(AttArgs a, const __grid_constant__ AttMaps maps) {
  using C = AttCfg<D, RT>;
  constexpr int kRowsC = C::kRowsC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (su32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* ring = smem;
  float* red = reinterpret_cast<float*>(smem + C::kRedAt);       // [warp][row][D]
  float* stat = reinterpret_cast<float*>(smem + C::kStatAt);     // [warp][2][row], then [warp] at kWarps * 2 * rows
  TileMeta* meta = reinterpret_cast<TileMeta*>(smem + C::kMetaAt);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarsAt);
  uint64_t* empty = full + C::kNST;
  uint64_t* join = empty + C::kNST;   // the consumer warps' meeting point
  long long* s_ll = reinterpret_cast<long long*>(smem + C::kMiscAt);  // [0] total [1] first tile of b, then ints
  volatile int* s_i = reinterpret_cast<volatile int*>(s_ll + 2);      // [0] b, [1] last to arrive
  int* status = a.status;

  if (tid == 0) {
    for (int i = 0; i < C::kNST; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    mbar_init(join, kWarps);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }

  // ---- this CTA's share: every thread adds up a run of sequences, then a scan
  __shared__ long long s_scan[kWarps + 1];
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Seq s = load_seq<RT>(a, b, blockIdx.x == 0);
    mine += (long long)s.tiles * s.groups * a.kv_heads;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps + 1; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const int G = (int)min((long long)gridDim.x, total);  // CTAs that get work: a tile each at least
  if ((int)blockIdx.x >= G) return;                       // (the whole CTA; nothing is in flight)
  const long long x0 = total * blockIdx.x / G, x1 = total * (blockIdx.x + 1) / G;
  if (x0 >= before && x0 < before + mine) {  // one thread
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const Seq s = load_seq<RT>(a, b, false);
      const long long nb = (long long)s.tiles * s.groups * a.kv_heads;
      if (x0 < at + nb) {
        s_ll[1] = at;
        s_i[0] = b;
        break;
      }
      at += nb;
    }
  }
  __syncthreads();
  Walk w;
  walk_start<RT>(w, a, s_i[0], s_ll[1], x0, x1 - x0);
  const int P = a.page_size;
  const int box = min(P, kTile);          // token rows of one copy
  const int nbox = kTile / box;

  if (warp == kWarps) {
    // ================================================================ producer
    // Eight tiles' pages and scales at a time: lane 4 t + g looks up 16-token
    // group g of tile t, so the two dependent reads are paid once for eight tiles.
    uint32_t n = 0;
    int si = 0;
    uint32_t ph = 0;
    bool alive = true;
    do {
      const int lo = a.window > 0 ? max(0, w.s.len - w.s.n + 1 - a.window) : 0;
      for (int tb = w.t0; tb < w.t1 && alive; tb += 8) {
        const int tl = tb + (lane >> 2);
        const int pos = (w.s.tile0 + tl) * kTile + 16 * (lane & 3);
        bool ok = tl < w.t1 && pos < w.s.len && pos + 16 > lo;
        int page = 0;
        float ks = 0.f, vs = 0.f;
        if (ok) {
          page = __ldg(a.page_table + (size_t)w.b * a.width + pos / P);
          if (page < 0 || page >= a.num_pages) {  // its tokens are masked
            atomicExch(status, MOE_ERR_INVALID_ARG);
            ok = false;
          } else {
            ks = __ldg(a.k_scale + (size_t)page * a.kv_heads + w.head);
            vs = __ldg(a.v_scale + (size_t)page * a.kv_heads + w.head);
          }
        }
        const uint32_t okm = __ballot_sync(0xffffffffu, ok);
        for (int t = 0; t < 8 && tb + t < w.t1; ++t) {
          const int m4 = (okm >> (4 * t)) & 15;
          // box i holds groups i * box / 16 ...; it is copied if any of them is wanted
          const int gpb = box >> 4;
          int boxes = 0;
          for (int i = 0; i < nbox; ++i) boxes += ((m4 >> (i * gpb)) & ((1 << gpb) - 1)) != 0;
          bool go = true;
          if (n >= (uint32_t)C::kNST) {
            if (lane == 0) go = mbar_wait_landed(empty + si, ph ^ 1u, status);
            go = __shfl_sync(0xffffffffu, go, 0);
          }
          if (!go) { alive = false; break; }
          if ((lane >> 2) == t) {
            meta[si].ks[lane & 3] = ks;
            meta[si].vs[lane & 3] = vs;
            if ((lane & 3) == 0) meta[si].mask = m4;
          }
          __syncwarp();
          if (lane == 0) mbar_expect_tx(full + si, (uint32_t)(boxes * 2 * box * D));
          __syncwarp();
          // lanes 0 .. nbox - 1 copy K boxes, the next nbox V boxes
          const int i = lane % nbox;
          const int src = 4 * t + __ffs((m4 >> (i * gpb)) & ((1 << gpb) - 1)) - 1 + i * gpb;
          const int pg = __shfl_sync(0xffffffffu, page, src & 31);
          if (lane < 2 * nbox && ((m4 >> (i * gpb)) & ((1 << gpb) - 1)) != 0) {
            const int at = (w.s.tile0 + tb + t) * kTile % P;  // first row inside the page (0 unless a page holds several tiles)
            uint8_t* dst = ring + (size_t)si * C::kStage + (lane < nbox ? 0 : C::kHalfTile) + i * box * D;
            tma_load_3d(dst, lane < nbox ? &maps.k : &maps.v, 0, at, pg * a.kv_heads + w.head, full + si);
          }
          __syncwarp();
          ++n;
          if (++si == C::kNST) { si = 0; ph ^= 1u; }
        }
      }
    } while (alive && walk_next<RT>(w, a));
    // every copy this CTA issued lands before it ends
    if (lane == 0)
      for (uint32_t j = (n > (uint32_t)C::kNST ? n - C::kNST : 0); j < n; ++j)
        mbar_wait_landed(full + (j % C::kNST), (j / C::kNST) & 1u, status);
    __syncwarp();
    return;
  }

  // ================================================================ consumers
  const int g = lane >> 2, q = lane & 3;
  const int fg = D == 128 ? ((g & 1) << 2 | g >> 1) : g;   // this thread's chunk of a V row (16 or 8 values)
  constexpr int kMT = D / 16;                              // 16-row tiles of V^T
  uint32_t jn = 0;                                         // meetings so far
  auto meet = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(join);
    return mbar_wait_landed(join, jn++ & 1u, status);
  };
  uint32_t n0 = 0;  // tiles of the pieces before this one
  bool alive = true;
  do {
    const int rows = min(kRowsC, w.s.n * a.G - w.grp * kRowsC);
    const int pos0 = w.s.len - w.s.n;  // position of the step's first token
    // ---- Q fragments: rows g of each row tile, upper part in a0 / a2, lower in a1 / a3
    uint32_t qf[RT][D / 32][4];
    float qs[RT];      // 1 / (row's scale), times the softmax scale
    int pos_r[RT];
    float slope[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int r = w.grp * kRowsC + rt * 8 + g;
      const bool live = rt * 8 + g < rows;
      const int i = live ? r / a.G : 0, hq = w.head * a.G + (live ? r % a.G : 0);
      pos_r[rt] = live ? pos0 + i : -1;
      slope[rt] = 0.f;
      if (MODS && a.slopes && live) slope[rt] = __ldg(a.slopes + hq) * kLog2e;
      const uint16_t* qp = reinterpret_cast<const uint16_t*>(a.q) + (long long)(w.s.start + i) * a.q_stride + hq * D;
      uint4 v[D / 64][2];
      float amax = 0.f;
      bool odd = false;
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          v[h][e] = live ? __ldg(reinterpret_cast<const uint4*>(qp + 64 * h + 16 * q + 8 * e)) : make_uint4(0, 0, 0, 0);
          const uint32_t x[4] = {v[h][e].x, v[h][e].y, v[h][e].z, v[h][e].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float f0 = fabsf(bf16_lo(x[k])), f1 = fabsf(bf16_hi(x[k]));
            odd |= !(f0 <= 3.4028235e38f) || !(f1 <= 3.4028235e38f);
            amax = fmaxf(amax, fmaxf(f0, f1));
          }
        }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const uint32_t any_odd = __ballot_sync(0xffffffffu, odd);
      // scale 2^(7 - exponent): the row's maximum lands in [128, 256); tiny rows
      // keep the largest scale a float can be divided by
      const int ex = max(1, min(253, 261 - (int)(__float_as_uint(amax) >> 23)));
      const float sc = __uint_as_float((uint32_t)ex << 23);
      qs[rt] = __uint_as_float((uint32_t)(254 - ex) << 23) * a.sm_scale;
      if (any_odd & (0xfu << (4 * g))) qs[rt] = __uint_as_float(0x7fc00000u);  // infinities and NaN make the row NaN
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t x[4] = {v[h][e].x, v[h][e].y, v[h][e].z, v[h][e].w};
          uint32_t up[2], low[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float f[4] = {bf16_lo(x[2 * k]) * sc, bf16_hi(x[2 * k]) * sc, bf16_lo(x[2 * k + 1]) * sc,
                                bf16_hi(x[2 * k + 1]) * sc};
            up[k] = f32x4_to_e4m3x4(f[0], f[1], f[2], f[3]);
            const float2 u0 = e4m3x2_to_f32x2((uint16_t)(up[k] & 0xffff)), u1 = e4m3x2_to_f32x2((uint16_t)(up[k] >> 16));
            low[k] = f32x4_to_e4m3x4((f[0] - u0.x) * 16.f, (f[1] - u0.y) * 16.f, (f[2] - u1.x) * 16.f,
                                     (f[3] - u1.y) * 16.f);
          }
          // 16 consecutive columns are 4 words: words 0, 1 in one MMA step, 2, 3 in the next
          qf[rt][2 * h + e][0] = up[0];
          qf[rt][2 * h + e][1] = low[0];
          qf[rt][2 * h + e][2] = up[1];
          qf[rt][2 * h + e][3] = low[1];
        }
    }
    float m[RT], l[RT], o[RT][kMT][4];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m[rt] = -INFINITY;
      l[rt] = 0.f;
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[rt][mt][i] = 0.f;
    }
    float R = 0.f;  // largest V scale so far: the accumulators' unit is R 2^-15
    // tokens every row sees lie in [lo_all, hi_all); tiles inside need no mask
    const int hi_all = pos0 + 1;
    const int lo_all = a.window > 0 ? max(0, w.s.len - a.window) : 0;
    const int lo_any = a.window > 0 ? max(0, pos0 + 1 - a.window) : 0;

    const int cnt = w.t1 - w.t0;
    for (int t = (int)((warp + kWarps - n0 % kWarps) % kWarps); t < cnt; t += kWarps) {
      const uint32_t sq = n0 + t;
      const int si = (int)(sq % C::kNST);
      if (!mbar_wait_landed(full + si, (sq / C::kNST) & 1u, status)) { alive = false; break; }
      const TileMeta& md = meta[si];
      const int mask = md.mask;
      const int base = (w.s.tile0 + w.t0 + t) * kTile;
      const bool part = mask != 15 || base + kTile > hi_all || base < lo_all;
      const uint32_t kt = su32(ring + (size_t)si * C::kStage), vt = kt + C::kHalfTile;

      // ---- scores: s[rt][2 j + i] is row g, token 16 (j / 2) + 8 (j % 2) + 4 i + q
      float s[RT][16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = 8 * j + 4 * (g & 1) + (g >> 1);
        float c[RT][4];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) c[rt][0] = c[rt][1] = c[rt][2] = c[rt][3] = 0.f;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const uint4 kv = lds128(chunk_at<D>(kt, row, 4 * h + q));
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const uint32_t(&f0)[4] = qf[rt][2 * h];
            const uint32_t(&f1)[4] = qf[rt][2 * h + 1];
            mma_e4m3(c[rt], f0[0], f0[1], f0[2], f0[3], kv.x, kv.y);
            mma_e4m3(c[rt], f1[0], f1[1], f1[2], f1[3], kv.z, kv.w);
          }
        }
        const float ks = md.ks[j >> 1];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const float f = qs[rt] * ks * (MODS ? 1.f : kLog2e);
          s[rt][2 * j] = fmaf(c[rt][2], 0.0625f, c[rt][0]) * f;
          s[rt][2 * j + 1] = fmaf(c[rt][3], 0.0625f, c[rt][1]) * f;
        }
      }
      if (MODS) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float x = s[rt][k];
            if (a.softcap > 0.f) x = a.softcap * tanhf(__fdividef(x, a.softcap));
            const int pos = base + 8 * (k >> 1) + 4 * (k & 1) + q;
            s[rt][k] = fmaf(slope[rt], (float)(pos - pos_r[rt]), x * kLog2e);
          }
      }
      if (part) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int pos = base + 8 * (k >> 1) + 4 * (k & 1) + q;
            const bool see = pos <= pos_r[rt] && (a.window <= 0 || pos > pos_r[rt] - a.window) && ((mask >> (k >> 2)) & 1);
            if (!see) s[rt][k] = -INFINITY;
          }
      }
      // ---- running maximum and sum
      float Rn = R;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((mask >> i) & 1) Rn = fmaxf(Rn, md.vs[i]);
      const float Rq = Rn > 0.f ? __fdividef(kPScale, Rn) : 0.f;
      const float rr = Rn == R ? 1.f : __fdividef(R, Rn);
      float al[RT];
      bool turn = Rn != R;
      uint32_t pb[RT][8];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float mx = s[rt][0];
#pragma unroll
        for (int k = 1; k < 16; ++k) mx = fmaxf(mx, s[rt][k]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[rt], mx);
        const float ms = mn == -INFINITY ? 0.f : mn;
        al[rt] = ex2(m[rt] - ms);
        turn |= mn > m[rt];
        m[rt] = mn;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float F = md.vs[j >> 1] * Rq;
          const float p0 = ex2(s[rt][2 * j] - ms), p1 = ex2(s[rt][2 * j + 1] - ms);
          sum += p0 + p1;
          // masked tokens of a group that was not loaded: vs is 0, p is 0
          const __half2 h2 = __floats2half2_rn(p0 * F, p1 * F);
          pb[rt][j] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        l[rt] = l[rt] * al[rt] + sum;
      }
      if (__any_sync(0xffffffffu, turn)) {
        R = Rn;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const float f = al[rt] * rr;  // of row g; the accumulator's columns are rows 2 q and 2 q + 1
          const float f0 = __shfl_sync(0xffffffffu, f, 8 * q), f1 = __shfl_sync(0xffffffffu, f, 8 * q + 4);
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            o[rt][mt][0] *= f0; o[rt][mt][2] *= f0;
            o[rt][mt][1] *= f1; o[rt][mt][3] *= f1;
          }
        }
      }
      // ---- O^T += V^T P^T, 16 tokens at a time
#pragma unroll
      for (int gr = 0; gr < 4; ++gr) {
        uint32_t v4[4][D / 32];  // tokens q, 4 + q, 8 + q, 12 + q of the group, this thread's chunk
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * gr + 4 * i + q;
          if constexpr (D == 128) {
            const uint4 x = lds128(chunk_at<D>(vt, row, fg));
            v4[i][0] = x.x; v4[i][1] = x.y; v4[i][2] = x.z; v4[i][3] = x.w;
          } else {
            const uint2 x = lds64(chunk_at<D>(vt, row, fg >> 1) + 8 * (fg & 1));
            v4[i][0] = x.x; v4[i][1] = x.y;
          }
          if (part) {
            // tokens no row sees may hold anything (an old page's codes, NaN)
            const int pos = base + row;
            if (pos >= w.s.len || pos < lo_any || !((mask >> gr) & 1)) {
#pragma unroll
              for (int k = 0; k < D / 32; ++k) v4[i][k] = 0;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
          e4m3x4_to_f16x4(__byte_perm(v4[0][k], v4[1][k], 0x5140), a0, a1);
          e4m3x4_to_f16x4(__byte_perm(v4[2][k], v4[3][k], 0x5140), a2, a3);
          e4m3x4_to_f16x4(__byte_perm(v4[0][k], v4[1][k], 0x7362), b0, b1);
          e4m3x4_to_f16x4(__byte_perm(v4[2][k], v4[3][k], 0x7362), b2, b3);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            mma_f16(o[rt][2 * k], a0, a1, a2, a3, pb[rt][2 * gr], pb[rt][2 * gr + 1]);
            mma_f16(o[rt][2 * k + 1], b0, b1, b2, b3, pb[rt][2 * gr], pb[rt][2 * gr + 1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + si);
    }
    if (!alive) break;
    n0 += cnt;

    // ---- the warps join: accumulators and statistics through shared memory
    if (jn > 0 && !meet()) break;  // the piece before has been read out
    {
      float* rw = red + (size_t)warp * kRowsC * D;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float sum = l[rt];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (q == 0) {
          stat[(warp * 2 + 0) * kRowsC + rt * 8 + g] = m[rt];
          stat[(warp * 2 + 1) * kRowsC + rt * 8 + g] = sum;
        }
        // columns 2 q, 2 q + 1 are rows; this thread's d are D / 8 consecutive ones from fg * D / 8
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int mt = 0; mt < kMT; mt += 2)
            *reinterpret_cast<float4*>(rw + (rt * 8 + 2 * q + c) * D + fg * (D / 8) + 2 * mt) =
                make_float4(o[rt][mt][c], o[rt][mt][2 + c], o[rt][mt + 1][c], o[rt][mt + 1][2 + c]);
      }
      if (lane == 0) stat[kWarps * 2 * kRowsC + warp] = R;
    }
    if (!meet()) break;
    const bool whole = w.t0 == 0 && w.t1 == w.s.tiles;
    constexpr int kVec = D / 4;  // float4 of a row
    const float* sR = stat + kWarps * 2 * kRowsC;
    for (int i = tid; i < kRowsC * kVec; i += kWarps * 32) {
      const int r = i / kVec, d = (i % kVec) * 4;
      if (r >= rows) continue;
      float M = -INFINITY;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) M = fmaxf(M, stat[(x * 2) * kRowsC + r]);
      const float ms = M == -INFINITY ? 0.f : M;
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float e = ex2(stat[(x * 2) * kRowsC + r] - ms);
        L += e * stat[(x * 2 + 1) * kRowsC + r];
        const float f = e * sR[x] * (1.f / kPScale);
        const float4 ov = *reinterpret_cast<const float4*>(red + ((size_t)x * kRowsC + r) * D + d);
        acc.x += ov.x * f; acc.y += ov.y * f; acc.z += ov.z * f; acc.w += ov.w * f;
      }
      if (whole) {
        att_store(a, w.s.start, w.grp * kRowsC + r, w.head, D, d, acc, M, L);
      } else {
        float* part = a.partials + ((size_t)blockIdx.x * 2 + (w.t0 == 0 ? 1 : 0)) * kRowsC * (D + 4);
        __stcg(reinterpret_cast<float4*>(part + (size_t)r * D + d), acc);
        if (d == 0) __stcg(reinterpret_cast<float2*>(part + (size_t)kRowsC * D + 2 * r), make_float2(M, L));
      }
    }
    if (!whole) {
      __threadfence();
      if (!meet()) break;
      // CTAs that hold a piece of this item
      const long long i0 = w.item0, i1 = w.item0 + w.s.tiles - 1;
      const int c_first = (int)(((i0 + 1) * G - 1) / total), c_last = (int)(((i1 + 1) * G - 1) / total);
      if (tid == 0) {
        __threadfence();
        const bool last = atom_add_acq_rel(a.tickets + c_first, 1) == c_last - c_first;
        if (last) a.tickets[c_first] = 0;  // ready for the next call
        s_i[1] = last;
      }
      if (!meet()) break;
      if (s_i[1]) {
        __threadfence();
        constexpr size_t kPart = (size_t)kRowsC * (D + 4);
        for (int i = tid; i < kRowsC * kVec; i += kWarps * 32) {
          const int r = i / kVec, d = (i % kVec) * 4;
          if (r >= rows) continue;
          float M = -INFINITY;
          for (int c = c_first; c <= c_last; ++c) {
            const float* part = a.partials + ((size_t)c * 2 + (c == c_first ? 1 : 0)) * kPart;
            M = fmaxf(M, __ldcg(part + (size_t)kRowsC * D + 2 * r));
          }
          const float ms = M == -INFINITY ? 0.f : M;
          float L = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int c = c_first; c <= c_last; ++c) {
            const float* part = a.partials + ((size_t)c * 2 + (c == c_first ? 1 : 0)) * kPart;
            const float2 st = __ldcg(reinterpret_cast<const float2*>(part + (size_t)kRowsC * D + 2 * r));
            const float4 ov = __ldcg(reinterpret_cast<const float4*>(part + (size_t)r * D + d));
            const float e = ex2(st.x - ms);
            L += e * st.y;
            acc.x += ov.x * e; acc.y += ov.y * e; acc.z += ov.z * e; acc.w += ov.w * e;
          }
          att_store(a, w.s.start, w.grp * kRowsC + r, w.head, D, d, acc, M, L);
        }
      }
    }
  } while (walk_next<RT>(w, a));
}

// K or V cache [num_pages * kv_heads][page_size][D] bytes; box = up to 64 rows of one page
bool map_cache(CUtensorMap* m, const uint8_t* base, int D, int P, long long tiles) {
  if (!encode_fn()) return false;
  const cuuint64_t dim[3] = {(cuuint64_t)D, (cuuint64_t)P, (cuuint64_t)tiles};
  const cuuint64_t stride[2] = {(cuuint64_t)D, (cuuint64_t)P * D};
  const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)std::min(P, kTile), 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(base), dim, stride, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int RT, bool MODS>
cudaError_t launch_cfg(const AttArgs& a, const AttMaps& maps, int ctas, cudaStream_t s) {
  using C = AttCfg<D, RT>;
  static const cudaError_t rc =
      cudaFuncSetAttribute(attention_kernel<D, RT, MODS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (rc != cudaSuccess) return rc;
  attention_kernel<D, RT, MODS><<<ctas, kThreads, C::kSmem, s>>>(a, maps);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const AttArgs& a, const AttMaps& maps, int ctas, cudaStream_t s) {
  const bool mods = a.softcap > 0.f || a.slopes;
  if (attention_row_tiles(a.G, a.max_new) == 1)
    return mods ? launch_cfg<D, 1, true>(a, maps, ctas, s) : launch_cfg<D, 1, false>(a, maps, ctas, s);
  return mods ? launch_cfg<D, 2, true>(a, maps, ctas, s) : launch_cfg<D, 2, false>(a, maps, ctas, s);
}

}  // namespace

// Rows that share one read of the cache: 8 where a sequence has no more, else 16.
int attention_row_tiles(int G, int max_new) { return (long long)G * max_new <= 8 ? 1 : 2; }

size_t attention_partial_bytes(int D, int G, int max_new) {
  return (size_t)kAttMaxCtas * 2 * 8 * attention_row_tiles(G, max_new) * (D + 4) * sizeof(float);
}

cudaError_t launch_attention(const AttArgs& a, int sms, cudaStream_t s) {
  if (a.B == 0 || a.total == 0) return cudaSuccess;
  AttMaps maps;
  const long long tiles = (long long)a.num_pages * a.kv_heads;
  if (!map_cache(&maps.k, a.k_cache, a.head_dim, a.page_size, tiles) ||
      !map_cache(&maps.v, a.v_cache, a.head_dim, a.page_size, tiles))
    return cudaErrorInvalidValue;
  const int ctas = std::min(sms, kAttMaxCtas);
  return a.head_dim == 64 ? launch_d<64>(a, maps, ctas, s) : launch_d<128>(a, maps, ctas, s);
}

}  // namespace moe
