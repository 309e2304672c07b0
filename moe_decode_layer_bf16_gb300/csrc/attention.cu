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
// Measured: 61 sequences of 300 to 16384 tokens, 526 MB, 87.9 us, 6.0 TB/s (0.88 of the
// copy rate); one of 131001 tokens 51.9 us, 5.2 TB/s; about 2 us until the lengths, the
// page numbers and the first tile are there, and 4 until the pieces are joined, are
// what short caches cost (777 tokens 9.3 us).
//
// Work split.  The unit is a tile of 32 tokens of one item (sequence, kv head,
// group of up to 8 RT rows); an item counts kItemCost tiles more for its start and
// end.  Every CTA (one per SM) adds up the sequences' units for itself and takes
// an equal share of all of them, and each of its warps (8, or 16 for heads of 64)
// an equal share of that, whatever the lengths: one long
// sequence fills the GPU like a batch of short ones.  (Only items of one or two
// tiles stay whole.)  A warp works alone: it
// looks up the pages, copies them (TMA, 128- or 64-byte swizzle) into its own ring
// of tiles, and keeps its own maximum, sum and accumulator.  An item inside one
// warp's share is finished by it; pieces are joined in order of position, once
// at the CTA's end through shared memory, and across CTAs through the workspace
// by the last CTA to arrive.
//
// Arithmetic of a tile.
//   S = Q K^T on mma m16n8k16 (f16): K's codes are converted to f16 (exact), and
//   each row of Q is scaled by a power of two to a maximum in [2^14, 2^15): exact
//   for values within 2^-31 of the row's largest and off by at most 2^-39 of it
//   below.  (With K as stored, on the E4M3 MMA, and Q as the sum of two E4M3 parts
//   in the upper and lower 8 rows, 4 tokens each of 16 sequences 37.5 us for 32.1,
//   1 x 99444 tokens with 128 heads on 8 63.7 for 51.9.)
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
#include <climits>

#include "async.cuh"
#include "common.cuh"
#include "kernels.h"
#include "step_rows.h"
#include "tcgen05.cuh"
#include "tmap.h"
#include "../../include/moe_decode.h"

namespace moe {

namespace {

// Units of an item beside its tiles: its start and end take a warp as long as two tiles (61
// sequences of 300 to 16384 tokens, us: 1 100.7, 2 87.9, 3 88.2, 4 89.2).
constexpr int kItemCost = 2;
// Items of so many tiles at most are not cut: a tile takes a warp 1.3 us, joining pieces
// 5 us (80 attention cases that perf/operators.py draws from random.Random(7), geometric
// mean in a graph: 0 10.99 us, 1 9.95, 2 9.88, 4 9.93, 8 10.50).
constexpr int kWholeTiles = 2;
// Where tiles as units come to more than 31 bits (a prompt of 93000 tokens, 128 heads on 8),
// a unit is 2^5 of them, or 2^10, ...: one unit more or less a warp is nothing there.
constexpr int kCoarser = 5, kCoarsest = 25;  // (2^25 tiles are the longest sequence)
static_assert((long long)kAttMaxItems * (kItemCost + 1) <= INT_MAX, "the coarsest units fit");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPScale = 32768.f;        // weights are rounded to f16 in units of 2^-15
// Where the largest V scale seen starts from: the smallest normal number, so that its
// reciprocal is finite.  (A block of zeros has this scale: 2^15 over it is not.)
constexpr float kMinUnit = 1.17549435e-38f;

// A piece of an item that a warp (or, in the workspace, a CTA) could not finish.
struct Piece {
  int item0;         // first unit of the item, -1: no piece
  int units;         // of the item
  int start, row0, rows, head;
};

template <int D, int RT>
struct AttCfg {
  // Small heads hold few accumulators, and more of their time goes into the
  // softmax of a byte's tokens than into waiting for the byte: more warps, with
  // 128 registers each, instead of 255 (37.1 -> 33.3 us on 48 windowed, capped
  // sequences of 16 heads of 64).
  static constexpr int kWarps = D == 64 ? 16 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kTile = 32;                         // tokens of a tile
  static constexpr int kGroups = kTile / 16;
  static constexpr int kRowsC = 8 * RT;                    // rows of an item
  static constexpr int kHalfTile = kTile * D;              // bytes of the K (or V) part of a tile
  static constexpr int kStage = 2 * kHalfTile;
  static constexpr int kNST = RT == 1 ? 3 : 2;             // ring stages of a warp
  static constexpr int kPartF = kRowsC * (D + 2);          // floats of a piece: accumulators, then (maximum, sum) a row
  // a warp's first piece has a place of its own, its last one lies over its ring
  static constexpr size_t kPartAt = (size_t)kWarps * kNST * kStage;
  static constexpr size_t kRecAt = kPartAt + (size_t)kWarps * kPartF * 4;
  static constexpr size_t kBarsAt = kRecAt + 2 * kWarps * sizeof(Piece);
  static constexpr size_t kMiscAt = kBarsAt + kWarps * kNST * 8;
  static constexpr size_t kNanAt = kMiscAt + 8;            // a bit for each warp that met a NaN
  static constexpr int kAlign = D == 64 ? 512 : 1024;      // of the swizzle's pattern
  static constexpr size_t kSmem = kAlign + kMiscAt + 16;
  static MOE_DEV float* part_of(uint8_t* smem, int w, int last) {  // where warp w leaves its first or last piece
    return reinterpret_cast<float*>(last ? smem + (size_t)w * kNST * kStage : smem + kPartAt + (size_t)w * kPartF * 4);
  }
  static_assert(kPartF * 4 <= kNST * kStage && kPartF % 4 == 0 && kSmem + kWarps * 8 <= 227 * 1024, "shared memory");
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
// tanh(y / (2 log2 e)) = 1 - 2 / (1 + 2^y): off by about 2^-23, absolutely, so a capped
// score by 2^-22 of the cap.  Caps above kFarCap take the other one.
constexpr float kFarCap = 256.f;
MOE_DEV float tanh_of(float y) {
  y = y > 80.f ? 80.f : y;  // (2^y stays finite, a NaN stays one)
  return 1.f - __fdividef(2.f, 1.f + ex2(y));
}
// the same relatively: below 1/4 the series of tanh z, whose next term, 62/2835 z^9, is 2^-21
// of it there
MOE_DEV float tanh_far(float y) {
  const float z = y * (0.5f * kLn2), z2 = z * z;
  const float t = z * fmaf(z2, fmaf(z2, fmaf(z2, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  return fabsf(z) < 0.25f ? t : tanh_of(y);
}
// two E4M3 pairs (the lower and the upper half of w) to two f16 pairs
MOE_DEV void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
      : "=r"(lo), "=r"(hi) : "r"(w));
}
MOE_DEV uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
// The bytes of w that are NaN codes, as 1 each
MOE_DEV uint32_t e4m3x4_nan(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) >> 7 & 0x01010101u; }
// 16-byte chunk c of token row t of a tile of D-byte rows, as TMA swizzles it
template <int D>
MOE_DEV uint32_t chunk_at(uint32_t base, int t, int c) {
  if constexpr (D == 128) return base + t * 128 + ((c ^ (t & 7)) << 4);
  return base + t * 64 + ((c ^ ((t >> 1) & 3)) << 4);
}

// A thread's chunk (D / 8 values) of a V row
template <int D>
MOE_DEV void load_v(uint32_t* v, uint32_t vt, int row, int fg) {
  if constexpr (D == 128) {
    const uint4 x = lds128(chunk_at<D>(vt, row, fg));
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else {
    const uint2 x = lds64(chunk_at<D>(vt, row, fg >> 1) + 8 * (fg & 1));
    v[0] = x.x; v[1] = x.y;
  }
}
template <int D>
MOE_DEV void store_v(const uint32_t* v, uint32_t vt, int row, int fg) {
  if constexpr (D == 128)
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(chunk_at<D>(vt, row, fg)), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3])
                 : "memory");
  else
    asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(chunk_at<D>(vt, row, fg >> 1) + 8 * (fg & 1)), "r"(v[0]), "r"(v[1])
                 : "memory");
}

// What a sequence asks for, from the device-side lengths; the same in every
// CTA.  Lengths out of range count as an empty sequence and are reported.
struct Seq {
  int start, n, len, tile0, units, groups;  // units of an item; groups: row groups
  // the first tile past the item's first u units, of 2^sh tiles each
  template <int kTile>
  MOE_DEV int tile_at(int u, int sh) const { return min((len + kTile - 1) / kTile, tile0 + (max(0, u - kItemCost) << sh)); }
  MOE_DEV bool cut() const { return units > kItemCost + kWholeTiles; }
};
// As read, through L2: a hint's reads must leave nothing behind in L1.  (And no read-only
// loads anywhere: the kernel starts while others may still write its inputs.)
struct Raw {
  int start, stop, len;
  Raw() = default;
  MOE_DEV Raw(const AttArgs& a, int b) {
    start = __ldcg(a.q_start + b);
    stop = __ldcg(a.q_start + b + 1);
    len = __ldcg(a.lens + b);
  }
  MOE_DEV bool operator==(const Raw& o) const { return start == o.start && stop == o.stop && len == o.len; }
};
template <int D, int RT>
MOE_DEV Seq make_seq(const AttArgs& a, const Raw& r, int sh, bool report) {
  constexpr int kTile = AttCfg<D, RT>::kTile;
  Seq s;
  bool bad = !step_rows_ok(r.start, r.stop, a.total);
  s.start = bad ? 0 : r.start;
  s.n = bad ? 0 : r.stop - r.start;
  s.len = r.len;
  const long long cap = (long long)a.width * a.page_size;
  if (s.len < 0 || s.len > cap) { s.len = 0; bad = true; }
  if (bad && report) atomicExch(a.status, MOE_ERR_INVALID_ARG);
  // the first token any row sees (the first row's window), then whole tiles
  const int lo = a.window > 0 ? max(0, s.len - s.n + 1 - a.window) : 0;
  s.tile0 = lo / kTile;
  s.units = kItemCost + (((s.len + kTile - 1) / kTile - s.tile0 + (1 << sh) - 1) >> sh);
  s.groups = (int)(((long long)s.n * a.G + 8 * RT - 1) / (8 * RT));
  return s;
}

// The pieces of a warp: units [u0, u1) of an item (b, head, group), of which
// the first kItemCost are no tiles.
struct Walk {
  int left;            // units still to hand out, this piece included
  int b, head, grp;
  int u0, u1;
  int item0;           // first unit of the item, counted over all items
  Seq s;
};
// Short items are not cut: the warp whose share holds an item's first unit takes all of it.
MOE_DEV void walk_end(Walk& w) {  // u1 from u0 and left
  w.u1 = w.s.cut() ? min(w.s.units, w.u0 + w.left) : w.s.units;
}
template <int D, int RT>
MOE_DEV bool walk_next(Walk& w, const AttArgs& a, int sh) {  // to the next piece
  w.left -= w.u1 - w.u0;
  if (w.left <= 0) return false;
  w.item0 += w.s.units;
  if (++w.grp == w.s.groups) {
    w.grp = 0;
    if (++w.head == a.kv_heads) {
      w.head = 0;
      do {  // (a sequence without rows has no units; one with rows follows, since units are left)
        if (++w.b >= a.B) return false;
        w.s = make_seq<D, RT>(a, Raw(a, w.b), sh, false);
      } while (w.s.groups == 0);
    }
  }
  w.u0 = 0;
  walk_end(w);
  return true;
}
// The first piece of units x ... x + count, if there is one: x lies in sequence b, whose
// units begin with b_first.
template <int D, int RT>
MOE_DEV bool walk_start(Walk& w, const AttArgs& a, int b, const Raw& r, int b_first, int x, int count, int sh) {
  w.left = count;
  w.b = b;
  w.s = make_seq<D, RT>(a, r, sh, false);
  const int it = (x - b_first) / w.s.units;
  w.head = it / max(1, w.s.groups);  // (none: only a hint's lengths that changed)
  w.grp = it - w.head * w.s.groups;
  w.item0 = b_first + it * w.s.units;
  w.u0 = x - w.item0;
  walk_end(w);
  return w.u0 == 0 || w.s.cut() || walk_next<D, RT>(w, a, sh);
}
// total * c / G without 64-bit divisions: c, G <= kAttMaxCtas
MOE_DEV int cta_share(int q, int r, int G, int c) { return q * c + r * c / G; }
// the CTA whose share holds unit x
MOE_DEV int cta_of(int q, int r, int G, int x) {
  int c = min(x / q, G - 1);
  while (cta_share(q, r, G, c) > x) --c;
  return c;
}

// Where a row of an item goes.
struct OutRow {
  size_t at;
  MOE_DEV OutRow(const AttArgs& a, int start, int row, int head) {
    at = (size_t)(start + row / a.G) * (size_t)(a.G * a.kv_heads) + head * a.G + row % a.G;
  }
  MOE_DEV uint16_t* out(const AttArgs& a, int D) const { return reinterpret_cast<uint16_t*>(a.out) + at * D; }
  MOE_DEV void lse(const AttArgs& a, float M, float L) const {
    if (a.lse) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
  }
};

// Four columns of a row over several pieces, each with its own maximum and sum.
// The W lanes of a row hold a piece's (maximum, sum) each.
template <int W>
struct Joined {
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  MOE_DEV float weight(float2 st) {  // this lane's piece's weight; M, L and acc follow
    float Mn = st.x;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) Mn = fmaxf(Mn, __shfl_xor_sync(0xffffffffu, Mn, o));
    Mn = fmaxf(Mn, M);
    const float ms = Mn == -INFINITY ? 0.f : Mn, e0 = ex2(M - ms);
    M = Mn;
    const float e = ex2(st.x - ms);
    float l = e * st.y;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    L = L * e0 + l;
    acc.x *= e0; acc.y *= e0; acc.z *= e0; acc.w *= e0;
    return e;
  }
  MOE_DEV void add(float e, int k, float4 o) {
    const float f = __shfl_sync(0xffffffffu, e, k, W);
    acc.x += o.x * f; acc.y += o.y * f; acc.z += o.z * f; acc.w += o.w * f;
  }
};

// Four columns of a finished row, and (first column) its log-sum-exp.
MOE_DEV void store4(const AttArgs& a, const Piece& p, int r, int D, int d, float4 acc, float M, float L) {
  const OutRow at(a, p.start, p.row0 + r, p.head);
  const float inv = L == 0.f ? 0.f : __fdividef(1.f, L);
  *reinterpret_cast<uint2*>(at.out(a, D) + d) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (d == 0) at.lse(a, M, L);
}

// Where a warp's ring stands: tiles copied and consumed so far, and whether no wait gave up.
struct Ring {
  uint32_t issued, used;
  bool alive;
};

// Every copy a warp issued lands before its CTA ends.
template <class C>
MOE_DEV void wait_ring(uint8_t* smem, Ring& st, int* status) {
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarsAt) + (threadIdx.x >> 5) * C::kNST;
  for (; st.used < st.issued; ++st.used) mbar_wait_landed(full + st.used % C::kNST, (st.used / C::kNST) & 1u, status);
}

// One piece of an item; kCareful: with the rows that do not see a token kept from the NaN
// in its V.
template <int D, int RT, bool MODS, bool kMulti, bool kCareful>
__device__ __forceinline__ void run_piece(const AttArgs& a, const AttMaps& maps, uint8_t* smem, const Walk& w, int sh,
                                          Ring& st) {
  using C = AttCfg<D, RT>;
  constexpr int kRowsC = C::kRowsC, kTile = C::kTile, kGroups = C::kGroups, kNST = C::kNST;
  constexpr int kMT = D / 16;  // 16-row tiles of V^T
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int fg = D == 128 ? ((g & 1) << 2 | g >> 1) : g;  // this thread's chunk of a V row (16 or 8 values)
  uint8_t* ring = smem + (size_t)warp * kNST * C::kStage;  // this warp's
  Piece* recs = reinterpret_cast<Piece*>(smem + C::kRecAt);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarsAt) + warp * kNST;
  int* status = a.status;
  const int P = a.page_size;
  const int box = min(P, kTile);  // token rows of one copy
  const int nbox = kTile / box, gpb = box >> 4;
  const int rows = min(kRowsC, w.s.n * a.G - w.grp * kRowsC);
  const int pos0 = w.s.len - w.s.n;  // position of the step's first token
  // tokens every row sees lie in [lo_all, hi_all), those some row sees in [lo_any, len)
  const int hi_all = pos0 + 1;
  const int lo_all = a.window > 0 ? max(0, w.s.len - a.window) : 0;
  const int lo_any = a.window > 0 ? max(0, pos0 + 1 - a.window) : 0;
  const int t0 = w.s.tile_at<kTile>(w.u0, sh), t1 = w.s.tile_at<kTile>(w.u1, sh);

  // ---- Q rows on their way before the cache's stream starts
  uint4 qv[RT][D / 64][2];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = w.grp * kRowsC + rt * 8 + g;
    const bool live = rt * 8 + g < rows;
    const int i = live ? r / a.G : 0, hq = w.head * a.G + (live ? r - i * a.G : 0);
    const uint16_t* qp = reinterpret_cast<const uint16_t*>(a.q) + (long long)(w.s.start + i) * a.q_stride + hq * D;
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        qv[rt][h][e] = live ? __ldcg(reinterpret_cast<const uint4*>(qp + 64 * h + 16 * q + 8 * e)) : make_uint4(0, 0, 0, 0);
  }
  // ---- pages: lane i looks up 16-token group i of a batch of 32 / kGroups
  // tiles.  The next batch's page numbers are read as this one begins, its
  // scales half-way through, so that neither read is waited for.
  constexpr int kBatch = 32 / kGroups;
  struct Look { int page; float ks, vs; uint32_t ok; };
  auto look_page = [&](Look& k, int tb) {
    const int pos = tb * kTile + 16 * lane;
    k.page = -2;  // not wanted
    if (tb + lane / kGroups < t1 && pos < w.s.len && pos + 16 > lo_any)
      k.page = __ldcg(a.page_table + (size_t)w.b * a.width + pos / P);
  };
  auto look_scale = [&](Look& k) {
    bool ok = k.page >= 0 && k.page < a.num_pages;
    if (!ok && k.page != -2) atomicExch(status, MOE_ERR_INVALID_ARG);  // its tokens are masked
    k.ks = k.vs = 0.f;
    if (ok) {
      k.ks = __ldcg(a.k_scale + (size_t)k.page * a.kv_heads + w.head);
      k.vs = __ldcg(a.v_scale + (size_t)k.page * a.kv_heads + w.head);
    }
    k.ok = __ballot_sync(0xffffffffu, ok);
  };
  Look cur, nxt;
  look_page(cur, t0);
  look_scale(cur);
  int cur0 = t0;  // first tile of cur
  int ti = t0;    // next tile to copy
  auto issue = [&]() {
    const Look& k = ti - cur0 < kBatch ? cur : nxt;
    const int r = (ti - cur0) % kBatch * kGroups;           // lane of the tile's first group
    const uint32_t m = (k.ok >> r) & ((1u << kGroups) - 1);
    const uint32_t bm = (1u << gpb) - 1;
    const int si = st.issued % kNST;
    uint8_t* dst = ring + (size_t)si * C::kStage;
    const int at = ti * kTile % P;  // first row inside the page: 0 unless a page holds several tiles
    // a box is copied if any of its groups is wanted
    int copies = 0;
    for (int i = 0; i < nbox; ++i) copies += ((m >> (i * gpb)) & bm) != 0;
    const bool one = elect_one();
    if (one) mbar_expect_tx(full + si, (uint32_t)(2 * copies * box * D));
    for (int i = 0; i < nbox; ++i) {
      const uint32_t want = (m >> (i * gpb)) & bm;
      if (!want) continue;
      const int pg = __shfl_sync(0xffffffffu, k.page, r + i * gpb + __ffs(want) - 1) * a.kv_heads + w.head;
      if (one) {
        tma_load_3d(dst + i * box * D, &maps.k, 0, at, pg, full + si);
        tma_load_3d(dst + C::kHalfTile + i * box * D, &maps.v, 0, at, pg, full + si);
      }
    }
    ++st.issued;
    ++ti;
  };
  nxt = cur;
  for (int i = 0; i < kNST && ti < t1; ++i) issue();
  look_page(nxt, t0 + kBatch);

  // ---- Q fragments: rows g of row tile 0 in a0 / a2, of row tile 1 in a1 / a3.  Step
  // 4 h + i takes columns 64 h + 16 q + 4 i ... + 3 from lane q: a word of the lane's
  // 16-byte chunk of K.
  uint32_t qf[D / 16][2 * RT];
  float qs[RT];      // 1 / (row's scale), times the softmax scale
  int pos_r[RT];
  float slope[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = w.grp * kRowsC + rt * 8 + g;
    const bool live = rt * 8 + g < rows;
    const int i = live ? r / a.G : 0, hq = w.head * a.G + (live ? r - i * a.G : 0);
    pos_r[rt] = live ? pos0 + i : -1;
    slope[rt] = 0.f;
    if (MODS && a.slopes && live) slope[rt] = __ldcg(a.slopes + hq) * kLog2e;
    const uint4(&v)[D / 64][2] = qv[rt];
    float amax = 0.f;
    bool odd = false;
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
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
    // scale 2^(14 - exponent): the row's maximum lands in [2^14, 2^15); tiny rows
    // keep the largest scale a float can be divided by
    const int ex = max(1, min(253, 268 - (int)(__float_as_uint(amax) >> 23)));
    const float sc = __uint_as_float((uint32_t)ex << 23);
    qs[rt] = __uint_as_float((uint32_t)(254 - ex) << 23) * a.sm_scale;
    if (any_odd & (0xfu << (4 * g))) qs[rt] = __uint_as_float(0x7fc00000u);  // infinities and NaN make the row NaN
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t x[4] = {v[h][e].x, v[h][e].y, v[h][e].z, v[h][e].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __half2 f = __floats2half2_rn(bf16_lo(x[k]) * sc, bf16_hi(x[k]) * sc);
          qf[4 * h + 2 * e + (k >> 1)][RT * (k & 1) + rt] = *reinterpret_cast<const uint32_t*>(&f);
        }
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
  float R = kMinUnit;  // largest V scale so far: the accumulators' unit is R 2^-15
  for (int t = t0; t < t1; ++t) {
    const int si = st.used % kNST;
    if (t - cur0 == kBatch) {
      cur = nxt;
      cur0 = t;
      look_page(nxt, t + kBatch);
    }
    if (t - cur0 == kBatch / 2) look_scale(nxt);
    const int r0 = (t - cur0) * kGroups;
    const int mask = (int)((cur.ok >> r0) & ((1u << kGroups) - 1));
    float ksg[kGroups], vsg[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      ksg[i] = __shfl_sync(0xffffffffu, cur.ks, r0 + i);
      vsg[i] = __shfl_sync(0xffffffffu, cur.vs, r0 + i);
    }
    const int base = t * kTile;
    const bool part = mask != (1 << kGroups) - 1 || base + kTile > hi_all || base < lo_all;
    const uint32_t kt = su32(ring + (size_t)si * C::kStage), vt = kt + C::kHalfTile;
    if (!mbar_wait_landed(full + si, (st.used / kNST) & 1u, status)) { st.alive = false; break; }
    ++st.used;

    if constexpr (kCareful) {
      // NaN codes of V in tokens that some rows see and others do not: rows that see one
      // become NaN there (where the product of "is NaN" and "sees the token" is not
      // zero), and the tile holds zeros in their place.
      if (part) {
#pragma unroll 1
        for (int gr = 0; gr < kGroups; ++gr) {
          uint32_t v4[4][D / 32], sees[RT][2];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 16 * gr + 4 * i + q, pos = base + row;
            const bool here = pos < w.s.len && pos >= lo_any && (pos >= hi_all || pos < lo_all) && ((mask >> gr) & 1);
            uint32_t v[D / 32];
            load_v<D>(v, vt, row, fg);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              const uint32_t nan = here ? e4m3x4_nan(v[k]) : 0u;
              v[k] &= ~(nan * 0xffu);
              v4[i][k] = nan * 0x38u;  // (the code of 1)
            }
            store_v<D>(v, vt, row, fg);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              const bool see = pos <= pos_r[rt] && (a.window <= 0 || pos > pos_r[rt] - a.window);
              const uint32_t one = see ? 0x3c00u << (16 * (i & 1)) : 0u;
              sees[rt][i >> 1] = (i & 1) ? sees[rt][i >> 1] | one : one;
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
              float c[4] = {0.f, 0.f, 0.f, 0.f}, d[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(c, a0, a1, a2, a3, sees[rt][0], sees[rt][1]);
              mma_f16(d, b0, b1, b2, b3, sees[rt][0], sees[rt][1]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (c[i] > 0.f) o[rt][2 * k][i] = NAN;
                if (d[i] > 0.f) o[rt][2 * k + 1][i] = NAN;
              }
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (a copy will take the stage)
        __syncwarp();
      }
    }

    // ---- scores: s[rt][2 j + i] is row g, token 16 (j / 2) + 8 (j % 2) + 4 i + q
    float s[RT][2 * kTile / 8];
#pragma unroll
    for (int j = 0; j < kTile / 8; ++j) {
      const int row = 8 * j + 4 * (g & 1) + (g >> 1);
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        const uint4 kv = lds128(chunk_at<D>(kt, row, 4 * h + q));
        const uint32_t kw[4] = {kv.x, kv.y, kv.z, kv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t(&f)[2 * RT] = qf[4 * h + i];
          uint32_t b0, b1;
          e4m3x4_to_f16x4(kw[i], b0, b1);
          mma_f16(c, f[0], RT == 2 ? f[1] : 0u, f[RT], RT == 2 ? f[2 * RT - 1] : 0u, b0, b1);
        }
      }
      const float ks = ksg[j >> 1];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const float f = qs[rt] * ks * (MODS ? 1.f : kLog2e);
        s[rt][2 * j] = c[2 * rt] * f;
        s[rt][2 * j + 1] = c[2 * rt + 1] * f;
      }
    }
    if (MODS) {
      const float cap_in = a.softcap > 0.f ? fminf(2.f * kLog2e / a.softcap, 3.4028235e38f) : 0.f;
      if (a.softcap > kFarCap) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int k = 0; k < kTile / 4; ++k) s[rt][k] = a.softcap * tanh_far(s[rt][k] * cap_in);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int k = 0; k < kTile / 4; ++k) {
          float x = s[rt][k];
          if (a.softcap > 0.f && a.softcap <= kFarCap) x = a.softcap * tanh_of(x * cap_in);
          const int pos = base + 8 * (k >> 1) + 4 * (k & 1) + q;
          s[rt][k] = fmaf(slope[rt], (float)(pos - pos_r[rt]), x * kLog2e);
        }
    }
    if (part) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int k = 0; k < kTile / 4; ++k) {
          const int pos = base + 8 * (k >> 1) + 4 * (k & 1) + q;
          const bool see = pos <= pos_r[rt] && (a.window <= 0 || pos > pos_r[rt] - a.window) && ((mask >> (k >> 2)) & 1);
          if (!see) s[rt][k] = -INFINITY;
        }
    }
    // ---- running maximum and sum
    float Rn = R;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) Rn = fmaxf(Rn, vsg[i]);  // (0 where a group was not read)
    const float Rq = __fdividef(1.f, Rn);
    const float rr = Rn == R ? 1.f : __fdividef(R, Rn);
    float al[RT];
    bool turn = Rn != R;
    uint32_t pb[RT][kTile / 8];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float mx = s[rt][0];
#pragma unroll
      for (int k = 1; k < kTile / 4; ++k) mx = fmaxf(mx, s[rt][k]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[rt], mx);
      const float ms = mn == -INFINITY ? 0.f : mn;
      al[rt] = ex2(m[rt] - ms);
      turn |= mn > m[rt];
      m[rt] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < kTile / 8; ++j) {
        const float F = vsg[j >> 1] * Rq * kPScale;
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
    for (int gr = 0; gr < kGroups; ++gr) {
      uint32_t v4[4][D / 32];  // tokens q, 4 + q, 8 + q, 12 + q of the group, this thread's chunk
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 16 * gr + 4 * i + q;
        load_v<D>(v4[i], vt, row, fg);
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
    __syncwarp();  // the stage has been read
    if (ti < t1) issue();
  }
  if (!st.alive) return;

  // A NaN in V reaches every row of the tile's products (as a NaN times a weight of zero
  // where a row does not see its token), so one row of each thread shows it.
  if (kMulti && !kCareful) {
    bool nan = false;
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) nan |= o[0][mt][0] != o[0][mt][0] || o[0][mt][2] != o[0][mt][2];
    if (nan) atomicOr(reinterpret_cast<uint32_t*>(smem + C::kNanAt), 1u << warp);
  }

  // ---- the end of a piece
  const bool whole = w.u0 == 0 && w.u1 == w.s.units;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    l[rt] += __shfl_xor_sync(0xffffffffu, l[rt], 1);
    l[rt] += __shfl_xor_sync(0xffffffffu, l[rt], 2);
  }
  // (R and 2^-15 one after the other: their product may be no normal number)
  if (whole) {
    // columns 2 q and 2 q + 1 of the accumulator are rows; this thread has
    // D / 8 consecutive values of each from fg * D / 8
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = rt * 8 + 2 * q + c;
        const float L = __shfl_sync(0xffffffffu, l[rt], 8 * q + 4 * c);
        const float M = __shfl_sync(0xffffffffu, m[rt], 8 * q + 4 * c);
        if (r < rows) {
          const float inv = L == 0.f ? 0.f : __fdividef(1.f / kPScale, L);
          const OutRow o_at(a, w.s.start, w.grp * kRowsC + r, w.head);
          uint32_t v[kMT];
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) v[mt] = pack_bf16(o[rt][mt][c] * inv * R, o[rt][mt][2 + c] * inv * R);
          uint4* dst = reinterpret_cast<uint4*>(o_at.out(a, D) + fg * (D / 8));
#pragma unroll
          for (int k = 0; k < kMT / 4; ++k) dst[k] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          if (g == 0) o_at.lse(a, M, L);
        }
      }
  } else {
    const int last = w.u0 == 0 ? 1 : 0;  // (a warp's piece that starts an item and does not end it is its last)
    float* p = C::part_of(smem, warp, last);
    auto unit = [&](float x) { return x * (1.f / kPScale) * R; };
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int mt = 0; mt < kMT; mt += 2)
          *reinterpret_cast<float4*>(p + (rt * 8 + 2 * q + c) * D + fg * (D / 8) + 2 * mt) =
              make_float4(unit(o[rt][mt][c]), unit(o[rt][mt][2 + c]), unit(o[rt][mt + 1][c]), unit(o[rt][mt + 1][2 + c]));
      if (q == 0) *reinterpret_cast<float2*>(p + kRowsC * D + 2 * (rt * 8 + g)) = make_float2(m[rt], l[rt]);
    }
    if (lane == 0) {
      Piece& rec = recs[2 * warp + last];
      rec.item0 = w.item0;
      rec.units = w.s.units;
      rec.start = w.s.start;
      rec.row0 = w.grp * kRowsC;
      rec.rows = rows;
      rec.head = w.head;
    }
  }
}

// A warp's pieces once more, with care: where V holds a NaN that a mask hides from some
// rows.  That hardly ever is, so the ordinary loop only notes that it met a NaN, and this
// stands out of line.  (A prompt of 2048 tokens behind 2048, us: NaN masked in the loop
// 1500, within the kernel 1170 to 1200, so 1159; none of it 1167.)
template <int D, int RT, bool MODS>
__device__ __noinline__ void careful_walk(const AttArgs& a, const AttMaps& maps, uint8_t* smem, int b, int b_first, int x,
                                          int count, int sh, uint32_t done) {
  using C = AttCfg<D, RT>;
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // a piece's sums lie where copies go now
  __syncwarp();
  Ring st{done, done, true};
  Walk w;
  for (bool more = walk_start<D, RT>(w, a, b, Raw(a, b), b_first, x, count, sh); more && st.alive;
       more = walk_next<D, RT>(w, a, sh))
    run_piece<D, RT, MODS, true, true>(a, maps, smem, w, sh, st);
  wait_ring<C>(smem, st, a.status);
}

template <int D, int RT, bool MODS, bool kMulti>
__global__ void __launch_bounds__((AttCfg<D, RT>::kThreads), 1)
    attention_kernel(const __grid_constant__ AttArgs a, const __grid_constant__ AttMaps maps) {
  using C = AttCfg<D, RT>;
  constexpr int kRowsC = C::kRowsC, kTile = C::kTile, kGroups = C::kGroups, kNST = C::kNST;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
  // Items of up to so many units (and more than kWholeTiles tiles) stay within a CTA where
  // a CTA's share is smaller than that: no joining through memory.  Graph, us, 0 / kWarps /
  // 2 kWarps / 3 kWarps: 19 sequences of 374 to 496 tokens, window 321, 16 heads on one,
  // 12.4 / 12.2 / 10.0 / 10.0; 7 x 3 rows of 200 to 400 tokens, 96 heads on 8, 15.7 / 15.7
  // / 12.6 / 12.6; 4 x 3 of 52 to 1514 tokens, 16 heads of 64 on 4, which then wait for
  // their longest, 11.4 / 11.8 / 11.7 / 11.7; the 80 drawn cases above 9.87 / 9.90 / 9.88
  // / 9.85.
  constexpr int kCtaUnits = 2 * kWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((C::kAlign - (su32(smem_raw) & (C::kAlign - 1))) & (C::kAlign - 1));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Piece* recs = reinterpret_cast<Piece*>(smem + C::kRecAt);                     // [warp][first, last]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarsAt) + warp * kNST;
  int* s_last = reinterpret_cast<int*>(smem + C::kMiscAt);                       // [2] last CTA to arrive, by piece
  int* status = a.status;
  auto part_of = [&](int w, int last) { return C::part_of(smem, w, last); };

  if (lane == 0) {
    for (int i = 0; i < kNST; ++i) mbar_init(full + i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    recs[2 * warp].item0 = recs[2 * warp + 1].item0 = -1;
    if (kMulti && warp == 0) *reinterpret_cast<uint32_t*>(smem + C::kNanAt) = 0;
  }

  grid_dep_launch();
  // ---- the shares: every thread adds up a run of sequences, then a scan
  __shared__ long long s_scan[kWarps];
  int2* s_from = reinterpret_cast<int2*>(s_scan);  // (afterwards) a warp's first sequence and its first unit
  int* s_before = reinterpret_cast<int*>(smem + C::kPartAt);  // [thread]: first unit of its sequences (the pieces come later)
  int* s_units = s_before + kThreads;                          // where it has one sequence: an item's units,
  Raw* s_raw = reinterpret_cast<Raw*>(s_units + kThreads);     // and what was read for it
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  const int P = a.page_size;
  const int gpb = min(P, kTile) >> 4;     // 16-token groups of one copy
  long long total = 0;
  int sh = 0, G = 0, Xq = 0, Xr = 0, X0 = 0, X1 = 0, wb = 0, wat = 0, wx = 0, wn = 0;
  auto warp_share = [&](int w) {  // X0 + (X1 - X0) * w / kWarps
    const int n = X1 - X0;
    return X0 + n / kWarps * w + n % kWarps * w / kWarps;
  };
  // Launched while the kernel before may still run.  What it may write is read
  // early all the same, but as a hint: the shares are worked out and the first tiles
  // brought into L2 from it.  After the kernel before is complete the lengths are
  // read again, and where they are others the shares are worked out again.
  // Nothing is written and no copy into shared memory made before.
  Raw wr;  // of sequence wb
  bool hint = per == 1;
  if (!hint) grid_dep_wait();
  for (;;) {
    long long mine = 0;
    int units1 = 0;
    Raw seen(a, b0 < a.B ? b0 : 0);
    for (int b = b0; b < b1; ++b) {
      const Seq s = make_seq<D, RT>(a, per == 1 ? seen : Raw(a, b), sh, blockIdx.x == 0 && !hint);
      mine = min(mine + (long long)s.units * s.groups * a.kv_heads, 1ll << 40);  // (too many either way)
      units1 = s.units;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    long long before = incl - mine;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    const bool fits = total <= INT_MAX;
    if (!fits && (hint || sh < kCoarsest)) {  // (a hint's lengths say nothing about the units' size)
      if (hint) grid_dep_wait(); else sh += kCoarser;
      hint = false;
      __syncthreads();  // the sums have been read
      continue;
    }
    s_before[tid] = mine > 0 && fits ? (int)before : -1;
    s_units[tid] = units1;
    s_raw[tid] = seen;
    __syncthreads();
    // CTAs that get work
    G = fits ? (int)min((long long)gridDim.x, (total + kWarps - 1) / kWarps) : 0;
    wn = 0;
    if ((int)blockIdx.x < G) {
      Xq = (int)total / G;
      Xr = (int)total - Xq * G;
      X0 = cta_share(Xq, Xr, G, blockIdx.x);
      X1 = cta_share(Xq, Xr, G, blockIdx.x + 1);
      // Where the shares are small, so are the items that stay within a CTA (the one
      // that holds the first of their units takes all): the first two steps move
      // the share's ends.  The last one is for the warp's share.  (One loop: the
      // kernel's first steps wait for their instructions.)
#pragma unroll 1
      for (int step = Xq < kCtaUnits ? 0 : 2; step < 3; ++step) {
        if (step == 2) {
          wx = warp_share(warp);
          wn = warp_share(warp + 1) - wx;
        }
        const int x = step == 0 ? X0 : step == 1 ? X1 : wx;
        if (x >= (int)total) continue;
        // the sequence unit x lies in, and its first unit: the last thread whose run
        // of sequences starts at or before x (and is not empty), then along that run
        int best = -1;  // lane l looks at a run of threads
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) {
          const int at = s_before[lane * (kThreads / 32) + k];
          if (at >= 0 && at <= x) best = k;
        }
        const uint32_t have = __ballot_sync(0xffffffffu, best >= 0);
        const int src = 31 - __clz(have);  // (unit 0 is somebody's, so there is one)
        const int t = __shfl_sync(0xffffffffu, lane * (kThreads / 32) + best, src);
        wat = s_before[t];
        int units = s_units[t];
        wr = s_raw[t];
        for (wb = min(a.B, t * per); per > 1; ++wb) {
          wr = Raw(a, wb);
          const Seq s = make_seq<D, RT>(a, wr, sh, false);
          units = s.units;
          const int nb = units * s.groups * a.kv_heads;
          if (x < wat + nb || wb + 1 >= a.B) break;
          wat += nb;
        }
        if (step < 2 && units > kItemCost + kWholeTiles && units <= kCtaUnits) {
          const int off = (x - wat) % units, to = off > 0 ? x - off + units : x;
          if (step == 0) X0 = to; else X1 = to;
        }
      }
    }
    if (!hint) break;
    if (wn > 0) {
      Walk h;
      const bool any = walk_start<D, RT>(h, a, wb, wr, wat, wx, wn, sh);
      const int t0 = h.s.tile_at<kTile>(h.u0, sh), t1 = min(h.s.tile_at<kTile>(h.u1, sh), t0 + kNST);
      const int pos = t0 * kTile + 16 * lane;  // a lane for each 16-token group
      if (any && t0 >= 0 && t0 + lane / kGroups < t1 && lane % gpb == 0 && pos < h.s.len && h.head < a.kv_heads) {
        const int page = __ldcg(a.page_table + (size_t)h.b * a.width + pos / P);
        if (page >= 0 && page < a.num_pages) {
          tma_prefetch_3d(&maps.k, 0, pos % P, page * a.kv_heads + h.head);
          tma_prefetch_3d(&maps.v, 0, pos % P, page * a.kv_heads + h.head);
        }
      }
    }
    grid_dep_wait();
    hint = false;
    if (__syncthreads_and(b0 >= a.B || Raw(a, b0) == seen)) {
      // (what the hint did not report)
      if (b0 < b1 && blockIdx.x == 0) make_seq<D, RT>(a, seen, sh, true);
      break;
    }
  }
  // (rows that several sequences count as theirs: the host has refused what rows counted once can come to)
  if (total > INT_MAX && tid == 0) atomicExch(status, MOE_ERR_INVALID_ARG);
  if ((int)blockIdx.x >= G) return;  // (the whole CTA; nothing is in flight)
  __syncthreads();  // s_before has been read

  Ring st{0, 0, true};
  if (wn > 0) {
    // (for careful_walk, instead of registers through the loop)
    if (kMulti && lane == 0) s_from[warp] = make_int2(wb, wat);
    Walk w;
    for (bool more = walk_start<D, RT>(w, a, wb, wr, wat, wx, wn, sh); more && st.alive; more = walk_next<D, RT>(w, a, sh))
      run_piece<D, RT, MODS, kMulti, false>(a, maps, smem, w, sh, st);
  }
  wait_ring<C>(smem, st, status);
  __syncwarp();
  if (kMulti && (*reinterpret_cast<volatile uint32_t*>(smem + C::kNanAt) >> warp & 1) && st.alive) {
    const int2 from = s_from[warp];
    const int x = warp_share(warp);
    careful_walk<D, RT, MODS>(a, maps, smem, from.x, from.y, x, warp_share(warp + 1) - x, sh, st.used);
  }
  __syncthreads();

  // ---- the CTA's pieces: those of one item are added, in order.  Every warp
  // finds the items for itself: lane x looks at piece x.
  constexpr int kVec = D / 4;          // lanes of a row, four columns each
  constexpr int kRPW = 32 / kVec;      // rows of a warp at a time
  static_assert(2 * kWarps <= 32, "a piece for each lane");
  const int d = lane % kVec * 4;
  const int my_item = lane < 2 * kWarps ? recs[lane].item0 : -1;
  const uint32_t there = __ballot_sync(0xffffffffu, my_item >= 0);
  const uint32_t below = there & ((1u << lane) - 1);
  const int prev_item = __shfl_sync(0xffffffffu, my_item, 31 - __clz(below | 1));
  const bool lead = my_item >= 0 && (below == 0 || prev_item != my_item);  // first piece of its item
  const uint32_t leads = __ballot_sync(0xffffffffu, lead);
  // items that reach beyond this CTA: at most one from before it, one past it
  const bool out = lead && (my_item < X0 || my_item + recs[lane & (2 * kWarps - 1)].units > X1);
  const uint32_t outs = __ballot_sync(0xffffffffu, out);
  auto item_pieces = [&](int x0) {  // from its first piece up to the next item's
    const uint32_t later = leads & ~((2u << x0) - 1);
    return there & ~((1u << x0) - 1) & ((later & (0u - later)) - 1);
  };
  auto nth = [](uint32_t m, int n) {  // bit of m number n
    for (; n > 0; --n) m &= m - 1;
    return __ffs(m) - 1;
  };
  // slot 0 continues an item of the CTA before this one, slot 1 starts one
  auto cta_part = [&](const Piece& rec) {
    return a.partials + ((size_t)blockIdx.x * 2 + (rec.item0 >= X0 ? 1 : 0)) * C::kPartF;
  };
  const int n_pairs = __popc(leads) * kRowsC;
  // a thread for each (item, row): the pieces' weights take the place of their maxima
  static_assert(2 * kWarps * kRowsC <= kThreads, "a thread for each row of each piece");
  if (tid < n_pairs) {
    const int x0 = nth(leads, tid / kRowsC), r = tid % kRowsC;
    const Piece rec = recs[x0];
    const uint32_t pieces = item_pieces(x0);
    const bool final_ = (outs >> x0 & 1) == 0;
    float2 st[2 * kWarps];  // (read together)
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int k = 0; k < 2 * kWarps; ++k) {
      st[k] = make_float2(-INFINITY, 0.f);
      if (pieces >> k & 1) st[k] = *reinterpret_cast<const float2*>(part_of(k >> 1, k & 1) + kRowsC * D + 2 * r);
      M = fmaxf(M, st[k].x);
    }
    const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int k = 0; k < 2 * kWarps; ++k) {
      st[k].x = ex2(st[k].x - ms);
      L += st[k].x * st[k].y;
    }
    const float inv = !final_ ? 1.f : L == 0.f ? 0.f : __fdividef(1.f, L);
#pragma unroll
    for (int k = 0; k < 2 * kWarps; ++k)
      if (pieces >> k & 1) part_of(k >> 1, k & 1)[kRowsC * D + 2 * r] = st[k].x * inv;
    if (r < rec.rows) {
      if (final_)
        OutRow(a, rec.start, rec.row0 + r, rec.head).lse(a, M, L);
      else
        __stcg(reinterpret_cast<float2*>(cta_part(rec) + kRowsC * D + 2 * r), make_float2(M, L));
    }
  }
  __syncthreads();
  // a warp for each four rows (or pairs of rows, D = 64) of an item, side by side
  constexpr int kChunk = 4 * kRPW, kChunks = kRowsC / kChunk;
  const int n_chunks = __popc(leads) * kChunks;
  for (int ch = warp; ch < n_chunks; ch += kWarps) {
    const int x0 = nth(leads, ch / kChunks), r0 = ch % kChunks * kChunk + lane / kVec;
    const Piece rec = recs[x0];
    float4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (uint32_t m = item_pieces(x0); m; m &= m - 1) {
      const int k = __ffs(m) - 1;
      const float* p = part_of(k >> 1, k & 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + i * kRPW;  // (rows past the item's last hold zeros)
        const float e = p[kRowsC * D + 2 * r];
        const float4 o = *reinterpret_cast<const float4*>(p + r * D + d);
        acc[i].x += o.x * e; acc[i].y += o.y * e; acc[i].z += o.z * e; acc[i].w += o.w * e;
      }
    }
    const bool final_ = (outs >> x0 & 1) == 0;
    float* part = cta_part(rec);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + i * kRPW;
      if (r >= rec.rows) continue;
      if (final_)
        *reinterpret_cast<uint2*>(OutRow(a, rec.start, rec.row0 + r, rec.head).out(a, D) + d) =
            make_uint2(pack_bf16(acc[i].x, acc[i].y), pack_bf16(acc[i].z, acc[i].w));
      else
        __stcg(reinterpret_cast<float4*>(part + (size_t)r * D + d), acc[i]);
    }
  }
  if (outs == 0) return;
  // ---- across CTAs: the last to arrive adds an item's pieces.  The counter's
  // release and acquire reach the other threads through the barriers.
  __syncthreads();
  const int n_out = __popc(outs);
  if (warp < n_out && lane == 0) {
    const Piece rec = recs[__ffs(warp == 0 ? outs : outs & (outs - 1)) - 1];
    const int c0 = cta_of(Xq, Xr, G, rec.item0), c1 = cta_of(Xq, Xr, G, rec.item0 + rec.units - 1);
    const bool last = atom_add_acq_rel(a.tickets + c0, 1) == c1 - c0;
    if (last) a.tickets[c0] = 0;  // ready for the next call
    s_last[warp] = last ? c0 | c1 << 16 : -1;
  }
  __syncthreads();
  // pieces read together (all D / 4 at once: more code that runs once; 25 long sequences,
  // 128 heads, us: 32 34.7, 16 33.5, 8 33.1; one of 51673 tokens 34.3, 34.9, 35.8)
  constexpr int kJoin = kVec < 16 ? kVec : 16;
  for (int i = 0; i < n_out; ++i) {
    const int last = s_last[i];
    if (last < 0) continue;
    const Piece rec = recs[__ffs(i == 0 ? outs : outs & (outs - 1)) - 1];
    const int c0 = last & 0xffff, c1 = last >> 16;
    for (int rb = warp * kRPW; rb < rec.rows; rb += kWarps * kRPW) {
      const int r = rb + lane / kVec;
      auto piece = [&](int c) { return a.partials + ((size_t)c * 2 + (c == c0)) * C::kPartF; };
      Joined<kVec> J;
      for (int c = c0; c <= c1; c += kJoin) {
        const int x = lane % kVec, n = min(kJoin, c1 + 1 - c);
        float2 st = make_float2(-INFINITY, 0.f);
        if (x < n) st = __ldcg(reinterpret_cast<const float2*>(piece(c + x) + kRowsC * D + 2 * r));
        float4 v[kJoin];  // all reads in flight
#pragma unroll
        for (int k = 0; k < kJoin; ++k)
          v[k] = k < n ? __ldcg(reinterpret_cast<const float4*>(piece(c + k) + (size_t)r * D + d))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
        const float e = J.weight(st);
#pragma unroll
        for (int k = 0; k < kJoin; ++k) J.add(e, k, v[k]);
      }
      if (r < rec.rows) store4(a, rec, r, D, d, J.acc, J.M, J.L);
    }
  }
}

// K or V cache [num_pages * kv_heads][page_size][D] bytes; box = rows of one page, up to a tile
bool map_cache(CUtensorMap* m, const uint8_t* base, int D, int P, long long tiles) {
  if (!encode_fn()) return false;
  const cuuint64_t dim[3] = {(cuuint64_t)D, (cuuint64_t)P, (cuuint64_t)tiles};
  const cuuint64_t stride[2] = {(cuuint64_t)D, (cuuint64_t)P * D};
  const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)std::min(P, 32), 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(base), dim, stride, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int RT, bool MODS, bool kMulti>
cudaError_t launch_cfg(const AttArgs& a, const AttMaps& maps, int ctas, cudaStream_t s) {
  using C = AttCfg<D, RT>;
  static OncePerDevice once;
  constexpr auto kernel = attention_kernel<D, RT, MODS, kMulti>;
  if (const cudaError_t rc = allow_smem(once, kernel, C::kSmem); rc != cudaSuccess) return rc;
  PdlLaunch L(dim3(ctas), dim3(C::kThreads), C::kSmem, s);
  return cudaLaunchKernelEx(&L.cfg, kernel, a, maps);
}

// Only calls with several new tokens a sequence have rows that see different tokens.  (Single
// tokens with what those need, us: 9 sequences of 3 to 17 tokens, 96 heads of 64 on 8,
// 6.8 for 5.9; one of 777 tokens, 56 heads of 128 on 8, 9.1 for 9.0.)
template <int D, int RT, bool MODS>
cudaError_t launch_mods(const AttArgs& a, const AttMaps& maps, int ctas, cudaStream_t s) {
  return a.max_new > 1 ? launch_cfg<D, RT, MODS, true>(a, maps, ctas, s) : launch_cfg<D, RT, MODS, false>(a, maps, ctas, s);
}

template <int D>
cudaError_t launch_d(const AttArgs& a, const AttMaps& maps, int ctas, cudaStream_t s) {
  const bool mods = a.softcap > 0.f || a.slopes;
  if (attention_row_tiles(a.G, a.max_new) == 1)
    return mods ? launch_mods<D, 1, true>(a, maps, ctas, s) : launch_mods<D, 1, false>(a, maps, ctas, s);
  return mods ? launch_mods<D, 2, true>(a, maps, ctas, s) : launch_mods<D, 2, false>(a, maps, ctas, s);
}

}  // namespace

// Rows that share one read of the cache: 8 where a sequence has no more, else 16 (16
// sequences of up to 8200 tokens, 7 rows a head and token, us with 8 / with 16: one
// token each 19.9 / 22.3, two 26.5 / 25.0, four 41.0 / 32.0).
int attention_row_tiles(int G, int max_new) { return (long long)G * max_new <= 8 ? 1 : 2; }

size_t attention_partial_bytes(int D, int G, int max_new) {
  return (size_t)kAttMaxCtas * 2 * 8 * attention_row_tiles(G, max_new) * (D + 2) * sizeof(float);
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
