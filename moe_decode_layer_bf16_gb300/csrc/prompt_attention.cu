// Causal attention of packed prompts over themselves, grouped heads, bf16: for row i of
// a prompt and query head h, over its rows j <= i (and j > i - window),
//   s_j = sm_scale q . k_j (capped, biased by distance);
//   out = sum_j exp(s_j) v_j / sum_j exp(s_j);  lse = log sum_j exp(s_j).
//
// What bounds it: the two products, 4 D flops for each visible pair of a row and a key,
// on the tensor cores; beside them an exponential for each pair.  Measured: one prompt of
// 8192 tokens, 56 heads of 128 on 8, 962 GFLOP, 617 to 672 us by the power cap's clock
// (1.43 to 1.56 PFLOP/s, 0.72 to 0.78 of the library product's burst rate; tensor pipe 63%
// busy); 16 prompts of 20 to 2048 tokens 154 us (1.0 PFLOP/s); 33 tokens 9.1 us.
//
// Rows.  The query heads of a key/value head see the same keys, so their rows are packed
// token by token: row r of a prompt and kv head is token r / G, head r % G.  An item is
// two tiles of 128 packed rows (or as many as whole tokens fill) of one prompt and kv head,
// each with its own range of key tiles (128 keys).  Packing wastes next to nothing whatever
// the group is and keeps the masked part of a tile small: 128 rows are 128 / G tokens.
//
// One CTA an SM takes items from a counter, the longest first (of 32 prompts at a time).
// Twenty warps: sixteen for the softmax, of which two share a row, half of its columns each;
// one issues the MMAs, one copies keys and values (TMA, a ring of tiles) and hands out the
// items, two fetch the queries and look through the values of tiles that not every row sees.
// For each key tile
//   S = Q K^T into tensor memory (tcgen05, fp32), a thread reads its half row of S,
//   p = 2^(s c - m c) in bf16 over S's first columns,
//   O += P V (P from tensor memory).
// While one tile's softmax runs, the tensor cores work on the other tile.  The running
// maximum m of a row is moved, and its O and sum rescaled, only when it grows by more than
// 2^8 (a known refinement of the softmax in one pass): until then the weights are up to 2^8,
// with the same relative precision, and a row's two warps need no word of each other but a
// vote.  (With a row a thread, 12 warps in all, the serving mix took 180 us and the long prompt
// as long as now; with four more warps that write the results while the next item begins 180,
// because they take registers and issue slots from the softmax.)
//
// What a masked position holds must not matter, but 0 x NaN is NaN: values of tiles
// that some row does not see in full (the diagonal, a window's edge, a prompt's end) are
// looked through before their product, infinities and NaN replaced by zeros, and put
// back at the end into the rows that see them (3 of the serving mix's 154 us).
#include <cuda.h>

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "async.cuh"
#include "common.cuh"
#include "kernels.h"
#include "step_rows.h"
#include "tcgen05.cuh"
#include "tmap.h"

namespace moe {

namespace {

// mbar_wait_landed for waits that are often long: the thread sleeps up to a millisecond at a
// time, where one that asks again and again takes its scheduler's slots from the softmax (a
// serving mix 189 -> 177 us).
constexpr unsigned long long kItemNs = 5000ull * 1000ull * 1000ull;  // an item of 2^24 keys takes 0.2 s
MOE_DEV bool wait(uint64_t* bar, uint32_t parity, int* status, unsigned long long limit = kWaitNs) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
  do {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(su32(bar)), "r"(parity), "r"(1000000u) : "memory");
    if (ok) return true;
    if (*(volatile int*)status == MOE_ERR_DEVICE_TIMEOUT) return false;
  } while (globaltimer_ns() - t0 < limit);
  atomicExch(status, MOE_ERR_DEVICE_TIMEOUT);
  return false;
}
// The same for a whole warp: its lanes go on or give up together.  (Each reads the clock and
// the status for itself, and one that went on alone would wait for the others at the next
// warp-wide instruction.)
MOE_DEV bool warp_wait(uint64_t* bar, uint32_t parity, int* status, unsigned long long limit = kWaitNs) {
  return __all_sync(0xffffffffu, wait(bar, parity, status, limit));
}

constexpr int kKeys = 128;    // keys of a tile
constexpr int kRows = 128;    // packed rows of a tile
constexpr int kBox = 128 * kKeys;  // bytes of 64 columns of 128 rows
constexpr int kSlots = 4;     // items handed out ahead
constexpr int kLooks = 4;     // tiles of values in the ring at most
constexpr int kThreads = 640;
constexpr int kMma = 16, kCopy = 17, kHelp = 18;  // warps (the softmax's are the first sixteen)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.f;  // log2 of the growth of a row's maximum that is let pass

template <int D>
struct Cfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBoxes * kBox;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kRing = 2 * kTileBytes;  // behind the two query tiles
  static constexpr int kBars = kRing + kStages * kTileBytes;
  static constexpr int kPairs = kBars + 768;        // a value of each softmax thread
  static constexpr int kSmem = kPairs + 2048;
};
static_assert(Cfg<128>::kStages <= 2 * kLooks && Cfg<64>::kStages <= 2 * kLooks, "barriers of values looked through");
static_assert(Cfg<128>::kSmem <= 232448 && Cfg<64>::kSmem <= 232448, "shared memory of a CTA");

// The key tiles of a tile of packed rows, and which of them some row does not see in full.
struct Range {
  int lo, hi;          // none: lo > hi
  int tok_lo, tok_hi;  // tokens of the tile's rows
  MOE_DEV bool has(int j) const { return j >= lo && j <= hi; }
  MOE_DEV bool edge(int j, int window) const {
    return kKeys * j + kKeys - 1 > tok_lo || (window > 0 && kKeys * j <= tok_hi - window);
  }
};
struct Item {
  int start, n, row0, head;  // the prompt's first row and length, the item's first packed row, kv head; n = 0: the end
  Range t[2];
  MOE_DEV int lo() const { return t[0].lo; }
  MOE_DEV int hi() const { return max(t[0].hi, t[1].hi); }
  MOE_DEV bool edge(int j, int window) const {
    return (t[0].has(j) && t[0].edge(j, window)) || (t[1].has(j) && t[1].edge(j, window));
  }
};
MOE_DEV Range range_of(int n, int r0, int rows, int G, int window) {
  Range r{1, 0, 0, 0};
  const int last = n * G - 1;
  if (r0 > last) return r;
  r.tok_lo = r0 / G;
  r.tok_hi = min(r0 + rows - 1, last) / G;
  r.lo = window > 0 ? max(0, r.tok_lo - window + 1) / kKeys : 0;
  r.hi = r.tok_hi / kKeys;
  return r;
}

// What the MMA warp does with a key tile: a word beside its place in the ring, for tile t:
enum Command : uint32_t {
  kHas = 1,       // << t: the tile takes part
  kFirst = 4,     // << t: it is its first
  kLast = 16,     // << t: and its last
  kEdge = 64,     // the values are looked through before they are used
  kEnd = 128      // no more items
};

struct Bars {
  uint64_t kv_full[8], kv_empty[8];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2];
  uint64_t item_full[kSlots], item_empty[kSlots], v_done[kSlots], v_ok[kLooks], drained;
  Item item[kSlots];
  uint32_t cmd[8];
  int bad[kSlots];  // the item met infinities or NaN among values that it looked through
  uint32_t tmem;
};
static_assert(sizeof(Bars) <= 768, "room behind the ring");

// Instruction descriptor of kind::f16: fp32 accumulator, A and B bf16, A K-major; B
// K-major or, for the values, N-major.
MOE_DEV constexpr uint32_t bf16_desc(int n, bool b_n_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_n_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kRows >> 4) << 24);
}
// Shared-memory descriptor of an N-major tile in TMA's 128-byte swizzled layout: 64
// columns of N a box, boxes kBox apart (leading dimension), groups of 8 rows of K 1024
// bytes apart (stride dimension).
MOE_DEV uint64_t n_major_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kBox >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}
MOE_DEV void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
MOE_DEV void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
MOE_DEV void tc_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 bf16 values, rounded, to 32 bytes of memory: one store, where the place is a multiple of
// 32 bytes (a store's address is one of its size), else two.
MOE_DEV void store16(void* to, const float* f, bool whole) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    asm volatile("st.global.v4.b32 [%0], {%1,%2,%3,%4};\n st.global.v4.b32 [%0 + 16], {%5,%6,%7,%8};" ::"l"(to), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  }
}
MOE_DEV void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

MOE_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
MOE_DEV float max3(float x, float y, float z) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
  return m;
}
// (x, y) = (x, y) * c + d, two at a time
MOE_DEV void fma2(float& x, float& y, float c, float d) {
  asm("{\n .reg .b64 a, b, e;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %2};\n mov.b64 e, {%3, %3};\n"
      " fma.rn.f32x2 a, a, b, e;\n mov.b64 {%0, %1}, a;\n}"
      : "+f"(x), "+f"(y)
      : "f"(c), "f"(d));
}
// (x, y) = (x, y) * (u, v) + d
MOE_DEV void fma2(float& x, float& y, float u, float v, float d) {
  asm("{\n .reg .b64 a, b, e;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n mov.b64 e, {%4, %4};\n"
      " fma.rn.f32x2 a, a, b, e;\n mov.b64 {%0, %1}, a;\n}"
      : "+f"(x), "+f"(y)
      : "f"(u), "f"(v), "f"(d));
}
// (x, y) += (u, v) * c
MOE_DEV void bias2(float& x, float& y, float u, float v, float c) {
  asm("{\n .reg .b64 a, b, e;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n mov.b64 e, {%4, %4};\n"
      " fma.rn.f32x2 a, b, e, a;\n mov.b64 {%0, %1}, a;\n}"
      : "+f"(x), "+f"(y)
      : "f"(u), "f"(v), "f"(c));
}
MOE_DEV void mul2(float& x, float& y, float u, float v) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
      : "+f"(x), "+f"(y)
      : "f"(u), "f"(v));
}
MOE_DEV void add2(float& x, float& y, float c, float d) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
      : "+f"(x), "+f"(y)
      : "f"(c), "f"(d));
}

// tanh z: for |z| < kClose z times a polynomial in z^2, the interpolation of tanh(z) / z at
// Chebyshev's nodes of z^2 < kClose^2, off by 6e-8 of it; else 1 - 2 / (1 + e^(2 z)), off by
// 2^-20.4 of it at most.  (The choice is each score's own: a row does not depend on what
// others hold.)
constexpr float kClose = 0.375f;
MOE_DEV float tanh_far(float z) {
  const float y = z * (2.f * kLog2e);
  return 1.f - __fdividef(2.f, 1.f + ex2(y > 80.f ? 80.f : y));  // (2^y stays finite, a NaN stays one)
}

// A row's scores capped and biased, times log2 e; gap: the first one's key minus the row.
template <int N>
MOE_DEV void modified(const PromptArgs& p, float* s, float slope, float gap) {
  const float cap = p.softcap;
  if (cap > 0.f) {
    const float in = p.cap_in, out = cap * kLog2e;
    const float c0 = 0.99999994f * out, c1 = -0.33331971f * out, c2 = 0.13284431f * out, c3 = -0.048268908f * out;
    auto close = [&](float& x, float& y) {  // out * tanh
      float u = x, v = y, f = c3, g = c3;
      mul2(u, v, x, y);
      fma2(f, g, u, v, c2);
      fma2(f, g, u, v, c1);
      fma2(f, g, u, v, c0);
      mul2(x, y, f, g);
    };
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      mul2(s[i], s[i + 1], in, in);
      most = max3(most, fabsf(s[i]), fabsf(s[i + 1]));
    }
    if (__any_sync(0xffffffffu, most >= kClose)) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float x = s[i], y = s[i + 1];
        close(s[i], s[i + 1]);
        if (!(fabsf(x) < kClose)) s[i] = out * tanh_far(x);
        if (!(fabsf(y) < kClose)) s[i + 1] = out * tanh_far(y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 2) close(s[i], s[i + 1]);
    }
  } else {
    const float scale = p.sm_scale * kLog2e;
#pragma unroll
    for (int i = 0; i < N; i += 2) mul2(s[i], s[i + 1], scale, scale);
  }
  if (p.slopes) {
    float x = gap, y = gap + 1.f;  // (whole numbers below 2^24: exact)
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      bias2(s[i], s[i + 1], x, y, slope);
      add2(x, y, 2.f, 2.f);
    }
  }
}

// Whether one of two bf16 values is infinite or NaN, as bits 15 and 31.
MOE_DEV uint32_t not_finite(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
MOE_DEV uint32_t finite_or_zero(uint32_t w) {
  const uint32_t b = not_finite(w);
  return w & ~((b >> 15) * 0xffffu);
}

// A row that sees one of the prompt's infinities or NaN that were replaced gets them back:
// in its half of the columns, from c0.
template <int D>
__device__ __noinline__ void put_back(const PromptArgs& p, const Item& it, int t, int tok, int c0, __nv_bfloat16* out) {
  const Range& r = it.t[t];
  for (int j = r.lo; j <= r.hi; ++j) {
    if (!it.edge(j, p.window)) continue;
    const int k0 = max(kKeys * j, p.window > 0 ? tok - p.window + 1 : 0), k1 = min(kKeys * j + kKeys - 1, tok);
    for (int k = k0; k <= k1; ++k) {
      const uint32_t* v = reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint16_t*>(p.v) +
                                                            (long long)(it.start + k) * p.v_stride + (size_t)it.head * D + c0);
      for (int c = 0; c < D / 4; ++c) {
        const uint32_t w = __ldcg(v + c), b = not_finite(w);
        if (b & 0x8000u) out[2 * c] = __float2bfloat16(__bfloat162float(out[2 * c]) + bf16_lo(w));
        if (b >> 31) out[2 * c + 1] = __float2bfloat16(__bfloat162float(out[2 * c + 1]) + bf16_hi(w));
      }
    }
  }
}

// kMods: scores are capped or biased (or the scale is not positive).
template <int D, bool kMods>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attention_kernel(const __grid_constant__ PromptArgs p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& b = *reinterpret_cast<Bars*>(smem + C::kBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* status = p.status;
  if (su32(smem) & 1023u) {  // (the tiles' swizzle wants it; no other memory of the CTA lies before)
    if (tid == 0) atomicExch(status, MOE_ERR_CUDA);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(b.kv_full + i, 1);
      mbar_init(b.kv_empty + i, 3);  // the MMAs that read it, two helpers
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(b.q_full + t, 1);
      mbar_init(b.q_empty + t, 1);
      mbar_init(b.s_full + t, 1);
      mbar_init(b.p_full[t], 4);
      mbar_init(b.p_full[t] + 1, 4);
      mbar_init(b.o_full + t, 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(b.item_full + i, 1);
      mbar_init(b.item_empty + i, 18);  // sixteen softmax warps, two helpers
      mbar_init(b.v_done + i, 2);
    }
    for (int i = 0; i < kLooks; ++i) mbar_init(b.v_ok + i, 2);
    mbar_init(&b.drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&b.tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();  // (not before the tensor memory is this CTA's: the next kernel may want some and wait for this one)
  // All of tensor memory is this CTA's, so it starts at 0: S (and P) of tile t at 128 t, O at 256 + 128 t.
  constexpr uint32_t tmem = 0;
  grid_dep_wait();
  const int G = p.G, window = p.window;

  // The k-th item of this CTA: every role but the copying warp, which makes them.
  auto item = [&](int k, Item* it) {
    if (!wait(b.item_full + k % kSlots, (k / kSlots) & 1, status, kItemNs)) return false;
    *it = b.item[k % kSlots];
    return it->n > 0;
  };
  auto item_done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(b.item_empty + k % kSlots);
  };

  if (warp < kMma) {
    // ================================================================ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // Tile t's warp for rows 32 q .. 32 q + 31 and half h of the columns.  The two warps of
    // the same rows agree on what is theirs together: at a barrier of their own.
    const int q = warp & 3, t = warp >> 2 & 1, h = warp >> 3, pair = 1 + 4 * t + q;
    const uint32_t quad = (uint32_t)(32 * q) << 16;
    const uint32_t ts = tmem + quad + 128 * t, to = tmem + quad + 256 + 128 * t + D / 2 * h;
    float* mine = reinterpret_cast<float*>(smem + C::kPairs) + 256 * t + 128 * h + 32 * q + lane;
    const float* theirs = mine + (h ? -128 : 128);
    auto either = [&](bool x) {  // of the rows' two warps
      int y;
      asm volatile(
          "{\n .reg .pred p, r;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.or.pred r, %2, 64, p;\n selp.s32 %0, 1, 0, r;\n}"
          : "=r"(y) : "r"((int)x), "r"(pair) : "memory");
      return y != 0;
    };
    const float c = kMods ? 1.f : p.sm_scale * kLog2e;
    const int heads = G * p.kv_heads;
    uint32_t steps = 0, items = 0;
    Item it;
    // (A wait that fails leaves the status set, and every later one gives up in a millisecond: a pair's
    // warps go through the same barriers to the item's end either way.)
    for (int k = 0;; ++k) {
      const bool more = item(k, &it);
      if (either(!more)) break;
      const Range rg = it.t[t];
      if (rg.lo > rg.hi) {
        item_done(k);
        continue;
      }
      const int r = 32 * q + lane, row = it.row0 + t * p.rows + r;
      const bool live = r < p.rows && row < it.n * G;
      const int tok = min(row / G, it.n - 1), head = it.head * G + (live ? row - row / G * G : 0);
      const float slope = kMods && p.slopes ? p.slopes[head] * kLog2e : 0.f;
      float m = -INFINITY, mc = 0.f, l0 = 0.f, l1 = 0.f;  // maximum in use, times c; two parts of the half's sum
      for (int j = rg.lo; j <= rg.hi; ++j, ++steps) {
        wait(b.s_full + t, steps & 1, status);
        tc_fence_after();
        float s[kKeys / 2];
        tc_ld32(ts + 64 * h, s);
        tc_ld32(ts + 64 * h + 32, s + 32);
        tc_wait_ld();
        if constexpr (kMods) modified<kKeys / 2>(p, s, slope, (float)(kKeys * j + 64 * h - tok));
        if (rg.edge(j, window)) {
          const int last = tok - kKeys * j - 64 * h, first = window > 0 ? last - window + 1 : -kKeys;
          // bits of the columns that the row sees
          const uint64_t upto = last < 0 ? 0ull : last >= 63 ? ~0ull : (2ull << last) - 1;
          const uint64_t seen = first <= 0 ? upto : first > 63 ? 0ull : upto & (~0ull << first);
          const uint32_t w0 = (uint32_t)seen, w1 = (uint32_t)(seen >> 32);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            s[i] = w0 & (1u << i) ? s[i] : -INFINITY;
            s[i + 32] = w1 & (1u << i) ? s[i + 32] : -INFINITY;
          }
        }
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = max3(s[3 * i], s[3 * i + 1], s[3 * i + 2]);
#pragma unroll
        for (int i = 12; i + 1 < kKeys / 2; i += 2) top[i / 2 & 3] = max3(top[i / 2 & 3], s[i], s[i + 1]);
        const float mt = fmaxf(max3(top[0], top[1], top[2]), top[3]);
        // Where a row's maximum grows by much, the maximum in use follows; what lies in rows past
        // the tile's has no part in it.  (Past this barrier both warps have read their scores, and
        // weights may take the scores' place.)
        tc_fence_before();
        const bool grown = either(live && (mt - m) * c > kGrow);
        tc_fence_after();
        if (grown) {
          *mine = mt;
          either(false);
          // each row's by its own scores alone: what the warps' other rows hold, other heads and later
          // tokens, must not move its last bits
          const float both = fmaxf(mt, *theirs);
          const bool up = live && (both - m) * c > kGrow;
          const float mn = up ? both : m, mcn = up ? both * c : mc;
          const float f = !up ? 1.f : m == -INFINITY ? 0.f : ex2(mc - mcn);
          l0 *= f;
          l1 *= f;
          if (j > rg.lo) {  // (this tile's products so far were complete before S was)
#pragma unroll 1
            for (int i = 0; i < D / 2; i += 16) {  // (rare: unrolled, its registers would be missed elsewhere)
              float o[16];
              tc_ld16(to + i, o);
              tc_wait_ld();
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * f);
              tc_st16(to + i, w);
            }
            // both halves of O are rescaled before either warp's weights let products at them
            tc_wait_st();
            tc_fence_before();
            either(false);
            tc_fence_after();
          }
          m = mn;
          mc = mcn;
        }
#pragma unroll
        for (int i = 0; i < kKeys / 2; i += 32) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x = s[i + e], y = s[i + e + 1];
            fma2(x, y, c, -mc);
            x = ex2(x);
            y = ex2(y);
            add2(l0, l1, x, y);
            w[e / 2] = pack_bf16(x, y);
          }
          tc_st16(ts + 32 * h + i / 2, w);
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b.p_full[t] + h);
      }
      // ---------------------------------------------------------------- the rows' results
      either(false);
      *mine = l0 + l1;
      either(false);
      const float l = h ? *theirs + *mine : *mine + *theirs, inv = 1.f / l;
      wait(b.o_full + t, items++ & 1, status);
      tc_fence_after();
      const size_t at = (size_t)(it.start + tok) * heads + head;
      uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + at * D + D / 2 * h;
#pragma unroll
      for (int i = 0; i < D / 2; i += 16) {
        float o[16];
        tc_ld16(to + i, o);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] *= inv;
        if (live) store16(out + i, o, p.out32);
      }
      tc_fence_before();
      if (p.lse && live && h == 0) p.lse[at] = (mc + log2f(l)) * kLn2;
      wait(b.v_done + k % kSlots, (k / kSlots) & 1, status);
      if (b.bad[k % kSlots] && live)
        put_back<D>(p, b.item[k % kSlots], t, tok, D / 2 * h, reinterpret_cast<__nv_bfloat16*>(out));
      item_done(k);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == kMma) {
      // ================================================================ MMA
      if (elect_one()) {
        // What the MMAs take is made of constants and of counters that only this thread moves,
        // so that it stays in uniform registers.
        uint32_t edges = 0, pq = 0, pp = 0;  // phases of the two tiles' barriers, a bit each
        const uint32_t sq = su32(smem), sring = su32(smem + C::kRing);
        struct Place {
          uint32_t st = 0, ph = 0;
          MOE_DEV void next() {
            if (++st == C::kStages) {
              st = 0;
              ph ^= 1;
            }
          }
        };
        auto landed = [&](const Place& n) { return wait(b.kv_full + n.st, n.ph, status); };
        // O += P V of tile t; V in ring place n
        auto product = [&](auto tc, const Place& n, uint32_t cmd) {
          constexpr int t = decltype(tc)::value;
          const uint64_t dv = n_major_desc(sring + n.st * C::kTileBytes);
          constexpr uint32_t d = 256 + 128 * t, a = 128 * t, idesc = bf16_desc(D, true);
          const uint32_t ph = pp >> t & 1;
          pp ^= 1u << t;
          if (!wait(b.p_full[t], ph, status)) return false;
          tc_fence_after();
          mma_ts(d, a, dv, idesc, cmd & (kFirst << t) ? 0 : 1);
#pragma unroll
          for (int s = 1; s < kKeys / 32; ++s) mma_ts(d, a + 8 * s, dv + (uint64_t)(s * (2048 >> 4)), idesc, 1);
          if (!wait(b.p_full[t] + 1, ph, status)) return false;
          tc_fence_after();
#pragma unroll
          for (int s = kKeys / 32; s < kKeys / 16; ++s) mma_ts(d, a + 8 * s, dv + (uint64_t)(s * (2048 >> 4)), idesc, 1);
          if (cmd & (kLast << t)) tc_commit(b.o_full + t);
          return true;
        };
        // S = Q K^T of tile t; K in ring place n
        auto scores = [&](auto tc, const Place& n, uint32_t cmd) {
          constexpr int t = decltype(tc)::value;
          if (cmd & (kFirst << t)) {
            if (!wait(b.q_full + t, pq >> t & 1, status)) return false;
            pq ^= 1u << t;
            tc_fence_after();
          }
          const uint64_t dq = smem_desc(sq + t * C::kTileBytes), dk = smem_desc(sring + n.st * C::kTileBytes);
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint64_t at = (uint64_t)((s / 4 * kBox + s % 4 * 32) >> 4);
            mma_ss(128 * t, dq + at, dk + at, bf16_desc(kKeys, false), s > 0);
          }
          tc_commit(b.s_full + t);
          if (cmd & (kLast << t)) tc_commit(b.q_empty + t);
          return true;
        };
        using T0 = std::integral_constant<int, 0>;
        using T1 = std::integral_constant<int, 1>;
        // A step is a key tile of an item: its scores, with the products of the step before
        // (whose item may be another one).
        uint32_t cmd = 0, old = 0;
        Place key, val;
        while (true) {
          bool early = false;
          if (old) {
            if (!landed(val)) break;
            if (old & kEdge) {
              if (!wait(b.v_ok + edges % kLooks, edges / kLooks & 1, status)) break;
              ++edges;
            }
            if ((old & kHas) && !product(T0(), val, old)) break;
            // tile 0's scores come between the products where their data are there
            if (mbar_try_wait(b.kv_full + key.st, key.ph)) {
              cmd = b.cmd[key.st];
              early = (cmd & kHas) && (!(cmd & kFirst) || mbar_try_wait(b.q_full, pq & 1));
              if (early && !scores(T0(), key, cmd)) break;
            }
            if ((old & (kHas << 1)) && !product(T1(), val, old)) break;
            tc_commit(b.kv_empty + val.st);
          }
          if (!landed(key)) break;
          cmd = b.cmd[key.st];
          if (cmd & kEnd) break;
          if ((cmd & kHas) && !early && !scores(T0(), key, cmd)) break;
          if ((cmd & (kHas << 1)) && !scores(T1(), key, cmd)) break;
          tc_commit(b.kv_empty + key.st);
          old = cmd;
          val = key;
          val.next();
          key = val;
          key.next();
        }
        // No MMA, and no arrival at a barrier that one is to make, may still be under way when the
        // CTA leaves (the last tiles' ring places and queries are given back, and nobody waits for them).
        tc_commit(&b.drained);
        mbar_wait_landed(&b.drained, 0, status);
      }
      __syncwarp();
    } else if (warp == kCopy) {
      // ================================================================ items, keys and values
      asm volatile("fence.proxy.async.global;" ::: "memory");
      uint32_t ring = 0;
      bool alive = true, ended = false;
      // A run of 32 prompts at a time, a lane each.  Their items come by level, the longest first:
      // at level L the L-th block of rows of each prompt that has one.
      int b0 = -32, before = 0, level = 0, start = 0, n = 0, blocks = 0, last = 0;  // before: items before this level; last: the last row so far
      int next = blockIdx.x;
      for (int k = 0; alive; ++k) {
        int ahead = 0;
        if (lane == 0) ahead = atomicAdd(p.tickets, 1);
        uint32_t who = 0;  // the prompts that have a block at this level
        while (b0 < p.B) {
          who = __ballot_sync(0xffffffffu, level > 0 && blocks >= level);
          const int each = __popc(who) * p.kv_heads;
          if (each > 0) {
            // the levels down to the next shorter prompt's have as many items each
            const int below = __reduce_max_sync(0xffffffffu, blocks < level ? blocks : 0);
            const int down = min((next - before) / each, level - below);
            before += down * each;
            level -= down;
            if (level > below) break;
            continue;
          }
          b0 += 32;
          start = n = 0;
          bool bad = false;
          if (b0 + lane < p.B) {
            start = p.q_start[b0 + lane];
            const int stop = p.q_start[b0 + lane + 1];
            bad = !step_rows_ok(start, stop, p.total);
            if (!bad) n = stop - start;
          }
          // a prompt that starts before an earlier one ends is none either
          int end = n > 0 ? start + n : 0;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int before_it = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end = max(end, before_it);
          }
          int prior = __shfl_up_sync(0xffffffffu, end, 1);
          prior = lane > 0 ? max(prior, last) : last;
          last = max(last, __shfl_sync(0xffffffffu, end, 31));
          const bool on = n > 0 && p.lens && p.lens[b0 + lane] != n;  // (it goes on from tokens that are no rows here)
          if (n > 0 && (start < prior || on)) {
            n = 0;
            bad = true;
          }
          if (bad && blockIdx.x == 0) atomicExch(status, MOE_ERR_INVALID_ARG);
          blocks = (n * G + 2 * p.rows - 1) / (2 * p.rows);
          level = __reduce_max_sync(0xffffffffu, blocks);
        }
        const bool end = b0 >= p.B;
        Item it{};
        if (!end) {
          const int idx = (next - before) / p.kv_heads;
          const uint32_t mine = __ballot_sync(0xffffffffu, (who >> lane & 1) && __popc(who & ((1u << lane) - 1)) == idx);
          const int from = __ffs(mine) - 1;
          it.start = __shfl_sync(0xffffffffu, start, from);
          it.n = __shfl_sync(0xffffffffu, n, from);
          it.row0 = (level - 1) * 2 * p.rows;
          it.head = (next - before) % p.kv_heads;
          it.t[0] = range_of(it.n, it.row0, p.rows, G, window);
          it.t[1] = range_of(it.n, it.row0 + p.rows, p.rows, G, window);
        }
        if (!warp_wait(b.item_empty + k % kSlots, ((k / kSlots) & 1) ^ 1, status, kItemNs)) break;
        if (lane == 0) {
          b.item[k % kSlots] = it;
          b.bad[k % kSlots] = 0;
          mbar_arrive(b.item_full + k % kSlots);
        }
        __syncwarp();
        if (elect_one()) {
          auto command = [&](int j) {
            uint32_t c = it.edge(j, window) ? kEdge : 0;
            for (int t = 0; t < 2; ++t)
              if (it.t[t].has(j))
                c |= (kHas | (j == it.t[t].lo ? kFirst : 0) | (j == it.t[t].hi ? kLast : 0)) << t;
            return c;
          };
          if (end) {
            const uint32_t st = ring % C::kStages;
            if (wait(b.kv_empty + st, (ring / C::kStages & 1) ^ 1, status)) {
              b.cmd[st] = kEnd;
              mbar_arrive(b.kv_full + st);
              ended = true;
            }
          }
          for (int j = it.lo(); !end && j <= it.hi(); ++j) {
            for (int kv = 0; kv < 2; ++kv, ++ring) {
              const uint32_t st = ring % C::kStages;
              if (!wait(b.kv_empty + st, (ring / C::kStages & 1) ^ 1, status)) { alive = false; break; }
              if (!kv) b.cmd[st] = command(j);
              mbar_expect_tx(b.kv_full + st, C::kTileBytes);
              for (int x = 0; x < C::kBoxes; ++x)
                tma_load_3d(smem + C::kRing + st * C::kTileBytes + x * kBox, kv ? &vmap : &kmap, 64 * x, it.head,
                            it.start + kKeys * j, b.kv_full + st);
            }
            if (!alive) break;
          }
        }
        ended = __any_sync(0xffffffffu, ended);
        if (end) break;
        ring = __shfl_sync(0xffffffffu, __reduce_max_sync(0xffffffffu, ring), 0);
        alive = __all_sync(0xffffffffu, alive);
        next = (int)gridDim.x + __shfl_sync(0xffffffffu, ahead, 0);
      }
      // nothing may still be on its way when the CTA leaves (at the regular end all has been used)
      for (uint32_t r = ring > C::kStages ? ring - C::kStages : 0; !ended && r < ring; ++r)
        mbar_wait_landed(b.kv_full + r % C::kStages, r / C::kStages & 1, status);
      // the last CTA leaves the counters as it found them
      if (lane == 0 && atom_add_acq_rel(p.tickets + 1, 1) == (int)gridDim.x - 1) p.tickets[0] = p.tickets[1] = 0;
    } else {
      // ================================================================ queries; values that not every row sees
      const int t = warp - kHelp;
      asm volatile("fence.proxy.async.global;" ::: "memory");
      constexpr int kChunks = D / 8;  // 16-byte pieces of a row
      uint32_t ring = 0, fills = 0, edges = 0;
      bool alive = true;
      Item it;
      for (int k = 0; alive && __all_sync(0xffffffffu, item(k, &it)); ++k) {
        if (it.t[t].lo <= it.t[t].hi) {
          if (!warp_wait(b.q_empty + t, (fills & 1) ^ 1, status, kItemNs)) break;
          ++fills;
          if (p.rows % G == 0) {
            // whole tokens: one copy for 64 columns
            if (elect_one()) {
              mbar_expect_tx(b.q_full + t, p.rows * D * 2);
              for (int x = 0; x < C::kBoxes; ++x)
                tma_load_4d(smem + t * C::kTileBytes + x * kBox, &qmap, 64 * x, 0, it.head, it.start + it.t[t].tok_lo, b.q_full + t);
            }
            __syncwarp();
          } else {
            // a pass of the warp is kStep rows; a row's step to the next pass is some tokens and heads
            constexpr int kStep = 32 / kChunks;
            const int ch = lane % kChunks, r0 = lane / kChunks, row = it.row0 + t * p.rows + r0;
            const int left = it.n * G - it.row0 - t * p.rows;  // rows of the tile (it may be over)
            const int tok = row / G, toks = kStep / G, more = kStep - toks * G;
            int g = row - tok * G;
            const uint16_t* src = reinterpret_cast<const uint16_t*>(p.q) + (long long)(it.start + tok) * p.q_stride +
                                  (size_t)(it.head * G + g) * D + ch * 8;
            const long long step = toks * p.q_stride + more * D, wrap = p.q_stride - G * D;
            const uint32_t to = su32(smem) + t * C::kTileBytes + ch / 8 * kBox + r0 * 128;
#pragma unroll 8
            for (int i = 0; i < kRows; i += kStep) {
              const bool in = r0 + i < left;
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * 128 + ((ch % 8 ^ ((r0 + i) & 7)) << 4)),
                           "l"(in ? src : reinterpret_cast<const uint16_t*>(p.q)), "r"(in ? 16 : 0)
                           : "memory");
              src += step;
              g += more;
              if (g >= G) {
                g -= G;
                src += wrap;
              }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(b.q_full + t);
          }
        }
        // every tile of the ring is waited for and given back in turn: a wait that skips one
        // could not tell its phase from the last but one
        for (int i = 0; alive && i < 2 * (it.hi() - it.lo() + 1); ++i, ++ring) {
          const uint32_t st = ring % C::kStages;
          if (!warp_wait(b.kv_full + st, ring / C::kStages & 1, status)) { alive = false; break; }
          if (!(i & 1) || !it.edge(it.lo() + i / 2, window)) {
            __syncwarp();
            if (lane == 0) mbar_arrive(b.kv_empty + st);
            continue;
          }
          // this warp's half of the tile (in any order: the swizzle stays within it)
          uint4* half = reinterpret_cast<uint4*>(smem + C::kRing + st * C::kTileBytes + t * (C::kTileBytes / 2)) + lane;
          uint32_t any = 0;
#pragma unroll 8
          for (int x = 0; x < C::kTileBytes / 2 / 512; ++x) {
            const uint4 w = half[32 * x];
            any |= not_finite(w.x) | not_finite(w.y) | not_finite(w.z) | not_finite(w.w);
          }
          if (__any_sync(0xffffffffu, any != 0)) {
            for (int x = 0; x < C::kTileBytes / 2 / 512; ++x) {
              const uint4 w = half[32 * x];
              half[32 * x] = make_uint4(finite_or_zero(w.x), finite_or_zero(w.y), finite_or_zero(w.z), finite_or_zero(w.w));
            }
            b.bad[k % kSlots] = 1;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(b.v_ok + edges % kLooks);
            mbar_arrive(b.kv_empty + st);
          }
          ++edges;
        }
        __syncwarp();
        if (alive && lane == 0) mbar_arrive(b.v_done + k % kSlots);
        if (alive) item_done(k);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (fills > 0) mbar_wait_landed(b.q_full + t, (fills - 1) & 1, status);  // (nothing on its way when the CTA leaves)
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Rows of a [total][kv_heads][D] array, `stride` elements apart, in boxes of 64 columns
// of one head and 128 rows; rows past the end read as zeros.
bool map_rows(CUtensorMap* m, const void* base, int D, int heads, int total, long long stride) {
  if (!encode_fn()) return false;
  const cuuint64_t dim[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)total};
  const cuuint64_t step[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, kKeys}, es[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dim, step, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as [total][kv_heads][G][D], in boxes of 64 columns, the G heads of a kv head
// and a tile's tokens.
bool map_queries(CUtensorMap* m, const PromptArgs& a, int D) {
  const cuuint64_t dim[4] = {(cuuint64_t)D, (cuuint64_t)a.G, (cuuint64_t)a.kv_heads, (cuuint64_t)a.total};
  const cuuint64_t step[3] = {(cuuint64_t)D * 2, (cuuint64_t)a.G * D * 2, (cuuint64_t)a.q_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)a.G, 1, (cuuint32_t)(a.rows / a.G)}, es[4] = {1, 1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.q), dim, step, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kMods>
cudaError_t launch_as(const PromptArgs& a, int sms, cudaStream_t s) {
  static OncePerDevice once;
  if (const cudaError_t rc = allow_smem(once, prompt_attention_kernel<D, kMods>, Cfg<D>::kSmem); rc != cudaSuccess) return rc;
  CUtensorMap qmap{}, kmap, vmap;
  if (!map_rows(&kmap, a.k, D, a.kv_heads, a.total, a.k_stride) || !map_rows(&vmap, a.v, D, a.kv_heads, a.total, a.v_stride))
    return cudaErrorUnknown;
  if (a.rows % a.G == 0 && !map_queries(&qmap, a, D)) return cudaErrorUnknown;
  // items at most: a started one for each prompt and head beside the full ones
  const long long items = ((long long)a.total * a.G / (2 * a.rows) + std::min(a.B, a.total)) * a.kv_heads;
  PdlLaunch L(dim3((unsigned)std::min<long long>(items, sms)), dim3(kThreads), Cfg<D>::kSmem, s);
  return cudaLaunchKernelEx(&L.cfg, prompt_attention_kernel<D, kMods>, a, qmap, kmap, vmap);
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs& args, int sms, cudaStream_t s) {
  PromptArgs a = args;
  // A tile's rows: whole tokens, which one copy brings, where that fills it to 7 / 8; else 128.
  const int whole = kRows / a.G * a.G;
  a.rows = 8 * whole >= 7 * kRows ? whole : kRows;
  a.out32 = ((uintptr_t)a.out & 31) == 0;  // (a row's 16 values lie a multiple of 32 bytes behind)
  // The cap times log2 e and the factor under the tanh stay finite: no score comes near the caps'
  // ends, and with the factor at its own every score but zero has the cap for its size.
  if (a.softcap > 0.f) a.softcap = std::min(std::max(a.softcap, 0x1p-100f), 0x1p100f);
  a.cap_in = a.softcap > 0.f ? std::min(std::max(a.sm_scale / a.softcap, -FLT_MAX), FLT_MAX) : 0.f;
  const float c = a.sm_scale * kLog2e;
  const bool mods = a.softcap > 0.f || a.slopes || !(c > 1e-30f && c < 1e30f);
  if (a.D == 64) return mods ? launch_as<64, true>(a, sms, s) : launch_as<64, false>(a, sms, s);
  return mods ? launch_as<128, true>(a, sms, s) : launch_as<128, false>(a, sms, s);
}

}  // namespace moe
