// Pages of the cache given to a step's new tokens and taken back, on the GPU: block
// tables, row starts, positions and slots from the requests' lengths.
//
// The free pages are a stack.  A sequence's page need is
// ceil((len + new) / P) - ceil(len / P); running sums of the needs say which pages of
// the stack's top it gets, and whether it gets any: once the sums pass what the stack
// holds, no later sequence that needs pages fits either, so nothing has to be decided
// in turn.  Running sums of the rows that are given make q_start.
//
// One cluster of CTAs, each with a run of the sequences; they exchange their sums through
// shared memory.  Rows and pages of a run are then written by one thread each, which
// finds its sequence among the run's running sums by bisection: coalesced, and even
// whatever the lengths are.  Bound by latency: a launch and three dependent reads.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "../../include/moe_decode.h"

namespace cg = cooperative_groups;

namespace moe {

namespace {

constexpr int kThreads = 1024;
constexpr int kMaxCluster = 8;

struct Sums {
  long long pages, rows;
};

MOE_DEV Sums operator+(const Sums& a, const Sums& b) { return {a.pages + b.pages, a.rows + b.rows}; }

// The sum over the threads before this one; *all gets the sum over the CTA.
MOE_DEV Sums scan_before(Sums v, Sums* s_warp, Sums* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums up = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums w{__shfl_up_sync(0xffffffffu, up.pages, o), __shfl_up_sync(0xffffffffu, up.rows, o)};
    if (lane >= o) up = up + w;
  }
  __syncthreads();  // (s_warp may still be read)
  if (lane == 31) s_warp[warp] = up;
  __syncthreads();
  Sums w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums x{__shfl_up_sync(0xffffffffu, w.pages, o), __shfl_up_sync(0xffffffffu, w.rows, o)};
    if (lane >= o) w = w + x;
  }
  *all = {__shfl_sync(0xffffffffu, w.pages, 31), __shfl_sync(0xffffffffu, w.rows, 31)};
  const Sums before{__shfl_sync(0xffffffffu, w.pages, warp > 0 ? warp - 1 : 0),
                    __shfl_sync(0xffffffffu, w.rows, warp > 0 ? warp - 1 : 0)};
  up = {up.pages - v.pages, up.rows - v.rows};
  return warp > 0 ? up + before : up;
}

// The sums of the CTAs before this one, and of all.
MOE_DEV Sums cluster_before(cg::cluster_group& cluster, Sums mine, Sums* s_part, Sums* all) {
  if (threadIdx.x == 0) *s_part = mine;
  cluster.sync();
  Sums before{0, 0}, total{0, 0};
  const int rank = (int)cluster.block_rank(), n = (int)cluster.num_blocks();
  for (int r = 0; r < n; ++r) {
    const Sums v = *cluster.map_shared_rank(s_part, r);
    if (r < rank) before = before + v;
    total = total + v;
  }
  *all = total;
  return before;
}

// The last of the n entries of `first` (ascending, first[0] <= i) that is at most i.
MOE_DEV int find(const int* first, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// A sequence's tokens held and asked for, pages held and needed.
struct Need {
  int len, fresh, held, pages;
};
MOE_DEV Need need_of(const PagesArgs& a, int b, bool* bad) {
  Need n{a.lens[b], a.fresh[b], 0, 0};
  const long long cap = (long long)a.width << a.shift;
  if (n.len < 0 || n.fresh < 0 || (long long)n.len + n.fresh > cap) {
    *bad = true;
    n.fresh = 0;
    return n;
  }
  const int up = (1 << a.shift) - 1;
  n.held = (n.len + up) >> a.shift;
  n.pages = ((n.len + n.fresh + up) >> a.shift) - n.held;
  return n;
}

__global__ void __launch_bounds__(kThreads) extend_kernel(PagesArgs a) {
  __shared__ Sums s_warp[kThreads / 32], s_part[2];
  __shared__ int s_row[kThreads], s_page[kThreads];      // the run's rows and pages before each sequence, from its own first
  __shared__ int s_len[kThreads], s_old[kThreads], s_held[kThreads];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  grid_dep_launch();
  grid_dep_wait();
  const int run = (a.B + ranks - 1) / ranks;
  const int b0 = min(rank * run, a.B), b1 = min(b0 + run, a.B);
  bool bad = false;
  const int stack = a.free_state[0];
  const int count = stack < 0 || stack > a.capacity ? 0 : stack;
  if (count != stack) bad = true;
  if (tid < kThreads / 32) s_warp[tid] = {0, 0};
  // what the run's sequences ask for
  Sums mine{0, 0}, all, part;
  for (int c = b0; c < b1; c += kThreads) {
    const int b = c + tid;
    Sums v{0, 0};
    if (b < b1) {
      const Need n = need_of(a, b, &bad);
      v = {n.pages, n.fresh};
    }
    scan_before(v, s_warp, &part);
    mine = mine + part;
  }
  const Sums asked0 = cluster_before(cluster, mine, &s_part[0], &all);
  const long long asked_pages = all.pages;
  // what they get
  auto given = [&](int c, const Sums& asked, Need* n, Sums* before) {
    const int b = c + tid;
    *n = Need{0, 0, 0, 0};
    if (b < b1) *n = need_of(a, b, &bad);
    Sums sum;
    *before = asked + scan_before({n->pages, n->fresh}, s_warp, &sum);
    const bool room = n->fresh == 0 || before->rows + n->fresh <= a.rows;
    if (!room) bad = true;
    if (!room || (n->pages > 0 && before->pages + n->pages > count)) n->fresh = n->pages = 0;
    return sum;
  };
  mine = {0, 0};
  Sums asked = asked0;
  for (int c = b0; c < b1; c += kThreads) {
    Need n;
    Sums before;
    const Sums sum = given(c, asked, &n, &before);
    scan_before({n.pages, n.fresh}, s_warp, &part);
    asked = asked + sum;
    mine = mine + part;
  }
  Sums got = cluster_before(cluster, mine, &s_part[1], &all);
  if (rank == 0 && tid == 0) {
    a.free_out[0] = stack - (int)all.pages;
    a.free_out[1] = (int)min(asked_pages - all.pages, (long long)INT32_MAX);
    a.q_start[a.B] = (int)all.rows;
  }
  asked = asked0;
  for (int c = b0; c < b1; c += kThreads) {
    const int m = min(kThreads, b1 - c), b = c + tid;
    Need n;
    Sums before;
    const Sums sum = given(c, asked, &n, &before);
    asked = asked + sum;
    const Sums at = scan_before({n.pages, n.fresh}, s_warp, &part);
    if (b < b1) {
      a.q_start[b] = (int)(got.rows + at.rows);
      a.lens_out[b] = n.len + n.fresh;
      s_row[tid] = (int)at.rows;
      s_page[tid] = (int)at.pages;
      s_len[tid] = n.len;
      s_held[tid] = n.held;
      // the page that is filled further
      s_old[tid] = n.fresh > 0 && (n.len & ((1 << a.shift) - 1)) ? a.page_table[(size_t)b * a.width + (n.len >> a.shift)] : -1;
    }
    __syncthreads();
    const int top = count - 1 - (int)got.pages;  // the run's first page on the stack
    for (int i = tid; i < (int)part.pages; i += kThreads) {
      const int s = find(s_page, m, i);
      const int page = a.free_pages[top - i];
      if (page < 0 || page >= a.num_pages) bad = true;
      a.page_table[(size_t)(c + s) * a.width + s_held[s] + (i - s_page[s])] = page;
    }
    for (int i = tid; i < (int)part.rows; i += kThreads) {
      const int s = find(s_row, m, i);
      const int pos = s_len[s] + (i - s_row[s]);
      const int j = (pos >> a.shift) - s_held[s];
      const int page = j < 0 ? s_old[s] : a.free_pages[top - (s_page[s] + j)];
      const bool ok = page >= 0 && page < a.num_pages;
      if (!ok) bad = true;
      a.positions[got.rows + i] = pos;
      a.slots[got.rows + i] = ok ? ((int64_t)page << a.shift) + (pos & ((1 << a.shift) - 1)) : -1;
    }
    got = got + part;
    __syncthreads();
  }
  for (long long i = all.rows + rank * kThreads + tid; i < a.rows; i += ranks * kThreads) {
    a.positions[i] = -1;
    a.slots[i] = -1;
  }
  if (bad) atomicExch(a.status, MOE_ERR_INVALID_ARG);
  cluster.sync();  // no CTA leaves while another still reads its sums
}

__global__ void __launch_bounds__(kThreads) release_kernel(PagesArgs a) {
  __shared__ Sums s_warp[kThreads / 32], s_part;
  __shared__ int s_page[kThreads];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  grid_dep_launch();
  grid_dep_wait();
  const int run = (a.B + ranks - 1) / ranks;
  const int b0 = min(rank * run, a.B), b1 = min(b0 + run, a.B);
  bool bad = false;
  const int stack = a.free_state[0];
  if (tid < kThreads / 32) s_warp[tid] = {0, 0};
  auto pages_of = [&](int b) {
    if (b >= b1 || !a.done[b]) return 0;
    const int len = a.lens[b];
    if (len < 0 || len > ((long long)a.width << a.shift)) {
      bad = true;
      return 0;
    }
    return (len + (1 << a.shift) - 1) >> a.shift;
  };
  Sums mine{0, 0}, all, part;
  for (int c = b0; c < b1; c += kThreads) {
    scan_before({pages_of(c + tid), 0}, s_warp, &part);
    mine = mine + part;
  }
  Sums to = cluster_before(cluster, mine, &s_part, &all);
  // a stack that cannot hold them all takes none: all conversations stay as they are
  const bool fits = stack >= 0 && stack <= a.capacity && all.pages <= a.capacity - stack;
  if (!fits) bad = true;
  for (int c = b0; c < b1; c += kThreads) {
    const int m = min(kThreads, b1 - c), b = c + tid;
    const int n = pages_of(b);
    const Sums at = scan_before({n, 0}, s_warp, &part);
    if (b < b1) {
      const int len = a.lens[b];
      s_page[tid] = (int)at.pages;
      a.lens_out[b] = fits && n > 0 ? 0 : len;  // (one of no tokens stays one)
    }
    __syncthreads();
    for (int i = tid; fits && i < (int)part.pages; i += kThreads) {
      const int s = find(s_page, m, i);
      const int page = a.page_table[(size_t)(c + s) * a.width + (i - s_page[s])];
      if (page < 0 || page >= a.num_pages) bad = true;
      a.free_pages[stack + to.pages + i] = page;
    }
    to = to + part;
    __syncthreads();
  }
  if (rank == 0 && tid == 0) {
    a.free_out[0] = stack + (fits ? (int)all.pages : 0);
    a.free_out[1] = 0;
  }
  if (bad) atomicExch(a.status, MOE_ERR_INVALID_ARG);
  cluster.sync();
}

template <class K>
cudaError_t launch(K kernel, const PagesArgs& a, int ranks, cudaStream_t s) {
  PdlLaunch L(dim3(ranks), dim3(kThreads), 0, s);
  cudaLaunchAttribute attr[2];
  attr[0] = L.attr[0];
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  L.cfg.attrs = attr;
  L.cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&L.cfg, kernel, a);
}

}  // namespace

cudaError_t launch_kv_pages_extend(const PagesArgs& a, cudaStream_t s) {
  return launch(extend_kernel, a, a.B <= kThreads && a.rows <= kThreads ? 1 : kMaxCluster, s);
}

cudaError_t launch_kv_pages_release(const PagesArgs& a, cudaStream_t s) {
  return launch(release_kernel, a, a.B <= 128 ? 1 : kMaxCluster, s);
}

}  // namespace moe
