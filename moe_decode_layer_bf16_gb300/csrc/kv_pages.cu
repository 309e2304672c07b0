// Pages of the cache given to a step's new tokens and taken back, on the GPU: block
// tables, row starts, positions and slots from the requests' lengths.
//
// The free pages are a stack.  A sequence's page need is
// ceil((len + new) / P) - ceil(len / P); running sums of the needs say which pages of
// the stack's top it gets, and whether it gets any: once the sums pass what the stack
// holds, no later sequence that needs pages fits either, so nothing has to be decided
// in turn.  Running sums of the rows that are given make q_start.
//
// Every CTA forms the running sums for itself (a thread each for up to 512 sequences at a
// time) and writes its share of the rows and pages, a thread each, which finds its sequence
// among the sums by bisection: coalesced, and even whatever the lengths are.  What a step
// in place overwrites (lengths, the stack's count) is written by the last CTA to have read
// it.  Bound by latency, a launch and three dependent reads: 64 sequences with a token each
// 3.3 us, 300 with 1 to 4096 new ones (151000 rows asked for) 6.0; 500 given back 4.3.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "../../include/moe_decode.h"

namespace moe {

namespace {

constexpr int kMaxThreads = 512;

struct Sums {
  long long pages, rows;
};

MOE_DEV Sums operator+(const Sums& a, const Sums& b) { return {a.pages + b.pages, a.rows + b.rows}; }

MOE_DEV Sums scan_warp(Sums v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums w{__shfl_up_sync(0xffffffffu, v.pages, o), __shfl_up_sync(0xffffffffu, v.rows, o)};
    if (lane >= o) v = v + w;
  }
  return v;
}

// The sum over the threads before this one; *all gets the sum over the CTA.
MOE_DEV Sums scan_before(Sums v, Sums* s_warp, Sums* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  Sums up = scan_warp(v);
  __syncthreads();  // (s_warp may still be read)
  if (lane == 31) s_warp[warp] = up;
  __syncthreads();
  const Sums w = scan_warp(lane < warps ? s_warp[lane] : Sums{0, 0});
  *all = {__shfl_sync(0xffffffffu, w.pages, 31), __shfl_sync(0xffffffffu, w.rows, 31)};
  const int from = warp > 0 ? warp - 1 : 0;
  const Sums before{__shfl_sync(0xffffffffu, w.pages, from), __shfl_sync(0xffffffffu, w.rows, from)};
  up = {up.pages - v.pages, up.rows - v.rows};
  return warp > 0 ? up + before : up;
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

// Whether this CTA is the last of the grid to come here.
MOE_DEV bool last_to_come(int* ticket) {
  __shared__ bool s_last;
  if (gridDim.x == 1) {
    __syncthreads();
    return true;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    s_last = atom_add_acq_rel(ticket, 1) == (int)gridDim.x - 1;
    if (s_last) *ticket = 0;  // ready for the next call
  }
  __syncthreads();
  return s_last;
}

// A sequence's tokens held and asked for, pages held and needed.
struct Need {
  int len, fresh, held, pages;
};

__global__ void __launch_bounds__(kMaxThreads) extend_kernel(PagesArgs a) {
  __shared__ Sums s_warp[kMaxThreads / 32];
  __shared__ int s_row[kMaxThreads], s_page[kMaxThreads];  // rows and pages before each sequence, from the first one's
  __shared__ int s_len[kMaxThreads], s_old[kMaxThreads], s_held[kMaxThreads];
  const int tid = threadIdx.x, threads = blockDim.x, page_tokens = 1 << a.shift;
  grid_dep_launch();
  grid_dep_wait();
  bool bad = false;
  const int stack = a.free_state[0];
  const int count = stack < 0 || stack > a.capacity ? 0 : stack;
  if (count != stack) bad = true;
  // the sequences from b0 on, a thread each: what this thread's asks for and gets
  Sums asked{0, 0}, got{0, 0};  // before these sequences
  auto sequences = [&](int b0, Sums* at, Sums* part) {
    Need n{0, 0, 0, 0};
    if (b0 + tid < a.B) {
      n.len = a.lens[b0 + tid];
      n.fresh = a.fresh[b0 + tid];
      if (n.len < 0 || n.fresh < 0 || (long long)n.len + n.fresh > (long long)a.width << a.shift) {
        bad = true;
        n.fresh = 0;
      } else {
        n.held = (n.len + page_tokens - 1) >> a.shift;
        n.pages = ((n.len + n.fresh + page_tokens - 1) >> a.shift) - n.held;
      }
    }
    *at = scan_before({n.pages, n.fresh}, s_warp, part);
    const bool room = n.fresh == 0 || asked.rows + at->rows + n.fresh <= a.rows;
    const bool fits = n.pages == 0 || asked.pages + at->pages + n.pages <= count;
    if (!room) bad = true;
    asked = asked + *part;
    if (__syncthreads_or(!room || !fits)) {  // not all of them are served
      if (!room || !fits) n.fresh = n.pages = 0;
      *at = scan_before({n.pages, n.fresh}, s_warp, part);
    }
    return n;
  };
  Need n;
  Sums at, part;
  for (int b0 = 0; b0 < a.B; b0 += threads) {
    const int m = min(threads, a.B - b0);
    n = sequences(b0, &at, &part);
    if (tid < m) {
      s_row[tid] = (int)at.rows;
      s_page[tid] = (int)at.pages;
      s_len[tid] = n.len;
      s_held[tid] = n.held;
      // the page that is filled further
      s_old[tid] = n.fresh > 0 && (n.len & (page_tokens - 1)) ? a.page_table[(size_t)(b0 + tid) * a.width + (n.len >> a.shift)] : -1;
    }
    __syncthreads();
    const int top = count - 1 - (int)got.pages;  // these sequences' first page on the stack
    const int first = blockIdx.x * threads + tid, step = gridDim.x * threads;
    for (int i = first; i < (int)part.pages; i += step) {
      const int s = find(s_page, m, i);
      const int page = a.free_pages[top - i];
      if (page < 0 || page >= a.num_pages) bad = true;
      a.page_table[(size_t)(b0 + s) * a.width + s_held[s] + (i - s_page[s])] = page;
    }
    for (int i = first; i < (int)part.rows; i += step) {
      const int s = find(s_row, m, i);
      const int pos = s_len[s] + (i - s_row[s]);
      const int j = (pos >> a.shift) - s_held[s];
      const int page = j < 0 ? s_old[s] : a.free_pages[top - (s_page[s] + j)];
      const bool ok = page >= 0 && page < a.num_pages;
      if (!ok) bad = true;
      a.positions[got.rows + i] = pos;
      a.slots[got.rows + i] = ok ? ((int64_t)page << a.shift) + (pos & (page_tokens - 1)) : -1;
    }
    got = got + part;
    if (b0 + threads < a.B) __syncthreads();
  }
  for (long long i = got.rows + blockIdx.x * threads + tid; i < a.rows; i += gridDim.x * threads) {
    a.positions[i] = -1;
    a.slots[i] = -1;
  }
  if (bad) atomicExch(a.status, MOE_ERR_INVALID_ARG);
  if (!last_to_come(a.ticket)) return;
  if (tid == 0) {
    a.free_out[0] = stack - (int)got.pages;
    a.free_out[1] = (int)min(asked.pages - got.pages, (long long)INT32_MAX);
    a.q_start[a.B] = (int)got.rows;
  }
  const bool once = a.B <= threads;  // this thread's sequence is still in hand
  asked = got = {0, 0};
  for (int b0 = 0; b0 < a.B; b0 += threads) {
    if (!once) n = sequences(b0, &at, &part);
    if (b0 + tid < a.B) {
      a.q_start[b0 + tid] = (int)(got.rows + at.rows);
      a.lens_out[b0 + tid] = n.len + n.fresh;
    }
    got = got + part;
  }
}

__global__ void __launch_bounds__(kMaxThreads) release_kernel(PagesArgs a) {
  __shared__ Sums s_warp[kMaxThreads / 32];
  __shared__ int s_page[kMaxThreads];
  const int tid = threadIdx.x, threads = blockDim.x;
  grid_dep_launch();
  grid_dep_wait();
  bool bad = false;
  const int stack = a.free_state[0];
  auto pages_of = [&](int b) {
    if (b >= a.B || !a.done[b]) return 0;
    const int len = a.lens[b];
    if (len < 0 || len > ((long long)a.width << a.shift)) {
      bad = true;
      return 0;
    }
    return (len + (1 << a.shift) - 1) >> a.shift;
  };
  const bool once = a.B <= threads;
  Sums all{0, 0}, to{0, 0}, at, part;
  int n = 0;
  for (int b0 = 0; b0 < a.B; b0 += threads) {
    n = pages_of(b0 + tid);
    at = scan_before({n, 0}, s_warp, &part);
    all = all + part;
  }
  // a stack that cannot hold them all takes none: all sequences stay as they are
  const bool fits = stack >= 0 && stack <= a.capacity && all.pages <= a.capacity - stack;
  if (!fits) bad = true;
  for (int b0 = 0; fits && b0 < a.B; b0 += threads) {
    const int m = min(threads, a.B - b0);
    if (!once) {
      n = pages_of(b0 + tid);
      at = scan_before({n, 0}, s_warp, &part);
    }
    if (tid < m) s_page[tid] = (int)at.pages;
    __syncthreads();
    for (int i = blockIdx.x * threads + tid; i < (int)part.pages; i += gridDim.x * threads) {
      const int s = find(s_page, m, i);
      const int page = a.page_table[(size_t)(b0 + s) * a.width + (i - s_page[s])];
      if (page < 0 || page >= a.num_pages) bad = true;
      a.free_pages[stack + to.pages + i] = page;
    }
    to = to + part;
    if (!once) __syncthreads();
  }
  if (bad) atomicExch(a.status, MOE_ERR_INVALID_ARG);
  if (!last_to_come(a.ticket)) return;
  if (tid == 0) {
    a.free_out[0] = stack + (fits ? (int)all.pages : 0);
    a.free_out[1] = 0;
  }
  for (int b = tid; b < a.B; b += threads) {
    const int len = a.lens[b], pages = once ? n : pages_of(b);
    a.lens_out[b] = fits && pages > 0 ? 0 : len;  // (one of no tokens stays one)
  }
}

// Fewer threads' sums are formed sooner (64 sequences, a token each: 256 threads 3.3 us, 1024
// 4.3; 500 sequences given back: 512 threads 4.4 us, 1024 4.9).
int threads_for(int B, long long each) { return B <= 256 && each <= 1024 ? 256 : kMaxThreads; }

// Up to a CTA an SM, all of which form the sums (300 sequences' 151000 rows on the GPU's 152 SMs
// 6.0 us, with 148 CTAs 10.7).
template <class K>
cudaError_t launch(K kernel, const PagesArgs& a, long long each, int sms, cudaStream_t s) {
  const int threads = threads_for(a.B, each);
  const int ctas = (int)std::min<long long>(sms, std::max<long long>(1, (each + threads - 1) / threads));
  PdlLaunch L(dim3(ctas), dim3(threads), 0, s);
  return cudaLaunchKernelEx(&L.cfg, kernel, a);
}

}  // namespace

cudaError_t launch_kv_pages_extend(const PagesArgs& a, int sms, cudaStream_t s) {
  return launch(extend_kernel, a, a.rows, sms, s);
}

// (how many pages there are is not known here: a quarter of the table's entries, say)
cudaError_t launch_kv_pages_release(const PagesArgs& a, int sms, cudaStream_t s) {
  return launch(release_kernel, a, (long long)a.B * a.width / 4, sms, s);
}

}  // namespace moe
