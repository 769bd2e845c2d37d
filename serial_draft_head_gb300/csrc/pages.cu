// pages.cu -- page tables from lengths that stay on the device (dspark_pages.h).
//
// Every block sums the requests' numbers up by itself, four a thread, and then does its
// share of the rows and pages: a row finds its request in the sums by bisection.  What a
// call changes that other blocks read (held, n_free) is written by the block that arrives
// last, after all have read.  One launch, bound by its chain of dependent loads; in a
// replayed graph 16 requests of 8 rows and their way back take 6.6 to 8.0 us, 1,024 requests
// of 128 rows 12.5.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/dspark_pages.h"

namespace dspark {
namespace pages {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = DSPARK_PAGES_MAX_REQUESTS / kThreads;   // requests a thread

struct Sums {
  int rows[DSPARK_PAGES_MAX_REQUESTS + 1];       // of the requests before
  int pages[DSPARK_PAGES_MAX_REQUESTS + 1];      // handed out to them, or taken back
  int length[DSPARK_PAGES_MAX_REQUESTS];         // -1: left out
  int held[DSPARK_PAGES_MAX_REQUESTS];           // before, or (trim) afterwards
  long long warp[2][kThreads / 32];
  int total;                                     // pages
  int last;
  int flagged;
};

// Exclusive sums over the block of two numbers a thread.
__device__ __forceinline__ void scan(Sums& s, long long (&x)[2]) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  long long incl[2] = {x[0], x[1]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long y = __shfl_up_sync(0xffffffffu, incl[k], o);
      if (lane >= o) incl[k] += y;
    }
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (lane == 31) s.warp[k][warp] = incl[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    long long before = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
      if (w < warp) before += s.warp[k][w];
    x[k] = before + incl[k] - x[k];
  }
}

// The request r < n with sum[r] <= i < sum[r + 1], for 0 <= i < sum[n].
__device__ __forceinline__ int find(const int* sum, int n, int i) {
  int lo = 0, hi = n;                            // sum[lo] <= i < sum[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sum[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Whether this block is the last of the grid to get here, and then s.flagged, whether a thread of
// any of them had its flag set: a block that has one counts kFlagged more.
constexpr int kFlagged = 1 << 16;
__device__ __forceinline__ bool arrive_last(Sums& s, int* count, bool flag = false) {
  const bool any = __syncthreads_or(flag);
  if (threadIdx.x == 0) {
    __threadfence();
    const int before = atomicAdd(count, any ? 1 + kFlagged : 1);
    s.last = before % kFlagged == (int)gridDim.x - 1;
    s.flagged = any || before >= kFlagged;
    if (s.last) *count = 0;
  }
  __syncthreads();
  return s.last;
}

__global__ void __launch_bounds__(kThreads) reset_kernel(const dspark_pages p) {
  const int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
  for (int64_t i = i0; i < p.n_pages; i += step) p.free[i] = p.n_pages - 1 - (int)i;
  for (int64_t i = i0; i < (int64_t)p.requests * p.max_pages; i += step)
    p.table[i / p.max_pages * p.table_stride + i % p.max_pages] = -1;
  for (int64_t i = i0; i < p.requests; i += step) p.held[i] = 0;
  if (i0 == 0) {
    *p.n_free = p.n_pages;
    p.state[0] = p.state[1] = 0;
  }
}

struct GrowArgs {
  dspark_pages p;
  const int32_t *length, *count;
  const uint32_t* mask;
  int64_t mask_stride;
  int mask_words, N;
  int32_t *first, *slot, *position;
};

__global__ void __launch_bounds__(kThreads) grow_kernel(const __grid_constant__ GrowArgs a) {
  __shared__ Sums s;
  const dspark_pages& p = a.p;
  const int R = p.requests, page = p.page_size;
  const int counted = *p.n_free;
  const bool miscounted = counted < 0 || counted > p.n_pages;   // then none is handed out
  const int n_free = miscounted ? 0 : counted;
  if (threadIdx.x == 0) s.total = 0;
  int length[kPer], rows[kPer], need[kPer], held[kPer];
  bool bad[kPer], wrong = miscounted;
  long long sum[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = threadIdx.x * kPer + k;
    length[k] = rows[k] = need[k] = held[k] = 0;
    bad[k] = false;
    if (r >= R) continue;
    length[k] = a.length[r];
    rows[k] = a.count[r];
    held[k] = p.held[r];
    const long long end = (long long)length[k] + rows[k];
    bad[k] = length[k] < 0 || rows[k] < 0 || end > (long long)p.max_pages * page || held[k] < 0 ||
             held[k] > p.max_pages;
    rows[k] = max(rows[k], 0);
    if (!bad[k]) need[k] = max((int)((end + page - 1) / page) - held[k], 0);
    sum[0] += rows[k];
    sum[1] += need[k];
  }
  scan(s, sum);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = threadIdx.x * kPer + k;
    const long long before = sum[0];
    sum[0] += rows[k];
    const long long until = sum[1] + need[k];
    if (r < R) {
      // served are those in order up to where the free pages end, and any that need none
      const bool served = need[k] == 0 || until <= n_free;
      const bool fits = sum[0] <= a.N;
      const bool out = bad[k] || !served || !fits;
      wrong |= out;
      // what one that is not served lacks stays in the sums, so nobody overtakes it, and who is
      // served is known from one scan
      s.rows[r] = (int)min(before, (long long)INT_MAX);
      s.pages[r] = (int)min(sum[1], (long long)INT_MAX);
      s.length[r] = bad[k] || !fits ? -1 : length[k];
      s.held[r] = served ? held[k] : -1;
      if (served && need[k] > 0) atomicMax(&s.total, (int)until);
      if (r == R - 1) {
        s.rows[R] = (int)min(sum[0], (long long)INT_MAX);
        s.pages[R] = (int)min(until, (long long)INT_MAX);
      }
    }
    sum[1] = until;
  }
  if (wrong && blockIdx.x == 0) atomicExch(p.state, DSPARK_EPAGES);
  __syncthreads();
  const int i0 = blockIdx.x * kThreads + threadIdx.x, step = gridDim.x * kThreads;
  for (int i = i0; i <= R; i += step) a.first[i] = s.rows[i];
  const int live = s.rows[R];
#pragma unroll 1
  for (int64_t n = i0; n < a.N; n += step) {
    int slot = -1, position = -1;
    if (n < live) {
      const int r = find(s.rows, R, (int)n);
      const int len = s.length[r], old = s.held[r];
      if (len >= 0) {
        const int at = len + ((int)n - s.rows[r]);
        position = at;
        if (a.mask) {
          position = len - 1;
          for (int w = 0; w < a.mask_words; ++w)
            position += __popc(__ldg(a.mask + n * a.mask_stride + w));
        }
        if (old >= 0) {
          const int i = at / page;
          const int pg = i < old ? p.table[r * p.table_stride + i]
                                 : p.free[n_free - 1 - (s.pages[r] + i - old)];
          if (pg >= 0 && pg < p.n_pages) slot = pg * page + (at - i * page);
          else atomicExch(p.state, DSPARK_EPAGES);
        }
      }
    }
    a.slot[n] = slot;
    a.position[n] = position;
  }
  const int total = s.total;
#pragma unroll 1
  for (int64_t i = i0; i < total; i += step) {   // i + step can pass 31 bits
    const int j = (int)i, r = find(s.pages, R, j);
    p.table[r * p.table_stride + s.held[r] + (j - s.pages[r])] = p.free[n_free - 1 - j];
  }
  if (arrive_last(s, p.state + 1)) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int r = threadIdx.x * kPer + k;
      if (r < R && need[k] > 0 && s.held[r] >= 0) p.held[r] = held[k] + need[k];
    }
    if (threadIdx.x == 0 && total > 0) *p.n_free = n_free - total;
  }
}

// Takes the entries below 0 out of x[0 .. n-1], which other blocks wrote; returns how many are
// left.  By one block, chunk by chunk: what a chunk writes lies in it or before it.
__device__ __noinline__ int close_up(Sums& s, int32_t* x, int n) {
  int kept = 0;
  __threadfence();
#pragma unroll 1
  for (int64_t at = 0; at < n; at += kThreads) {
    const int64_t i = at + threadIdx.x;
    const int pg = i < n ? __ldcg(x + i) : -1;
    long long rank[2] = {pg >= 0 ? 1 : 0, 0};
    scan(s, rank);                               // all have read
    if (pg >= 0) x[kept + (int)rank[0]] = pg;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) kept += (int)s.warp[0][w];
    __syncthreads();
  }
  return kept;
}

__global__ void __launch_bounds__(kThreads) trim_kernel(const dspark_pages p, const int32_t* length) {
  __shared__ Sums s;
  const int R = p.requests, page = p.page_size;
  const int n_free = *p.n_free;
  int gone[kPer], keep[kPer];
  bool wrong = false;
  long long sum[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = threadIdx.x * kPer + k;
    gone[k] = keep[k] = 0;
    if (r >= R) continue;
    const int held = p.held[r], len = length[r];
    const bool bad = len < 0 || len > (long long)p.max_pages * page || held < 0 || held > p.max_pages;
    keep[k] = bad ? held : min(held, (int)(((long long)len + page - 1) / page));
    gone[k] = held - keep[k];
    wrong |= bad;
    sum[0] += gone[k];
  }
  scan(s, sum);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = threadIdx.x * kPer + k;
    if (r < R) {
      s.pages[r] = (int)min(sum[0], (long long)INT_MAX);
      s.held[r] = keep[k];
      if (r == R - 1) s.pages[R] = (int)min(sum[0] + gone[k], (long long)INT_MAX);
    }
    sum[0] += gone[k];
  }
  __syncthreads();
  int total = s.pages[R];
  if (n_free < 0 || (long long)n_free + total > p.n_pages) {   // more than there are: nothing
    wrong = true;
    total = 0;
  }
  if (wrong && blockIdx.x == 0) atomicExch(p.state, DSPARK_EPAGES);
  bool lost = false;
#pragma unroll 1
  for (int64_t i = blockIdx.x * kThreads + threadIdx.x; i < total; i += gridDim.x * kThreads) {
    const int j = (int)i, r = find(s.pages, R, j);
    int32_t* entry = p.table + r * p.table_stride + s.held[r] + (j - s.pages[r]);
    const int pg = *entry;
    const bool is = pg >= 0 && pg < p.n_pages;
    lost |= !is;
    // the last to go is the first to be handed out again: the order that they came in
    p.free[n_free + total - 1 - j] = is ? pg : -1;
    *entry = -1;
  }
  if (arrive_last(s, p.state + 1, lost) && total > 0) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int r = threadIdx.x * kPer + k;
      if (r < R && gone[k] > 0) p.held[r] = keep[k];
    }
    int back = total;
    if (s.flagged) back = close_up(s, p.free + n_free, total);
    if (threadIdx.x == 0) {
      *p.n_free = n_free + back;
      if (s.flagged) atomicExch(p.state, DSPARK_EPAGES);
    }
  }
}

bool fine(const dspark_pages* p) {
  return p && p->table && p->held && p->free && p->n_free && p->state && p->requests >= 1 &&
         p->requests <= DSPARK_PAGES_MAX_REQUESTS && p->page_size >= 1 && p->n_pages >= 1 &&
         p->max_pages >= 1 && p->table_stride >= p->max_pages &&
         (int64_t)p->n_pages * p->page_size < ((int64_t)1 << 31) &&
         (int64_t)p->max_pages * p->page_size < ((int64_t)1 << 31);
}

int code(cudaError_t e) { return e == cudaSuccess ? DSPARK_OK : DSPARK_ECUDA; }

// As many blocks as the rows give two a thread; the pages follow them.
int blocks(int64_t items) {
  const int64_t n = (items + 2 * kThreads - 1) / (2 * kThreads);
  return (int)(n < 1 ? 1 : n > 304 ? 304 : n);
}

}  // namespace
}  // namespace pages
}  // namespace dspark

using namespace dspark::pages;

extern "C" {

int dspark_pages_reset(const dspark_pages* p, void* stream) {
  if (!fine(p)) return DSPARK_EINVAL;
  reset_kernel<<<blocks((int64_t)p->requests * p->max_pages + p->n_pages), kThreads, 0,
                 static_cast<cudaStream_t>(stream)>>>(*p);
  return code(cudaGetLastError());
}

int dspark_pages_grow(const dspark_pages* p, const int32_t* length, const int32_t* count, int N,
                      const uint32_t* mask, int64_t mask_stride, int mask_words, int32_t* first,
                      int32_t* slot, int32_t* position, void* stream) {
  if (!fine(p) || !length || !count || !first || N < 0 || (N > 0 && (!slot || !position)))
    return DSPARK_EINVAL;
  if (mask && (mask_words < 1 || mask_stride < 0)) return DSPARK_EINVAL;
  GrowArgs a{*p, length, count, N > 0 ? mask : nullptr, mask_stride, mask_words, N, first, slot, position};
  grow_kernel<<<blocks(N), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return code(cudaGetLastError());
}

int dspark_pages_trim(const dspark_pages* p, const int32_t* length, void* stream) {
  if (!fine(p) || !length) return DSPARK_EINVAL;
  // What goes back is not known here: at most all that can be held, at 16 pages a thread then.
  // 131,072 pages of 16 requests come and go in 17.6 us; with blocks for the requests alone, 1
  // here, their way back takes 213.  Where little goes back (16 pages of 6,400) 2.9 us either way.
  const int64_t most = std::min((int64_t)p->n_pages, (int64_t)p->requests * p->max_pages);
  trim_kernel<<<blocks(std::max((int64_t)4 * p->requests, most / 8)), kThreads, 0,
                static_cast<cudaStream_t>(stream)>>>(*p, length);
  return code(cudaGetLastError());
}

int dspark_pages_status(const dspark_pages* p, void* stream) {
  if (!fine(p)) return DSPARK_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int status = 0;
  cudaError_t e = cudaMemcpyAsync(&status, p->state, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(p->state, 0, sizeof(int), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e == cudaSuccess ? status : DSPARK_ECUDA;
}

}  // extern "C"
