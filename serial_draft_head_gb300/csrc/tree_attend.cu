// tree_attend.cu -- attention of drafted rows over a paged cache.
//
// Per row and head, over the visible keys j: s_j = scale q.k_j (capped:
// c tanh(s_j / c)), out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m) with the
// running maximum m, in one pass over K and V.  One block per (row, head):
// scores of 128 keys at a time, one key a thread, then the values, one element
// a thread.
#include <math.h>

#include "tree_common.cuh"

namespace dspark {
namespace tree {
namespace {

constexpr int kThreads = 128;

__device__ float block_max(float x, float* red) {
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
  __syncthreads();
  x = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  __syncthreads();
  return x;
}

__device__ float block_sum(float x, float* red) {
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
  __syncthreads();
  x = red[0] + red[1] + red[2] + red[3];
  __syncthreads();
  return x;
}

template <bool F16, bool E4M3>
__device__ __forceinline__ float element(const uint8_t* row, int i) {
  if (!E4M3) return to_float<F16>(reinterpret_cast<const uint16_t*>(row)[i]);
  return e4m3x2_to_float2(row[i]).x;
}

template <bool F16, bool E4M3>
__global__ void __launch_bounds__(kThreads) attend_kernel(const AttendArgs a) {
  __shared__ float q[DSPARK_TREE_MAX_HEAD_DIM], p[kThreads], red[4];
  __shared__ const uint8_t* vrow[kThreads];
  __shared__ float vscale[kThreads];
  __shared__ bool see_key[kThreads];
  const int n = blockIdx.x, head = blockIdx.y, kvh = head / a.G, tid = threadIdx.x;
  int lo = 0, hi = a.b.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.b.first[mid] <= n) lo = mid;
    else hi = mid - 1;
  }
  int row0, rows, start;
  const bool ok = request_rows(a.b, lo, &row0, &rows, &start) && rows <= a.max_nodes &&
                  (!a.mask || rows <= 32 * a.mask_words);
  if (!ok) {
    if (tid == 0) set_status(a.status, DSPARK_EPAGES);
    return;
  }
  if (n < row0 || n >= row0 + rows) return;
  const int node = n - row0, total = start + rows;
  if (tid < a.D)
    q[tid] = to_float<F16>(
        reinterpret_cast<const uint16_t*>(a.q + n * a.q_row + head * a.q_head)[tid]);
  __syncthreads();
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int t0 = 0; t0 < total; t0 += kThreads) {
    const int pos = t0 + tid;
    bool see = pos < total;
    if (see && pos >= start) {
      const int j = pos - start;
      see = a.mask ? (a.mask[n * a.mask_stride + j / 32] >> (j % 32)) & 1 : j <= node;
    }
    float s = -INFINITY;
    if (see) {
      int64_t page;
      int slot;
      if (locate(a.c, a.b, lo, pos, &page, &slot)) {
        const uint8_t* k = a.c.k + page * a.c.kst[0] + slot * a.c.kst[1] + kvh * a.c.kst[2];
        vrow[tid] = a.c.v + page * a.c.vst[0] + slot * a.c.vst[1] + kvh * a.c.vst[2];
        float x = 0.f;
        for (int i = 0; i < a.D; ++i) x += q[i] * element<F16, E4M3>(k, i);
        vscale[tid] = 1.f;
        if (E4M3) {
          x *= scale_value(a.c.ks[page * a.c.ksst[0] + slot * a.c.ksst[1] + kvh * a.c.ksst[2]]);
          vscale[tid] =
              scale_value(a.c.vs[page * a.c.vsst[0] + slot * a.c.vsst[1] + kvh * a.c.vsst[2]]);
        }
        s = x * a.scale;
        if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
      } else {
        set_status(a.status, DSPARK_EPAGES);
        see = false;
      }
    }
    see_key[tid] = see;
    const float m_new = fmaxf(m, block_max(s, red));
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    p[tid] = see ? expf(s - m_use) : 0.f;
    const float back = expf(m - m_use);
    l = l * back + block_sum(p[tid], red);
    acc *= back;
    if (tid < a.D)
      for (int i = 0; i < kThreads; ++i)
        if (see_key[i]) acc += p[i] * (element<F16, E4M3>(vrow[i], tid) * vscale[i]);
    m = m_new;
    __syncthreads();
  }
  if (tid < a.D) {
    const float o = l == 0.f ? 0.f : acc / l;
    a.out[((int64_t)n * a.Hq + head) * a.D + tid] = (uint16_t)pack2<F16>(o, 0.f);
  }
  if (a.lse && tid == 0) a.lse[(int64_t)n * a.Hq + head] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t attend_launch(const AttendArgs& a, bool f16, bool e4m3, cudaStream_t stream) {
  const dim3 grid(a.b.N, a.Hq);
  if (f16 && e4m3) attend_kernel<true, true><<<grid, kThreads, 0, stream>>>(a);
  else if (f16) attend_kernel<true, false><<<grid, kThreads, 0, stream>>>(a);
  else if (e4m3) attend_kernel<false, true><<<grid, kThreads, 0, stream>>>(a);
  else attend_kernel<false, false><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace tree
}  // namespace dspark
