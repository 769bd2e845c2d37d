// tree_cache.cu -- writing rows into the paged cache, reading them back, and
// moving the accepted path's rows to the front of the draft.
//
// All three are copies: bytes moved over the memory rate bounds them.  A row
// (one token, one head, K or V) of D <= 128 elements is handled by 16 lanes
// with 8 elements each, so one 16-byte load a lane brings a 16-bit row, the
// row's largest magnitude is four shuffles, and e4m3 codes leave as 8 bytes a
// lane.  Request and page of a token are looked up once per token and block,
// into shared memory.
#include "tree_common.cuh"

namespace dspark {
namespace tree {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 16;        // tokens per block
constexpr int kLanes = 16;         // lanes per row

struct Token {
  int64_t page;                    // -1: left out
  int slot;
};

// The request of row n is the last b with first[b] <= n.
__device__ __forceinline__ int request_of(const BatchView& q, int n) {
  int lo = 0, hi = q.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(q.first + mid) <= n) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ Token find_token(const RowsArgs& a, int n) {
  Token t{-1, 0};
  const int b = request_of(a.b, n);
  int row0, rows, start;
  if (!request_rows(a.b, b, &row0, &rows, &start)) {
    set_status(a.status, DSPARK_EPAGES);
    return t;
  }
  if (n < row0 || n >= row0 + rows) return t;    // a row of no request
  if (!locate(a.c, a.b, b, start + (n - row0), &t.page, &t.slot)) {
    set_status(a.status, DSPARK_EPAGES);
    t.page = -1;
  }
  return t;
}

__device__ __forceinline__ uint32_t max16(uint32_t x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

template <bool F16, bool E4M3>
__global__ void __launch_bounds__(kThreads) write_kernel(const RowsArgs a, int tok) {
  __shared__ Token toks[kMaxTok];
  const int n0 = blockIdx.x * tok;
  const int n_tok = min(tok, a.b.N - n0);
  if ((int)threadIdx.x < n_tok) toks[threadIdx.x] = find_token(a, n0 + threadIdx.x);
  __syncthreads();
  const int lane = threadIdx.x % kLanes;
  const bool in_row = lane * 8 < a.D;
  const int rows = n_tok * a.Hkv * 2;
  // the warp's two rows stay together: the shuffles need every lane
  for (int r0 = (threadIdx.x / 32) * 2; r0 < rows; r0 += kThreads / kLanes) {
    const int r = r0 + (threadIdx.x / kLanes) % 2;
    const int t = r / (a.Hkv * 2), hk = r % (a.Hkv * 2), head = hk >> 1;
    const bool is_v = hk & 1;
    Token tk{-1, 0};
    if (r < rows) tk = toks[t];
    const bool on = tk.page >= 0;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (on && in_row) {
      const uint8_t* src = is_v ? a.v + (n0 + t) * a.v_row + head * a.v_head
                                : a.k + (n0 + t) * a.k_row + head * a.k_head;
      x = __ldg(reinterpret_cast<const uint4*>(src) + lane);
    }
    const int64_t* st = is_v ? a.c.vst : a.c.kst;
    uint8_t* dst = (is_v ? a.c.v : a.c.k) + tk.page * st[0] + tk.slot * st[1] + head * st[2];
    if (!E4M3) {
      if (on && in_row) reinterpret_cast<uint4*>(dst)[lane] = x;
      continue;
    }
    float f[8];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] = to_float<F16>((uint16_t)(w[i / 2] >> (16 * (i & 1))));
      big = max(big, __float_as_uint(f[i]) & 0x7fffffffu);   // ordered as magnitudes, NaN last
    }
    big = max16(big);
    // a = m 2^x, 448 = 1.75 2^8: e = x - 8, one more where m > 1.75
    const int field = (int)(big >> 23);
    int byte = field - 8 + ((big & 0x7fffffu) > 0x600000u ? 1 : 0);
    byte = field == 255 ? 255 : max(byte, 0);
    const float inv = __uint_as_float((uint32_t)(254 - (byte == 255 ? 127 : byte)) << 23);
    uint32_t code[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_fp8x2_storage_t c2 = __nv_cvt_float2_to_fp8x2(
          make_float2(f[2 * i] * inv, f[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
      code[i / 2] |= (uint32_t)c2 << (16 * (i & 1));
    }
    if (byte == 255) code[0] = code[1] = 0x7f7f7f7fu;
    if (on && in_row) reinterpret_cast<uint2*>(dst)[lane] = make_uint2(code[0], code[1]);
    if (on && lane == 0) {
      const int64_t* ss = is_v ? a.c.vsst : a.c.ksst;
      (is_v ? a.c.vs : a.c.ks)[tk.page * ss[0] + tk.slot * ss[1] + head * ss[2]] = (uint8_t)byte;
    }
  }
}

template <bool F16, bool E4M3>
__global__ void __launch_bounds__(kThreads) read_kernel(const RowsArgs a, int tok) {
  __shared__ Token toks[kMaxTok];
  const int n0 = blockIdx.x * tok;
  const int n_tok = min(tok, a.b.N - n0);
  if ((int)threadIdx.x < n_tok) toks[threadIdx.x] = find_token(a, n0 + threadIdx.x);
  __syncthreads();
  const int lane = threadIdx.x % kLanes;
  if (lane * 8 >= a.D) return;
  const int rows = n_tok * a.Hkv * 2;
  for (int r = threadIdx.x / kLanes; r < rows; r += kThreads / kLanes) {
    const int t = r / (a.Hkv * 2), hk = r % (a.Hkv * 2), head = hk >> 1;
    const bool is_v = hk & 1;
    const Token tk = toks[t];
    if (tk.page < 0) continue;
    const int64_t* st = is_v ? a.c.vst : a.c.kst;
    const uint8_t* src = (is_v ? a.c.v : a.c.k) + tk.page * st[0] + tk.slot * st[1] + head * st[2];
    uint4 y;
    if (E4M3) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(src) + lane);
      const int64_t* ss = is_v ? a.c.vsst : a.c.ksst;
      const float s = scale_value(
          __ldg((is_v ? a.c.vs : a.c.ks) + tk.page * ss[0] + tk.slot * ss[1] + head * ss[2]));
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = e4m3x2_to_float2(((i < 2 ? x.x : x.y) >> (16 * (i & 1))) & 0xffffu);
        w[i] = pack2<F16>(saturate16<F16>(f.x * s), saturate16<F16>(f.y * s));
      }
      y = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      y = __ldg(reinterpret_cast<const uint4*>(src) + lane);
    }
    uint16_t* out = (is_v ? a.out_v : a.out_k) + ((int64_t)(n0 + t) * a.Hkv + head) * a.D;
    reinterpret_cast<uint4*>(out)[lane] = y;
  }
}

// Tokens per block: 16 where that still gives every SM four blocks, fewer for
// small calls, so that their rows spread over the SMs.
int tokens_per_block(int N, int sm_count) {
  int tok = kMaxTok;
  while (tok > 1 && (N + tok - 1) / tok < 4 * sm_count) tok >>= 1;
  return tok;
}

constexpr int kKeepThreads = 128;
constexpr int kKeepBatch = 8;

// One thread owns 16-byte column `c` of every row it moves and walks the path
// in order.  Row i goes to a slot that is the source of no later row (sources
// ascend strictly, so path[j] >= j > i for j > i), and a source that a row is
// moved onto has been read before by the same thread: loads of a batch come
// before its stores.  So no two threads touch the same bytes and nothing waits.
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const KeepArgs a) {
  extern __shared__ int32_t path[];
  __shared__ int bad;
  const int b = blockIdx.y;
  const int n = a.count[b], start = a.b.start[b];
  if (threadIdx.x == 0) bad = n < 0 || n > a.max_path || start < 0;
  __syncthreads();
  if (!bad) {
    const int32_t* p = a.path + (int64_t)b * a.path_stride;
    for (int i = threadIdx.x; i < n; i += kKeepThreads) {
      const int x = p[i];
      path[i] = x;
      int64_t page;
      int slot;
      if (x < 0 || (i > 0 && p[i - 1] >= x) || (int64_t)start + x >= a.b.max_pos ||
          !locate(a.c, a.b, b, start + x, &page, &slot) ||
          !locate(a.c, a.b, b, start + i, &page, &slot))
        bad = 1;
    }
  }
  __syncthreads();
  if (bad) {
    if (threadIdx.x == 0) set_status(a.status, DSPARK_EPAGES);
    return;
  }
  const int chunks = a.row_bytes / 16 * a.Hkv;    // of K; as many of V
  const int c = blockIdx.x * kKeepThreads + threadIdx.x;
  if (c < 2 * chunks) {
    const bool is_v = c >= chunks;
    const int cc = is_v ? c - chunks : c;
    const int head = cc / (a.row_bytes / 16), part = cc % (a.row_bytes / 16);
    const int64_t* st = is_v ? a.c.vst : a.c.kst;
    uint8_t* base = (is_v ? a.c.v : a.c.k) + head * st[2] + part * 16;
    for (int i0 = 0; i0 < n; i0 += kKeepBatch) {
      uint4 x[kKeepBatch];
#pragma unroll
      for (int j = 0; j < kKeepBatch; ++j) {
        if (i0 + j >= n) break;
        int64_t page;
        int slot;
        locate(a.c, a.b, b, start + path[i0 + j], &page, &slot);
        x[j] = *reinterpret_cast<const uint4*>(base + page * st[0] + slot * st[1]);
      }
#pragma unroll
      for (int j = 0; j < kKeepBatch; ++j) {
        if (i0 + j >= n) break;
        int64_t page;
        int slot;
        locate(a.c, a.b, b, start + i0 + j, &page, &slot);
        *reinterpret_cast<uint4*>(base + page * st[0] + slot * st[1]) = x[j];
      }
    }
  }
  const int s = c - 2 * chunks;                    // the scale bytes' columns follow
  if (a.scales && s >= 0 && s < 2 * a.Hkv) {
    const bool is_v = s >= a.Hkv;
    const int head = is_v ? s - a.Hkv : s;
    const int64_t* st = is_v ? a.c.vsst : a.c.ksst;
    uint8_t* base = (is_v ? a.c.vs : a.c.ks) + head * st[2];
    for (int i = 0; i < n; ++i) {
      int64_t page, to;
      int slot, to_slot;
      locate(a.c, a.b, b, start + path[i], &page, &slot);
      locate(a.c, a.b, b, start + i, &to, &to_slot);
      base[to * st[0] + to_slot * st[1]] = base[page * st[0] + slot * st[1]];
    }
  }
}

}  // namespace

cudaError_t write_launch(const RowsArgs& a, bool f16, bool e4m3, int sm_count,
                         cudaStream_t stream) {
  const int tok = tokens_per_block(a.b.N, sm_count);
  const dim3 grid((a.b.N + tok - 1) / tok);
  if (!e4m3) write_kernel<false, false><<<grid, kThreads, 0, stream>>>(a, tok);
  else if (f16) write_kernel<true, true><<<grid, kThreads, 0, stream>>>(a, tok);
  else write_kernel<false, true><<<grid, kThreads, 0, stream>>>(a, tok);
  return cudaGetLastError();
}

cudaError_t read_launch(const RowsArgs& a, bool f16, bool e4m3, int sm_count,
                        cudaStream_t stream) {
  const int tok = tokens_per_block(a.b.N, sm_count);
  const dim3 grid((a.b.N + tok - 1) / tok);
  if (!e4m3) read_kernel<false, false><<<grid, kThreads, 0, stream>>>(a, tok);
  else if (f16) read_kernel<true, true><<<grid, kThreads, 0, stream>>>(a, tok);
  else read_kernel<false, true><<<grid, kThreads, 0, stream>>>(a, tok);
  return cudaGetLastError();
}

cudaError_t keep_launch(const KeepArgs& a, cudaStream_t stream) {
  const int columns = a.row_bytes / 16 * a.Hkv * 2 + (a.scales ? 2 * a.Hkv : 0);
  const dim3 grid((columns + kKeepThreads - 1) / kKeepThreads, a.b.B);
  keep_kernel<<<grid, kKeepThreads, (size_t)a.max_path * sizeof(int32_t), stream>>>(a);
  return cudaGetLastError();
}

}  // namespace tree
}  // namespace dspark
