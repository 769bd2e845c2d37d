// tree_cache.cu -- writing rows into the paged cache, reading them back, and
// moving the accepted path's rows to the front of the draft.
//
// All three are copies: bytes moved over the memory rate bounds them (small
// calls: a launch and three dependent loads).  A row (one token, one head, K or
// V) is handled by the lanes that its 16-byte chunks need, a power of two, so a
// row's largest magnitude is a few shuffles; every thread has kBatch rows in
// flight before it works on the first.  Request and page of a token are looked
// up once per token and block, into shared memory.
//
// Prompts of 901 to 8,191 tokens (26,600 in all, 8 heads of 128) written as e4m3:
// 33.1 us, 5.0 TB/s of bytes read and written; 46,800 tokens read back: 51.3 us, 5.6.
// Writing is issued at 55% of the slots: a lane takes two chunks of the row, so that
// what a row costs beside its elements is spread over 16 of them (one chunk: 43.4).
// 16-bit, 36,900 tokens: 49.6 us written, 50.8 read, 6.1 and 5.9 TB/s.  128 tokens take
// 2.7 us on the device (16-bit 2.3), a path of 17 rows in each of 128 requests 7 us with
// the call: launches.  54,800 tokens as e2m1: 56 us written, 5.1 TB/s (62% of the issue slots),
// 53.5 read, 5.4.
#include "tc_ptx.cuh"
#include "tree_codes.cuh"

namespace dspark {
namespace tree {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 16;        // tokens per block
constexpr int kBatch = 2;          // rows in flight a thread

struct Token {
  int page, slot;                  // page -1: left out
};

// The block's tokens n0 .. n0 + n_tok - 1.  All threads look at all requests, each by
// itself, so that one whose numbers do not fit hides no other and is reported if it
// has no rows, too; a token's request is the one that holds its row (the last, if
// ranges overlap).
__device__ __forceinline__ void find_tokens(const RowsArgs& a, int n0, int n_tok, Token* toks) {
  __shared__ int owner[kMaxTok];
  if ((int)threadIdx.x < n_tok) owner[threadIdx.x] = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < a.b.B; b += kThreads) {
    int row0, rows, start;
    if (request_rows(a.b, b, &row0, &rows, &start)) {
      const int end = min(row0 + rows, n0 + n_tok);
      for (int n = max(row0, n0); n < end; ++n) atomicMax(&owner[n - n0], b);
    } else if (blockIdx.x == 0) {
      set_status(a.status, DSPARK_EPAGES);
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < n_tok) {
    const int b = owner[threadIdx.x];
    Token t{-1, 0};
    if (b >= 0) {                                  // else a row of no request
      int64_t page;
      const int pos = a.b.start[b] + (n0 + (int)threadIdx.x - a.b.first[b]);
      if (locate(a.c, a.b, b, pos, &page, &t.slot)) t.page = (int)page;
      else set_status(a.status, DSPARK_EPAGES);
    }
    toks[threadIdx.x] = t;
  }
  __syncthreads();
}

// Row r of the block: token r / (2 Hkv), then head, then K or V.
struct Place {
  int tok, head;
  bool v, on;
  Token t;
};

__device__ __forceinline__ Place place_of_row(const RowsArgs& a, int r, int rows,
                                              const Token* toks) {
  Place p;
  const int rr = min(r, rows - 1);
  p.tok = a.kv2.div(rr);
  const int hk = rr - p.tok * 2 * a.Hkv;
  p.head = hk >> 1;
  p.v = hk & 1;
  p.t = toks[p.tok];
  p.on = r < rows && p.t.page >= 0;
  return p;
}

// LANES lanes a row, 16 bytes of the cache each (8 elements, or 16 codes; e2m1: 8
// bytes, 16 codes).
template <bool F16, Held HELD, int LANES>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ RowsArgs a,
                                                         int tok) {
  __shared__ Token toks[kMaxTok];
  constexpr int kGroups = kThreads / LANES;
  constexpr int kLoads = HELD == k16 ? 1 : 2;      // 16-byte chunks of the row a lane
  // rows in flight: one where the work on a block of e2m1 hides the next loads by itself
  // (54,800 tokens: 1 56.5 us, 2 58.5, 3 59.0)
  constexpr int kRows = HELD == kE2M1 ? 1 : kBatch;
  const int n0 = blockIdx.x * tok;
  const int n_tok = min(tok, a.b.N - n0);
  find_tokens(a, n0, n_tok, toks);
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const bool in_row = lane * 8 * kLoads < a.D;
  const int rows = n_tok * a.Hkv * 2;
  // whole warps stay in the loop: the shuffles need every lane
  for (int r0 = 0; r0 < rows; r0 += kGroups * kRows) {
    uint4 x[kRows][kLoads];
    Place p[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      p[i] = place_of_row(a, r0 + group + i * kGroups, rows, toks);
      const uint4* src = reinterpret_cast<const uint4*>(
                             a.src[p[i].v] + (int64_t)(n0 + p[i].tok) * a.src_row[p[i].v] +
                             p[i].head * a.src_head[p[i].v]) + lane * kLoads;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        x[i][k] = make_uint4(0, 0, 0, 0);
        if (p[i].on && in_row) x[i][k] = __ldg(src + k);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      uint8_t* dst = a.c.x[p[i].v].at(p[i].t.page, p[i].t.slot, p[i].head);
      if (HELD == k16) {
        if (p[i].on && in_row) reinterpret_cast<uint4*>(dst)[lane] = x[i][0];
        continue;
      }
      if constexpr (HELD != k16) {
        const uint32_t w[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w,
                               x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
        store_codes<F16, HELD, LANES>(w, dst, a.c.scale[p[i].v].at(p[i].t.page, p[i].t.slot, p[i].head),
                                      lane, p[i].on && in_row, p[i].on);
      }
    }
  }
}

// LANES lanes a row, as they write it; e2m1: a lane has eight elements of the row's first
// part and eight of its second, so that each store of a warp fills whole sectors (prompts
// of 54,800 tokens read back: 53.9 us,
// 60.0 with sixteen next to each other).
template <bool F16, Held HELD, int LANES>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ RowsArgs a,
                                                        int tok) {
  __shared__ Token toks[kMaxTok];
  constexpr int kGroups = kThreads / LANES;
  constexpr int kEach = HELD == k16 ? 8 : 16;
  const int n0 = blockIdx.x * tok;
  const int n_tok = min(tok, a.b.N - n0);
  find_tokens(a, n0, n_tok, toks);
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  if (lane * (HELD == kE2M1 ? 8 : kEach) >= a.D) return;
  const bool upper = (LANES + lane) * 8 < a.D;     // e2m1: there is a second part
  const int rows = n_tok * a.Hkv * 2;
  for (int r0 = 0; r0 < rows; r0 += kGroups * kBatch) {
    uint4 x[kBatch];
    uint32_t byte[kBatch];
    Place p[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      p[i] = place_of_row(a, r0 + group + i * kGroups, rows, toks);
      byte[i] = 127;
      if (p[i].on) {
        const uint8_t* src = a.c.x[p[i].v].at(p[i].t.page, p[i].t.slot, p[i].head);
        const uint8_t* scale = a.c.scale[p[i].v].at(p[i].t.page, p[i].t.slot, p[i].head);
        if (HELD == kE2M1) {
          const uint32_t* codes = reinterpret_cast<const uint32_t*>(src) + lane;
          x[i] = make_uint4(__ldg(codes), upper ? __ldg(codes + LANES) : 0u, 0, 0);
          byte[i] = __ldg(scale + lane / 2);
          if (upper) byte[i] |= (uint32_t)__ldg(scale + (LANES + lane) / 2) << 8;
        } else {
          x[i] = ptx::ldg_nc_na(src + lane * 16);
          if (HELD == kE4M3) byte[i] = __ldg(scale);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (!p[i].on) continue;
      uint16_t* out = a.out[p[i].v] + ((int64_t)(n0 + p[i].tok) * a.Hkv + p[i].head) * a.D;
      uint4* dst = reinterpret_cast<uint4*>(out + lane * kEach);
      if (HELD == k16) {
        *dst = x[i];
        continue;
      }
      if constexpr (HELD == kE2M1) {
        // every value is exact in f16, and the bf16 that it becomes is exact too
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t s2 = (byte[i] >> (8 * h) & 0xffu) * 0x00800080u;
          const uint4 c = e2m1x8_to_f16(h ? x[i].y : x[i].x);
          uint32_t y[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            y[k] = mul_f16x2(y[k], s2);
            if (!F16) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y[k]));
              y[k] = pack2<false>(f.x, f.y);
            }
          }
          if (h == 0 || upper)
            reinterpret_cast<uint4*>(out)[h * LANES + lane] = make_uint4(y[0], y[1], y[2], y[3]);
        }
        continue;
      }
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint2 y[4];
      if (easy_scale<F16>(byte[i])) {
        const uint32_t m = scale_mul2<F16>(byte[i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          y[k] = scale_codes<F16>(w[k], m);
          if (!F16) y[k] = swap_middle(y[k]);
        }
      } else {
        const float s = scale_value(byte[i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 lo = e4m3x2_to_float2(w[k] & 0xffffu), hi = e4m3x2_to_float2(w[k] >> 16);
          y[k] = make_uint2(pack2<F16>(saturate16<F16>(lo.x * s), saturate16<F16>(lo.y * s)),
                            pack2<F16>(saturate16<F16>(hi.x * s), saturate16<F16>(hi.y * s)));
        }
      }
      dst[0] = make_uint4(y[0].x, y[0].y, y[1].x, y[1].y);
      dst[1] = make_uint4(y[2].x, y[2].y, y[3].x, y[3].y);
    }
  }
}

// N is at least 1, and up to 2^31 - 1.
int blocks_of(const RowsArgs& a, int tok) { return (a.b.N - 1) / tok + 1; }

// Tokens per block: 16 where that still gives every SM four blocks, fewer for
// small calls, so that their rows spread over the SMs, as long as a block's
// threads all have a row.  Device time, spread / 16 a block: 128 tokens of 16 rows
// written 2.7 / 5.7 us; with one token of 4 rows a block 1,000 tokens took 3.6 us to
// read, with 16 2.6.
int tokens_per_block(const RowsArgs& a, int lanes, int sm_count) {
  const int pass = kThreads / lanes;             // rows
  int tok = kMaxTok;
  while (tok > 1 && blocks_of(a, tok) < 4 * sm_count && tok / 2 * 2 * a.Hkv >= pass) tok >>= 1;
  return tok;
}

constexpr int kKeepThreads = 128;
constexpr int kKeepBatch = 8;

// One thread owns 16-byte column `c` of every row it moves and walks the path
// in order.  Row i goes to a slot that is the source of no later row (sources
// ascend strictly, so path[j] >= j > i for j > i), and a source that a row is
// moved onto has been read before by the same thread: loads of a batch come
// before its stores.  So no two threads touch the same bytes and nothing waits.
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const __grid_constant__ KeepArgs a) {
  __shared__ uint2 from[DSPARK_TREE_MAX_NODES], to[DSPARK_TREE_MAX_NODES];   // page, slot
  const int b = blockIdx.x;                        // the grid's long direction
  const int n = a.count[b], start = a.b.start[b];
  bool bad = n < 0 || n > a.max_path || start < 0;
  if (!bad) {
    const int32_t* path = a.path + (int64_t)b * a.path_stride;
    for (int i = threadIdx.x; i < n; i += kKeepThreads) {
      const int x = path[i];
      int64_t page = 0;
      int slot = 0;
      if (x < i || (i > 0 && path[i - 1] >= x) || (int64_t)start + x >= a.b.max_pos) {
        bad = true;
        break;
      }
      bad |= !locate(a.c, a.b, b, start + x, &page, &slot);
      from[i] = make_uint2((uint32_t)page, (uint32_t)slot);
      bad |= !locate(a.c, a.b, b, start + i, &page, &slot);
      to[i] = make_uint2((uint32_t)page, (uint32_t)slot);
    }
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_status(a.status, DSPARK_EPAGES);
    return;
  }
  const int parts = a.row_bytes / 16, chunks = parts * a.Hkv;    // of K; as many of V
  const int c = blockIdx.y * kKeepThreads + threadIdx.x;
  if (c < 2 * chunks) {
    const int v = c >= chunks;
    const int cc = c - v * chunks, head = cc / parts;
    const Rows rows = a.c.x[v];
    uint8_t* base = rows.of_head(head) + (cc - head * parts) * 16;
    for (int i0 = 0; i0 < n; i0 += kKeepBatch) {
      uint4 x[kKeepBatch];
#pragma unroll
      for (int j = 0; j < kKeepBatch; ++j)
        if (i0 + j < n)
          x[j] = *reinterpret_cast<const uint4*>(base + rows.offset(from[i0 + j].x, from[i0 + j].y));
#pragma unroll
      for (int j = 0; j < kKeepBatch; ++j)
        if (i0 + j < n)
          *reinterpret_cast<uint4*>(base + rows.offset(to[i0 + j].x, to[i0 + j].y)) = x[j];
    }
  }
  const int s = c - 2 * chunks;                    // the scale bytes' columns follow
  const int bytes = a.scale_bytes * a.Hkv;         // of K
  if (s >= 0 && s < 2 * bytes) {
    const int v = s >= bytes, ss = s - v * bytes, head = ss / a.scale_bytes;
    const Rows rows = a.c.scale[v];
    uint8_t* base = rows.of_head(head) + (ss - head * a.scale_bytes);
    for (int i0 = 0; i0 < n; i0 += kKeepBatch) {
      uint8_t x[kKeepBatch];
#pragma unroll
      for (int j = 0; j < kKeepBatch; ++j)
        if (i0 + j < n) x[j] = base[rows.offset(from[i0 + j].x, from[i0 + j].y)];
#pragma unroll
      for (int j = 0; j < kKeepBatch; ++j)
        if (i0 + j < n) base[rows.offset(to[i0 + j].x, to[i0 + j].y)] = x[j];
    }
  }
}

template <bool F16, Held HELD, int LANES>
void launch_write(const RowsArgs& a, int sm_count, cudaStream_t stream) {
  const int tok = tokens_per_block(a, LANES, sm_count);
  write_kernel<F16, HELD, LANES><<<blocks_of(a, tok), kThreads, 0, stream>>>(a, tok);
}

template <bool F16, Held HELD, int LANES>
void launch_read(const RowsArgs& a, int sm_count, cudaStream_t stream) {
  const int tok = tokens_per_block(a, LANES, sm_count);
  read_kernel<F16, HELD, LANES><<<blocks_of(a, tok), kThreads, 0, stream>>>(a, tok);
}

// Half the lanes for heads of up to 64 elements: lanes without elements cost as
// much as the others (prompts over e4m3: 19.4 us against 27.8 with those of 128).
template <bool F16, Held HELD>
void write_for(const RowsArgs& a, int sm_count, cudaStream_t stream) {
  constexpr int kEach = HELD == k16 ? 8 : 16;
  if (a.D <= 64) launch_write<F16, HELD, 64 / kEach>(a, sm_count, stream);
  else launch_write<F16, HELD, 128 / kEach>(a, sm_count, stream);
}

template <bool F16, Held HELD>
void read_for(const RowsArgs& a, int sm_count, cudaStream_t stream) {
  constexpr int kEach = HELD == k16 ? 8 : 16;
  if (a.D <= 64) launch_read<F16, HELD, 64 / kEach>(a, sm_count, stream);
  else launch_read<F16, HELD, 128 / kEach>(a, sm_count, stream);
}

}  // namespace

// A 16-bit cache holds the rows' own bits, whichever of the two types.
cudaError_t write_launch(const RowsArgs& a, bool f16, Held held, int sm_count,
                         cudaStream_t stream) {
  if (held == k16) write_for<false, k16>(a, sm_count, stream);
  else if (held == kE4M3 && f16) write_for<true, kE4M3>(a, sm_count, stream);
  else if (held == kE4M3) write_for<false, kE4M3>(a, sm_count, stream);
  else if (f16) write_for<true, kE2M1>(a, sm_count, stream);
  else write_for<false, kE2M1>(a, sm_count, stream);
  return cudaGetLastError();
}

cudaError_t read_launch(const RowsArgs& a, bool f16, Held held, int sm_count,
                        cudaStream_t stream) {
  if (held == k16) read_for<false, k16>(a, sm_count, stream);
  else if (held == kE4M3 && f16) read_for<true, kE4M3>(a, sm_count, stream);
  else if (held == kE4M3) read_for<false, kE4M3>(a, sm_count, stream);
  else if (f16) read_for<true, kE2M1>(a, sm_count, stream);
  else read_for<false, kE2M1>(a, sm_count, stream);
  return cudaGetLastError();
}

cudaError_t keep_launch(const KeepArgs& a, cudaStream_t stream) {
  const int columns = (a.row_bytes / 16 + a.scale_bytes) * a.Hkv * 2;
  const dim3 grid(a.b.B, (columns + kKeepThreads - 1) / kKeepThreads);
  keep_kernel<<<grid, kKeepThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace tree
}  // namespace dspark
