// tree_common.cuh -- what the draft-check kernels share: the device view of a
// paged cache and of a call's requests, element conversions, and the
// arguments of the launches (tree_cache.cu, tree_attend.cu).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dspark_tree.h"

namespace dspark {
namespace tree {

// n / d for 0 <= n < 2^31 by one multiplication: with L = ceil(log2 d) and
// mul = ceil(2^(31+L) / d) < 2^32, floor(n * mul / 2^(31+L)) is exact.
struct FastDiv {
  uint32_t mul;
  int shift;                 // L
  int d;
  __host__ static FastDiv of(int d) {
    FastDiv f;
    int L = 0;
    while (((int64_t)1 << L) < d) ++L;
    f.shift = L;
    f.mul = (uint32_t)((((uint64_t)1 << (31 + L)) + (uint64_t)d - 1) / (uint64_t)d);
    f.d = d;
    return f;
  }
  __device__ __forceinline__ int div(int n) const {
    return (int)(__umulhi((uint32_t)n << 1, mul) >> shift);
  }
};

// Rows of one array of the cache, strides in bytes.  Those of pages and slots
// are below 2^31, so an offset is two 32 x 32 -> 64 bit products.
struct Rows {
  uint8_t* p;
  int64_t head;
  uint32_t page, slot;
  __device__ __forceinline__ uint8_t* of_head(int h) const { return p + h * head; }
  __device__ __forceinline__ uint64_t offset(uint32_t pg, uint32_t sl) const {
    return (uint64_t)pg * page + (uint64_t)sl * slot;
  }
  __device__ __forceinline__ uint8_t* at(uint32_t pg, uint32_t sl, int h) const {
    return of_head(h) + offset(pg, sl);
  }
};

struct CacheView {
  Rows x[2];                 // K, V
  Rows scale[2];             // their scale bytes, e4m3 only
  int64_t n_pages;
  FastDiv page;
};

struct BatchView {
  const int32_t* pages;
  const int32_t* start;
  const int32_t* first;
  int64_t pages_stride;
  int64_t max_pos;           // max_pages * page_size, at most DSPARK_TREE_MAX_LENGTH
  int B, N;
};

// Status words set by the kernels (any of them: the host reads one word).
__device__ __forceinline__ void set_status(int* status, int code) {
  atomicExch(status, code);
}

// Rows and context length of request b; false if they do not fit the arrays.
__device__ __forceinline__ bool request_rows(const BatchView& q, int b, int* row0, int* rows,
                                             int* start) {
  const int f0 = q.first[b], f1 = q.first[b + 1], s = q.start[b];
  *row0 = f0;
  *rows = 0;
  *start = s;
  if (f0 < 0 || f1 < f0 || f1 > q.N || s < 0 || (int64_t)s + (f1 - f0) > q.max_pos) return false;
  *rows = f1 - f0;
  return true;
}

// Page and slot of position pos (0 <= pos < max_pos) of request b; false if
// the table's entry is no page of the cache.
__device__ __forceinline__ bool locate(const CacheView& c, const BatchView& q, int b, int pos,
                                       int64_t* page, int* slot) {
  const int i = c.page.div(pos);
  *slot = pos - i * c.page.d;
  const int p = __ldg(q.pages + (int64_t)b * q.pages_stride + i);
  *page = p;
  return p >= 0 && p < c.n_pages;
}

// 2^(byte - 127) of a scale byte; 255 is NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}

template <bool F16>
__device__ __forceinline__ float to_float(uint16_t x) {
  return F16 ? __half2float(__ushort_as_half(x)) : __uint_as_float((uint32_t)x << 16);
}

// Two floats to the 16-bit type, nearest even, `lo` in the low half.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Values past the type's range become its largest finite one (NaN stays).
template <bool F16>
__device__ __forceinline__ float saturate16(float x) {
  const float top = F16 ? 65504.f : 3.38953139e38f;
  return fabsf(x) > top ? copysignf(top, x) : x;
}

// Four e4m3 codes as f16, exactly.
__device__ __forceinline__ uint2 e4m3x4_to_f16(uint32_t w) {
  uint2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  return r;
}

// Two e4m3 codes to floats.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) {
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __half22float2(__half2(r));
}

// Four e4m3 codes (bytes 0 .. 3) times 2^(byte - 127) in the 16-bit type, exact
// for the scales of `easy_scale`.  bf16: a code's seven low bits moved to bf16's
// exponent and mantissa fields stand for |code| 2^-120, the sign bit is put on
// after the product; the pairs come as bytes (0, 2) and (1, 3), which needs no
// byte permutation, so elements 1 and 2 of every four change places (attend lays
// Q out the same way, and O's columns change back at the end).
template <bool F16>
__device__ __forceinline__ uint2 scale_codes(uint32_t w, uint32_t mul2) {
  uint2 r;
  if (F16) {
    const uint2 c = e4m3x4_to_f16(w);
    const __half2 m = *reinterpret_cast<const __half2*>(&mul2);
    const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&c.x), m);
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&c.y), m);
    r.x = *reinterpret_cast<const uint32_t*>(&x);
    r.y = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    const uint32_t even = (w << 4) & 0x07f007f0u, odd = (w >> 4) & 0x07f007f0u;
    const __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&mul2);
    const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&even), m);
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&odd), m);
    r.x = *reinterpret_cast<const uint32_t*>(&x) ^ ((w << 8) & 0x80008000u);
    r.y = *reinterpret_cast<const uint32_t*>(&y) ^ (w & 0x80008000u);
  }
  return r;
}

// The order above of four elements (two packed pairs).
__device__ __forceinline__ uint2 swap_middle(uint2 x) {
  return make_uint2(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.x, x.y, 0x7632));
}

// Scales whose product with any code is a finite number of the 16-bit type and
// whose multiplier is one too: 2^(byte - 7) for bf16, 2^(byte - 127) for f16.
template <bool F16>
__device__ __forceinline__ bool easy_scale(uint32_t byte) {
  return byte <= 134 && (!F16 || byte >= 113);
}

template <bool F16>
__device__ __forceinline__ uint32_t scale_mul2(uint32_t byte) {
  return F16 ? (byte - 112) * 0x04000400u : byte * 0x00800080u + 120u * 0x00800080u;
}

struct AttendArgs {
  CacheView c;
  BatchView b;
  const uint8_t* q;
  int64_t q_row, q_head;     // bytes
  const uint32_t* mask;
  int64_t mask_stride;
  int mask_words;
  float scale, softcap;
  uint16_t* out;
  float* lse;
  int Hq, Hkv, G, D;
  int max_nodes;
  FastDiv group;             // by G
  int n_cta;
  // partial results of items that several CTAs share: per CTA two parts of
  // part_rows rows: O (fp32, [D / 4][part_rows][4]) and {m, l} a row
  float* part_o;
  float2* part_ml;
  int4* part_of;             // per part: {request, head, row group, first worker | parts << 16}
  int part_rows;
  int* arrived;              // few rows: parts written of the item whose first is a worker's, 0 between calls
  int* status;
};

// Head dimension as the kernel lays it out, and rows of one part.
// (Half the lanes and columns for heads of up to 64 elements: 64 elements run as
// 64 / as 128, 128 tokens over e4m3 205 / 289 us, 64 x 64 313 / 379 us.)
inline int padded_dim(int D) { return D <= 64 ? 64 : 128; }
constexpr int kGroupRows = 256;    // rows (nodes x heads of one group) of a work item

// Tiled-copy maps of K and V of a 16-bit cache: {D, slot, head, page}, boxes of
// 64 elements by `rows` slots, swizzled.  rows = 0: no map, 16-byte copies.
struct TileMaps {
  CUtensorMap k, v;
  int rows;
};

// Few rows a cached head, on mma.sync (tree_attend_few.cu).
cudaError_t few_setup(bool f16, int D);
cudaError_t few_launch(const AttendArgs& a, bool f16, bool e4m3, cudaStream_t stream);

cudaError_t attend_setup(bool f16, int D);
cudaError_t attend_launch(const AttendArgs& a, const TileMaps& maps, bool f16, bool e4m3,
                          cudaStream_t stream);

// Packed rows of the cache calls: strides in bytes.
struct RowsArgs {
  CacheView c;
  BatchView b;
  const uint8_t* src[2];     // write: K and V rows
  int64_t src_row[2], src_head[2];
  uint16_t* out[2];          // read: destination rows
  int Hkv, D;
  FastDiv kv2;               // by 2 Hkv, the cached rows of a token
  int* status;
};

cudaError_t write_launch(const RowsArgs& a, bool f16, bool e4m3, int sm_count,
                         cudaStream_t stream);
cudaError_t read_launch(const RowsArgs& a, bool f16, bool e4m3, int sm_count,
                        cudaStream_t stream);

struct KeepArgs {
  CacheView c;
  BatchView b;
  const int32_t* path;
  const int32_t* count;
  int64_t path_stride;
  int max_path;
  int Hkv, row_bytes;        // bytes of one head's row
  bool scales;
  int* status;
};

cudaError_t keep_launch(const KeepArgs& a, cudaStream_t stream);

}  // namespace tree
}  // namespace dspark
