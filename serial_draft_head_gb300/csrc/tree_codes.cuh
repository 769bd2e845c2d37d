// tree_codes.cuh -- rows in 16 bits to the codes and scales that the cache holds (the
// header has the rules), by the lanes of a row, 16 elements each.
#pragma once

#include "tree_common.cuh"

namespace dspark {
namespace tree {

// A block of 16 elements to e2m1 codes and its scale byte (the header has the rule).
// x / s only has to fall on the right side of the codes' borders: x has 11 significant
// bits at most and a border times s seven, so x / s is on a border or 2^-13 away from
// it, and the product by fl(1 / s), off by 2^-21, rounded to a multiple of 2^-16 (by
// adding 192 and taking it off again) is on the border or the same side of it.
template <bool F16>
__device__ __forceinline__ uint2 block_to_e2m1(const uint32_t (&w)[8], uint32_t* byte) {
  uint32_t big2 = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) big2 = __vmaxu2(big2, w[k] & 0x7fff7fffu);
  const uint32_t big = __float_as_uint(to_float<F16>((uint16_t)max(big2 & 0xffffu, big2 >> 16)));
  const bool bad = big >= 0x7f800000u;
  *byte = bad ? 255u : e2m1_scale_byte(big);
  const float s = __half2float(__ushort_as_half((uint16_t)(*byte << 7)));
  const float inv = *byte == 0 || bad ? 0.f : 1.f / s;
  uint32_t code[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint16_t x = (uint16_t)(w[4 * h + k / 2] >> (16 * (k & 1)));
      y[k] = fmaf(to_float<F16>(x), inv, 192.f) - 192.f;
    }
    code[h] = float8_to_e2m1(y);
  }
  return bad ? make_uint2(0u, 0u) : make_uint2(code[0], code[1]);
}

// The 16 elements w of lane `lane` of a row (zeros past its end) as codes to `dst`, the
// row's place, and its scales to `scale`; LANES lanes a row, all of them here.  in_row:
// the lane has elements to store; on: the row is stored.
template <bool F16, Held HELD, int LANES>
__device__ __forceinline__ void store_codes(const uint32_t (&w)[8], uint8_t* dst, uint8_t* scale,
                                            int lane, bool in_row, bool on) {
  if constexpr (HELD == kE2M1) {                 // a lane has a block of its own
    uint32_t byte;
    const uint2 code = block_to_e2m1<F16>(w, &byte);
    if (in_row) {
      reinterpret_cast<uint2*>(dst)[lane] = code;
      scale[lane] = (uint8_t)byte;
    }
  } else {
    uint32_t big2 = 0;                           // magnitudes in order, NaN last
#pragma unroll
    for (int k = 0; k < 8; ++k) big2 = __vmaxu2(big2, w[k] & 0x7fff7fffu);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
      big2 = __vmaxu2(big2, __shfl_xor_sync(0xffffffffu, big2, o));
    const uint32_t big = __float_as_uint(to_float<F16>((uint16_t)max(big2 & 0xffffu, big2 >> 16)));
    // a = m 2^x, 448 = 1.75 2^8: e = x - 8, one more where m > 1.75
    const int field = (int)(big >> 23);
    int byte = field - 8 + ((big & 0x7fffffu) > 0x600000u ? 1 : 0);
    byte = field == 255 ? 255 : max(byte, 0);
    const float inv = __uint_as_float((uint32_t)(254 - (byte == 255 ? 127 : byte)) << 23);
    uint32_t code[4];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const __nv_fp8x2_storage_t c2 = __nv_cvt_float2_to_fp8x2(
          make_float2(to_float<F16>((uint16_t)w[k]) * inv, to_float<F16>((uint16_t)(w[k] >> 16)) * inv),
          __NV_SATFINITE, __NV_E4M3);
      code[k / 2] = k % 2 ? code[k / 2] | (uint32_t)c2 << 16 : (uint32_t)c2;
    }
    if (byte == 255) {
#pragma unroll
      for (int k = 0; k < 4; ++k) code[k] = 0x7f7f7f7fu;
    }
    if (in_row)
      reinterpret_cast<uint4*>(dst)[lane] = make_uint4(code[0], code[1], code[2], code[3]);
    if (on && lane == 0) *scale = (uint8_t)byte;
  }
}

}  // namespace tree
}  // namespace dspark
