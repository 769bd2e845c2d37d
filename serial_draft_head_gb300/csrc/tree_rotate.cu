// tree_rotate.cu -- norms of query and key heads and the rotation by their positions in
// one pass, on the way to attention and into the cache (the header has the formulas).
//
// A row (one token, one head) is handled by D / 16 lanes, rounded up to 4 or 8, 16
// elements each: for rotation by halves an 8-element chunk of the first half and the one
// that it turns with, so that a pair is in one thread and only the norm's sum crosses
// lanes.  A warp has a token (or, so that few tokens fill the device, a share of its
// heads): it works out the token's sines and cosines, one a lane, keeps them, times the
// norm's weights, in registers, and goes through the heads with five rounds' loads in flight.
// Nothing is handed between warps.
//
// Angles: a frequency is held in turns a position, as a 64-bit fraction, so that position
// times frequency modulo one turn is one integer product, exact at any position; its
// upper 32 bits go to fp32 and to sincospi.
//
// Everything between the loads and the stores is fp32; k is rounded to the handle's type
// before it is quantised, as if it had been stored and written.
//
// What bounds it: memory.  32,284 tokens of 32 + 8 + 8 heads of 128: into a 16-bit cache 132
// us, 6.0 TB/s of bytes read and written; q and k alone 107 us, 6.2; into e2m1 148 (the
// quantising).  With the next rows in registers instead of five rounds of copies into
// shared memory 172.  128 tokens: 4.6 us, a chain of the slot, the position, the angles and
// the rows.
#include "tc_ptx.cuh"
#include "tree_codes.cuh"

namespace dspark {
namespace tree {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kDepth = 5;          // rounds of a warp's loads in flight, a KB each

// The sum of a row's squares, in all its lanes.
template <int LANES>
__device__ __forceinline__ float row_squares(const uint64_t (&u)[4], const uint64_t (&z)[4]) {
  uint64_t squares = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) squares = ptx::fma_f32x2(u[k], u[k], ptx::fma_f32x2(z[k], z[k], squares));
  float sum, odd;
  ptx::unpack_f32x2(squares, &sum, &odd);
  sum += odd;
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// The power of two, 2^-120 to 2^top, that brings a row's largest element near 1.
template <int LANES>
__device__ __forceinline__ float row_unit(const uint64_t (&u)[4], const uint64_t (&z)[4], int top) {
  float big = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float lo, hi;
    ptx::unpack_f32x2(u[k], &lo, &hi);
    big = fmaxf(big, fmaxf(fabsf(lo), fabsf(hi)));
    ptx::unpack_f32x2(z[k], &lo, &hi);
    big = fmaxf(big, fmaxf(fabsf(lo), fabsf(hi)));
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
  const int e = 127 - (int)(__float_as_uint(big) >> 23);
  return __uint_as_float((uint32_t)(127 + min(max(e, -120), top)) << 23);
}

// PLACE: k and v go to the cache, as HELD says; else k to out_k and there is no v.  2^`shift`
// warps a token.
template <bool F16, bool PLACE, Held HELD, int LANES>
__global__ void __launch_bounds__(kThreads, 6) rotate_kernel(const __grid_constant__ RotateArgs a, int shift) {
  __shared__ float2 turns[kWarps][8 * LANES];      // {cosine, sine} of the token's pairs
  __shared__ uint4 rows_in[kWarps][kDepth][2][32]; // each lane the chunks that it copied itself
  constexpr int kGroups = 32 / LANES;              // rows at a time
  const int warp = threadIdx.x / 32, wl = threadIdx.x % 32, lane = wl % LANES, group = wl / LANES;
  const int64_t job = (int64_t)blockIdx.x * kWarps + warp;
  if (job >> shift >= a.N) return;
  const int n = (int)(job >> shift), share = (int)(job & ((1 << shift) - 1));
  int64_t page = 0;
  int place = 0;
  if (PLACE) {
    const int slot = __ldg(a.slot + n);
    if (slot < 0 || slot >= a.slots) {             // left out
      if (slot >= 0 && wl == 0) set_status(a.status, DSPARK_EPAGES);
      return;
    }
    page = a.c.page.div(slot);
    place = slot - (int)page * a.c.page.d;
  }
  const int half = a.R / 16;                       // chunks of half a turned part
  const bool in_row = lane * 16 < a.D, turned = lane < half;
  // the lane's two chunks
  const int c0 = turned ? (a.pairs ? 2 * lane : lane) : 2 * lane;
  const int c1 = turned && !a.pairs ? lane + half : c0 + 1;
  // rounds: kGroups heads each, those of q, then k, then v
  const int of_q = (a.Hq + kGroups - 1) / kGroups, of_kv = (a.Hkv + kGroups - 1) / kGroups;
  const int rounds = of_q + of_kv * (PLACE ? 2 : 1), step = 1 << shift;
  int in = 0;
  auto load = [&](int round) {
    const int i = round < of_q ? 0 : round < of_q + of_kv ? 1 : 2;
    const int head = (round - (i == 0 ? 0 : i == 1 ? of_q : of_q + of_kv)) * kGroups + group;
    if (in_row && round < rounds && head < (i == 0 ? a.Hq : a.Hkv)) {
      const uint4* src = reinterpret_cast<const uint4*>(a.src[i] + n * a.src_row[i] + head * a.src_head[i]);
      ptx::cp_async16(&rows_in[warp][in][0][wl], src + (i == 2 ? 2 * lane : c0));
      ptx::cp_async16(&rows_in[warp][in][1][wl], src + (i == 2 ? 2 * lane + 1 : c1));
    }
    ptx::cp_async_commit();
    if (++in == kDepth) in = 0;
  };
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) load(share + i * step);
  const int64_t pos = __ldg(a.position + n);
  for (int f = wl; f < a.R / 2; f += 32) {
    const int32_t part = (int32_t)((uint64_t)pos * __ldg(a.turns + f) >> 32);
    float s, c;
    sincospif((float)part * 0x1p-31f, &s, &c);
    // pair f is pair f % 8 of lane f / 8
    turns[warp][f % 8 * LANES + f / 8] = make_float2(c, s);
  }
  __syncwarp();
  // a pair (u, z), each times the norm's factor, becomes u k0 - z k1, z k2 + u k3; one that
  // is not turned u k0, z k2.  Two pairs at once.
  uint64_t k0[4], k1[4], k2[4], k3[4];
  auto weigh = [&](bool key) {
    const float* norm = key ? a.k_norm : a.q_norm;
    float w0[8], w1[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w0[k] = w1[k] = 1.f;
    if (norm && in_row) {
      const float4* g = reinterpret_cast<const float4*>(norm);
      const float4 y[4] = {__ldg(g + 2 * c0), __ldg(g + 2 * c0 + 1), __ldg(g + 2 * c1), __ldg(g + 2 * c1 + 1)};
      const float e[16] = {y[0].x, y[0].y, y[0].z, y[0].w, y[1].x, y[1].y, y[1].z, y[1].w,
                           y[2].x, y[2].y, y[2].z, y[2].w, y[3].x, y[3].y, y[3].z, y[3].w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        w0[k] = a.pairs ? e[2 * k] : e[k];
        w1[k] = a.pairs ? e[2 * k + 1] : e[8 + k];
      }
    }
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const float2 s = turned ? turns[warp][k * LANES + lane] : make_float2(1.f, 0.f);
      const float2 t = turned ? turns[warp][(k + 1) * LANES + lane] : make_float2(1.f, 0.f);
      k0[k / 2] = ptx::pack_f32x2(w0[k] * s.x, w0[k + 1] * t.x);
      k1[k / 2] = ptx::pack_f32x2(-w1[k] * s.y, -w1[k + 1] * t.y);
      k2[k / 2] = ptx::pack_f32x2(w1[k] * s.x, w1[k + 1] * t.x);
      k3[k / 2] = ptx::pack_f32x2(w0[k] * s.y, w0[k + 1] * t.y);
    }
  };
  int weights = -1;                                // whose they are: of q 0, of k 1
#pragma unroll 1
  for (int round = share; round < rounds; round += step) {
    load(round + (kDepth - 1) * step);
    ptx::cp_async_wait_group<kDepth - 1>();
    const int i = round < of_q ? 0 : round < of_q + of_kv ? 1 : 2;       // the warp's rows are of one kind
    const int head = (round - (i == 0 ? 0 : i == 1 ? of_q : of_q + of_kv)) * kGroups + group;
    const bool live = head < (i == 0 ? a.Hq : a.Hkv);
    uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (in_row && live) {
      x[0] = rows_in[warp][in][0][wl];             // the oldest
      x[1] = rows_in[warp][in][1][wl];
    }
    uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    if (i < 2) {
      if (weights != i) {
        weights = i;
        weigh(i == 1);
      }
      uint64_t u[4], z[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // two words: the pairs 2 k and 2 k + 1
        const uint32_t v0 = a.pairs ? w[2 * k] : w[k], v1 = a.pairs ? w[2 * k + 1] : w[4 + k];
        const float a0 = to_float<F16>((uint16_t)v0), a1 = to_float<F16>((uint16_t)(v0 >> 16));
        const float b0 = to_float<F16>((uint16_t)v1), b1 = to_float<F16>((uint16_t)(v1 >> 16));
        u[k] = a.pairs ? ptx::pack_f32x2(a0, b0) : ptx::pack_f32x2(a0, a1);
        z[k] = a.pairs ? ptx::pack_f32x2(a1, b1) : ptx::pack_f32x2(b0, b1);
      }
      if (i == 0 ? a.q_norm != nullptr : a.k_norm != nullptr) {
        float sum = row_squares<LANES>(u, z), eps = a.eps;
        if (!F16) {
          // squares can leave fp32 (bf16 past 2^63; below 2^-40 without an eps): such a row is
          // brought near 1 by a power of two, which the norm takes out again
          const bool far = !(sum <= 3.40282347e38f && sum >= a.least);
          if (__any_sync(0xffffffffu, far && live)) {
            const float unit = row_unit<LANES>(u, z, a.eps > 0.f ? 60 : 120), by = far ? unit : 1.f;
            const uint64_t by2 = ptx::pack_f32x2(by, by);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              u[k] = ptx::mul_f32x2(u[k], by2);
              z[k] = ptx::mul_f32x2(z[k], by2);
            }
            eps = eps * by * by;                   // 0 stays 0
            sum = row_squares<LANES>(u, z);
          }
        }
        const float r = rsqrtf(sum * a.inv_dim + eps);
        const uint64_t r2 = ptx::pack_f32x2(r, r);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          u[k] = ptx::mul_f32x2(u[k], r2);
          z[k] = ptx::mul_f32x2(z[k], r2);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint64_t y0 = ptx::mul_f32x2(u[k], k0[k]), y1 = ptx::mul_f32x2(z[k], k2[k]);
        if (turned) {
          y0 = ptx::fma_f32x2(z[k], k1[k], y0);
          y1 = ptx::fma_f32x2(u[k], k3[k], y1);
        }
        float a0, a1, b0, b1;
        ptx::unpack_f32x2(y0, &a0, &a1);
        ptx::unpack_f32x2(y1, &b0, &b1);
        if (a.pairs) {
          w[2 * k] = pack2<F16>(a0, b0);
          w[2 * k + 1] = pack2<F16>(a1, b1);
        } else {
          w[k] = pack2<F16>(a0, a1);
          w[4 + k] = pack2<F16>(b0, b1);
        }
      }
    }
    if (!PLACE || i == 0 || HELD == k16) {
      if (live && in_row) {
        uint4* dst;
        if (PLACE && i > 0) dst = reinterpret_cast<uint4*>(a.c.x[i - 1].at((uint32_t)page, place, head));
        else dst = reinterpret_cast<uint4*>((i ? a.out_k : a.out_q) + ((int64_t)n * (i ? a.Hkv : a.Hq) + head) * a.D);
        dst[i == 2 ? 2 * lane : c0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[i == 2 ? 2 * lane + 1 : c1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
      continue;
    }
    if constexpr (PLACE && HELD != k16) {
      if (i == 1 && !a.pairs) {
        // a row of k as it lies: lane i chunks 2 i and 2 i + 1
        uint32_t natural[8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 2 * lane + e;              // is the first or second chunk of a lane
          const bool first = c < half, second = !first && c < 2 * half;
          const int from = first ? c : second ? c - half : lane;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t lo = __shfl_sync(0xffffffffu, w[k], from, LANES);
            const uint32_t hi = __shfl_sync(0xffffffffu, w[4 + k], from, LANES);
            natural[4 * e + k] = first ? lo : second ? hi : w[4 * e + k];
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = natural[k];
      }
      const int to = live ? head : 0;
      store_codes<F16, HELD, LANES>(w, a.c.x[i - 1].at((uint32_t)page, place, to),
                                    a.c.scale[i - 1].at((uint32_t)page, place, to), lane, live && in_row, live);
    }
  }
}

template <bool F16, bool PLACE, Held HELD, int LANES>
void launch(const RotateArgs& a, int sm_count, cudaStream_t stream) {
  // a token's heads over as many warps as give every SM 16, at least two rounds each
  constexpr int kGroups = 32 / LANES;
  const int of_kv = (a.Hkv + kGroups - 1) / kGroups;
  const int rounds = (a.Hq + kGroups - 1) / kGroups + of_kv * (PLACE ? 2 : 1);
  int shift = 0;
  while (2 << shift <= rounds && (int64_t)a.N << shift < (int64_t)16 * sm_count) ++shift;
  const int64_t jobs = (int64_t)a.N << shift;
  rotate_kernel<F16, PLACE, HELD, LANES>
      <<<(unsigned)((jobs + kWarps - 1) / kWarps), kThreads, 0, stream>>>(a, shift);
}

template <bool F16, bool PLACE, Held HELD>
void launch_lanes(const RotateArgs& a, int sm_count, cudaStream_t stream) {
  if (a.D <= 64) launch<F16, PLACE, HELD, 4>(a, sm_count, stream);
  else launch<F16, PLACE, HELD, 8>(a, sm_count, stream);
}

template <bool F16>
void launch_held(const RotateArgs& a, bool place, Held held, int sm_count, cudaStream_t stream) {
  if (!place) launch_lanes<F16, false, k16>(a, sm_count, stream);
  else if (held == k16) launch_lanes<F16, true, k16>(a, sm_count, stream);
  else if (held == kE4M3) launch_lanes<F16, true, kE4M3>(a, sm_count, stream);
  else launch_lanes<F16, true, kE2M1>(a, sm_count, stream);
}

}  // namespace

cudaError_t rotate_launch(const RotateArgs& a, bool place, bool f16, Held held, int sm_count,
                          cudaStream_t stream) {
  if (f16) launch_held<true>(a, place, held, sm_count, stream);
  else launch_held<false>(a, place, held, sm_count, stream);
  return cudaGetLastError();
}

}  // namespace tree
}  // namespace dspark
