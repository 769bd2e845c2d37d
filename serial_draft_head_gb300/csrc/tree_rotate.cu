// tree_rotate.cu -- norms of query and key heads and the rotation by their positions in
// one pass, on the way to attention and into the cache (the header has the formulas).
//
// A row (one token, one head) is handled by D / 16 lanes, rounded up to 4 or 8, 16
// elements each: for rotation by halves an 8-element chunk of the first half and the one
// that it turns with, so that a pair is in one thread and only the norm's sum crosses
// lanes.  A block has 1, 2 or 4 tokens; sines and cosines of a token are worked out once,
// one a thread, and kept in registers over its heads.
//
// Angles: a frequency is held in turns a position, as a 64-bit fraction, so that position
// times frequency modulo one turn is one integer product, exact at any position; its
// upper 32 bits go to fp32 and to sincospi.
//
// Everything between the loads and the stores is fp32; k is rounded to the handle's type
// before it is quantised, as if it had been stored and written.
#include "tc_ptx.cuh"
#include "tree_codes.cuh"

namespace dspark {
namespace tree {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 4;         // tokens of a block

// PLACE: k and v go to the cache, as HELD says; else k to out_k and there is no v.
template <bool F16, bool PLACE, Held HELD, int LANES>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const __grid_constant__ RotateArgs a, int tok) {
  __shared__ float2 turn[kMaxTok][LANES][9];       // [token][lane][of its pairs], a column spare
  constexpr int kGroups = kThreads / LANES;        // rows at a time
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int per = kGroups / tok;                   // groups of a token
  const int t = group / per, n = blockIdx.x * tok + t;
  const int half = a.R / 16;                       // chunks of half a turned part
  const bool in_row = lane * 16 < a.D, turned = lane < half;
  // the lane's two chunks
  const int c0 = turned ? (a.pairs ? 2 * lane : lane) : 2 * lane;
  const int c1 = turned && !a.pairs ? lane + half : c0 + 1;
  int slot = 0;
  bool on = n < a.N;
  if (PLACE && on) {
    slot = a.slot[n];
    on = slot >= 0 && slot < a.slots;
    if (slot >= a.slots && lane == 0) set_status(a.status, DSPARK_EPAGES);
  }
  const int heads = a.Hq + a.Hkv * (PLACE ? 2 : 1);
  uint4 x[2], next[2];
  auto load = [&](int h) {
    next[0] = next[1] = make_uint4(0, 0, 0, 0);
    if (!on || !in_row || h >= heads) return;
    const int i = h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2;
    const int head = h - (i == 0 ? 0 : i == 1 ? a.Hq : a.Hq + a.Hkv);
    const uint4* src = reinterpret_cast<const uint4*>(a.src[i] + (int64_t)n * a.src_row[i] +
                                                      head * a.src_head[i]);
    next[0] = __ldg(src + (i == 2 ? 2 * lane : c0));
    next[1] = __ldg(src + (i == 2 ? 2 * lane + 1 : c1));
  };
  load(group % per);
  // sines and cosines of the block's tokens, pair i of a token for lane i / 8
  for (int i = threadIdx.x; i < tok * (a.R / 2); i += kThreads) {
    const int tt = i / (a.R / 2), f = i - tt * (a.R / 2), row = blockIdx.x * tok + tt;
    const int64_t pos = row < a.N ? a.position[row] : 0;
    const int32_t part = (int32_t)((uint64_t)pos * __ldg(a.turns + f) >> 32);
    float s, c;
    sincospif((float)part * 0x1p-31f, &s, &c);
    turn[tt][f / 8][f % 8] = make_float2(c, s);
  }
  __syncthreads();
  float2 cs[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) cs[k] = turned ? turn[t][lane][k] : make_float2(0.f, 0.f);
  int64_t page = 0;
  int place = 0;
  if (PLACE && on) {
    page = a.c.page.div(slot);
    place = slot - (int)page * a.c.page.d;
  }
#pragma unroll 1
  for (int h0 = 0; h0 < heads; h0 += per) {        // whole warps stay in the loop: the shuffles
    const int h = h0 + group % per;
    x[0] = next[0];
    x[1] = next[1];
    load(h + per);
    const bool q = h < a.Hq, v = PLACE && h >= a.Hq + a.Hkv, live = on && h < heads;
    const int head = q ? h : v ? h - a.Hq - a.Hkv : h - a.Hq;
    uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    if (!__all_sync(0xffffffffu, v)) {
      float y[16];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        y[2 * k] = to_float<F16>((uint16_t)w[k]);
        y[2 * k + 1] = to_float<F16>((uint16_t)(w[k] >> 16));
      }
      const float* norm = q ? a.q_norm : a.k_norm;
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) sum = fmaf(y[k], y[k], sum);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (norm && in_row) {
        const float r = rsqrtf(sum * a.inv_dim + a.eps);
        const float4* g0 = reinterpret_cast<const float4*>(norm) + 2 * c0;
        const float4* g1 = reinterpret_cast<const float4*>(norm) + 2 * c1;
        const float4 g[4] = {__ldg(g0), __ldg(g0 + 1), __ldg(g1), __ldg(g1 + 1)};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          y[4 * k] *= r * g[k].x;
          y[4 * k + 1] *= r * g[k].y;
          y[4 * k + 2] *= r * g[k].z;
          y[4 * k + 3] *= r * g[k].w;
        }
      }
      if (!turned) {
      } else if (a.pairs) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float u = y[2 * k], z = y[2 * k + 1];
          y[2 * k] = fmaf(u, cs[k].x, -z * cs[k].y);
          y[2 * k + 1] = fmaf(z, cs[k].x, u * cs[k].y);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float u = y[k], z = y[8 + k];
          y[k] = fmaf(u, cs[k].x, -z * cs[k].y);
          y[8 + k] = fmaf(z, cs[k].x, u * cs[k].y);
        }
      }
      if (!v) {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = pack2<F16>(y[2 * k], y[2 * k + 1]);
      }
    }
    const bool cached = PLACE && !q;
    if (!cached || HELD == k16) {
      if (live && in_row) {
        uint4* dst = !cached ? reinterpret_cast<uint4*>((q ? a.out_q : a.out_k) +
                                                        ((int64_t)n * (q ? a.Hq : a.Hkv) + head) * a.D)
                             : reinterpret_cast<uint4*>(a.c.x[v].at((uint32_t)page, place, head));
        dst[v ? 2 * lane : c0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[v ? 2 * lane + 1 : c1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
    if constexpr (PLACE && HELD != k16) {
      if (!__any_sync(0xffffffffu, cached)) continue;
      // a row of k as it lies: lane i chunks 2 i and 2 i + 1
      if (!a.pairs) {
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
        for (int k = 0; k < 8; ++k) w[k] = v ? w[k] : natural[k];
      }
      store_codes<F16, HELD, LANES>(w, a.c.x[v].at((uint32_t)page, place, cached ? head : 0),
                                    a.c.scale[v].at((uint32_t)page, place, cached ? head : 0), lane,
                                    live && cached && in_row, live && cached);
    }
  }
}

template <bool F16, bool PLACE, Held HELD, int LANES>
void launch(const RotateArgs& a, int sm_count, cudaStream_t stream) {
  // four tokens a block share what a block costs, unless that leaves SMs without one
  int tok = kMaxTok;
  while (tok > 1 && (a.N - 1) / tok + 1 < 2 * sm_count) tok >>= 1;
  rotate_kernel<F16, PLACE, HELD, LANES><<<(a.N - 1) / tok + 1, kThreads, 0, stream>>>(a, tok);
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
