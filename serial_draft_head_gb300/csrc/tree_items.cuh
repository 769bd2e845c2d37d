// tree_items.cuh -- how the attention kernels (tree_attend.cuh, tree_attend_few.cu,
// tree_attend_few4.cuh) cut their work, and the parts of the softmax they share.
//
// Per cached head the rows that read it are (node, query head of the group):
// T * G of them.  A work item is (request, cached head, up to ROWS of its rows)
// over all its keys, cut into tiles of KEYS keys; a tile of one item is a unit,
// and so that short items do not pile up on one worker, EXTRA more units stand
// before an item's first for what it costs beside its tiles (Q, the result, the
// way into the loop).  The units of all items, in order, are split evenly over
// the workers (one CTA a SM, or, over e2m1, up to four in it): the lengths are known on the
// device only, so every CTA sums them up itself.  An item that lies inside one worker's share is
// finished there; one that several workers share leaves parts (unnormalised O,
// maximum, sum), at most one a worker, joined in an order that does not depend on
// timing: by the worker that is last to leave its part (few rows: 16 rows a part, over e2m1
// 8, 16 or 32), or by a second kernel over all SMs (tcgen05: up to 256 rows a part).
//
// Mathematics, per row, one pass over the tiles in the base-2 exponent:
//   x_j = log2(e) * scale * q.k_j              (capped: log2(e) c tanh(s / c))
//   p_j = 2^(x_j - m),  l = sum p_j,  O = sum p_j v_j
// m follows the running maximum lazily: it moves, and O and l are rescaled, only when
// the maximum has grown by more than 8, so p <= 2^8, and the rescaling of O is rare.
// For products in f16 m stands 7 below the maximum that set it, so that weights down
// to 2^-21 of the largest stay normal numbers: p <= 2^15 then, and f16 ends at 65,504.
// O and l in fp32 keep their relative precision.  p is rounded once to the 16-bit type
// for the second product (half a unit, as the result itself is rounded); l sums the
// unrounded p.  Over e2m1 in bf16 on tcgen05 it is otherwise: m moves when the maximum has
// grown by more than 64, so p <= 2^64, and rows are divided by the sum of the rounded p
// (grow_limit and Sum in tree_attend.cuh have the reasons).
#pragma once

#include <math.h>

#include "tc_ptx.cuh"
#include "tree_common.cuh"

namespace dspark {
namespace tree {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Raw scores to base-2 exponents.  Caps beyond 2^100 or below 2^-100 do to scores in
// fp32 what those do.
struct Score {
  float sl2;        // |scale| log2(e): a negative scale turns Q's signs
  float cap2;       // softcap log2(e), 0 without a cap
  float cap_in;     // 2 sl2 / softcap: tanh(y) = 1 - 2 / (2^(2 y log2(e)) + 1)
  float cap_y;      // |scale| / softcap

  __device__ static Score of(const AttendArgs& a) {
    Score s;
    const float c = fminf(fmaxf(a.softcap, 0x1p-100f), 0x1p100f);
    s.sl2 = fabsf(a.scale) * kLog2e;
    s.cap2 = a.softcap > 0.f ? c * kLog2e : 0.f;
    s.cap_in = 2.f * s.sl2 / c;
    s.cap_y = fabsf(a.scale) / c;
    return s;
  }
};

// Up to |y| = 0.75 (y = s / c) tanh(y) / y is a polynomial in y^2, fitted to it by
// weighted least squares, within 6.5e-8 of it, so that a score keeps its relative
// precision under any cap.  Past that, c - 2c / (e^2y + 1) does; below, its
// difference would cancel (c 2^-22 off whatever the score).
constexpr float kNearCap = 0.75f;
__device__ __forceinline__ constexpr float tanh_coef(int i) {
  constexpr float k[6] = {1.f,           -0.333329588f, 0.133254066f,
                          -0.0533444323f, 0.0195829086f, -0.00471625756f};
  return k[i];
}

// A capped score's exponent less `sub` in the two forms.  Which one it gets goes by
// the score alone, so a row's weights do not depend on the rows and keys beside it;
// that a whole warp needs only the first saves the second's special functions.
__device__ __forceinline__ float capped_near(const Score& sc, float raw, float sub) {
  const float y = raw * sc.cap_y, u = y * y;
  float t = sc.cap2 * tanh_coef(5);
#pragma unroll
  for (int i = 4; i >= 0; --i) t = fmaf(t, u, sc.cap2 * tanh_coef(i));
  return fmaf(y, t, -sub);
}

__device__ __forceinline__ float capped_past(const Score& sc, float raw, float sub) {
  return sc.cap2 - 2.f * sc.cap2 * rcp(ex2(raw * sc.cap_in) + 1.f) - sub;
}

__device__ __forceinline__ bool past_near(const Score& sc, float raw) {
  return fabsf(raw * sc.cap_y) > kNearCap;
}

__device__ __forceinline__ float capped(const Score& sc, float raw, float sub) {
  return past_near(sc, raw) ? capped_past(sc, raw, sub) : capped_near(sc, raw, sub);
}

// a / b for a >= 0, b > 0: 32-bit arithmetic where that does.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// `total` units over the workers that get any (one at least), evenly: those with one more than
// the others lie between them, so that where the items are alike and divide the
// workers (one long request: 8 heads on 152 SMs) no share crosses an item's end
// (99 us for 17 rows over 131,000 tokens; 103.5 with the longer shares first).
struct Cut {
  int64_t total, per;
  int rest, workers;

  __device__ static __forceinline__ Cut of(int64_t total, int n_cta) {
    Cut c;
    c.total = total;
    c.workers = (int)(total < n_cta ? max(total, (int64_t)1) : n_cta);   // one without units
    c.per = quotient(total, c.workers);
    c.rest = (int)(total - c.per * c.workers);
    return c;
  }
  __device__ __forceinline__ int64_t start(int worker) const {
    return worker * per + worker * rest / workers;
  }
  // The worker whose share holds unit u.
  __device__ __forceinline__ int holder(int64_t u) const {
    int c = (int)quotient(u * workers, total);
    while (start(c + 1) <= u) ++c;
    while (start(c) > u) --c;
    return c;
  }
};

// A worker's share: its units, how all were cut, and the place of its first (t0 <
// 0: one of the units before an item's tiles).
struct Share {
  int64_t unit0, units;
  Cut cut;
  int b0, head0, group0, t0;
};

template <int KEYS, int ROWS, int EXTRA>
struct Work {
  // Rows of request b as attend takes them (0 if they do not fit), key tiles and
  // row groups.
  struct Request {
    int row0, rows, start, tiles, groups;
  };

  __device__ static __forceinline__ Request load_request(const AttendArgs& a, int b, bool* ok) {
    Request r;
    *ok = request_rows(a.b, b, &r.row0, &r.rows, &r.start) && r.rows <= a.max_nodes &&
          (!a.mask || r.rows <= 32 * a.mask_words);
    if (!*ok) r.rows = 0;
    r.tiles = (int)(((int64_t)r.start + r.rows + KEYS - 1) / KEYS);
    r.groups = (r.rows * a.G + ROWS - 1) / ROWS;
    return r;
  }

  // The shares of the CTA's WORKERS workers, by all its THREADS threads: sums the requests'
  // units in order.
  template <int THREADS, int WORKERS = 1>
  __device__ static __forceinline__ void plan(const AttendArgs& a, Share* share,
                                              int64_t* warp_sum) {
    constexpr int kPer = (DSPARK_TREE_MAX_REQUESTS + THREADS - 1) / THREADS;
    int64_t mine[kPer], sum = 0;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int per = (a.b.B + THREADS - 1) / THREADS;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int b = threadIdx.x * per + k;
      mine[k] = 0;
      if (k < per && b < a.b.B) {
        bool ok;
        const Request r = load_request(a, b, &ok);
        if (ok && r.rows > 0) mine[k] = (int64_t)(r.tiles + EXTRA) * r.groups * a.Hkv;
        if (!ok && blockIdx.x == 0) set_status(a.status, DSPARK_EPAGES);
      }
      sum += mine[k];
    }
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    if (threadIdx.x < WORKERS) share[threadIdx.x].units = 0;
    __syncthreads();
    int64_t before = incl - sum, total = 0;
#pragma unroll
    for (int k = 0; k < THREADS / 32; ++k) {
      const int64_t y = warp_sum[k];
      if (k < warp) before += y;
      total += y;
    }
    const Cut cut = Cut::of(total, a.n_cta);
#pragma unroll 1
    for (int k = 0; k < WORKERS; ++k, ++share) {
      const int worker = blockIdx.x * WORKERS + k;
      const int64_t u0 = cut.start(worker);
      // the thread whose requests hold the share's first unit writes it
      if (worker < cut.workers && u0 >= before && u0 < before + sum) {
        int64_t at = before;
#pragma unroll 1
        for (int b = threadIdx.x * per; b < a.b.B; ++b) {
          bool ok;
          const Request r = load_request(a, b, &ok);
          const int64_t units = (int64_t)(r.tiles + EXTRA) * r.groups * a.Hkv;
          if (u0 < at + units) {
            share->unit0 = u0;
            share->units = cut.start(worker + 1) - u0;
            share->cut = cut;
            const int64_t item = quotient(u0 - at, r.tiles + EXTRA);
            const int head = (int)quotient(item, r.groups);
            share->b0 = b;
            share->t0 = (int)(u0 - at - item * (r.tiles + EXTRA)) - EXTRA;
            share->head0 = head;
            share->group0 = (int)(item - (int64_t)head * r.groups);
            break;
          }
          at += units;
        }
      }
    }
    __syncthreads();
  }

  // One worker's part of an item: key tiles t0 .. t1-1 of `tiles`.
  struct Segment {
    int b, row0, rows, start, head, group, t0, t1, tiles;
    int64_t item_end;                   // unit after the item's last
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
  };

  struct Walker {
    Request r;
    int b, head, group, t0;
    int64_t left, unit;

    __device__ void init(const AttendArgs& a, const Share& s) {
      left = s.units;
      unit = s.unit0;
      b = s.b0;
      head = s.head0;
      group = s.group0;
      t0 = s.t0;
      bool ok;
      if (left > 0) r = load_request(a, b, &ok);
    }

    __device__ bool next(const AttendArgs& a, Segment* s) {
      while (left > 0) {
        const int64_t rest = r.tiles - t0;
        const int n = (int)(rest < left ? rest : left);
        s->b = b;
        s->row0 = r.row0;
        s->rows = r.rows;
        s->start = r.start;
        s->head = head;
        s->group = group;
        s->t0 = t0 > 0 ? t0 : 0;
        s->t1 = t0 + n;
        s->tiles = r.tiles;
        s->item_end = unit + rest;
        left -= n;
        unit += n;
        t0 += n;
        if (t0 == r.tiles) {
          t0 = -EXTRA;
          if (++group == r.groups) {
            group = 0;
            if (++head == a.Hkv) {
              head = 0;
              bool ok;
              if (left > 0) do {
                  r = load_request(a, ++b, &ok);
                } while (r.rows == 0 && b + 1 < a.b.B);
              if (r.rows == 0) left = 0;  // the arrays changed under the kernel
            }
          }
        }
        if (s->t1 > s->t0) return true;   // else no more than units before the tiles
      }
      return false;
    }
  };

  // The tiles of a share, in order.
  struct Cursor {
    int b, head, group, t, seg;         // seg: segments begun before this one
    int rows, start, tiles, groups;     // of the request
    int64_t left;                       // tiles from this one on

    __device__ void load(const AttendArgs& a) {
      bool ok;
      const Request r = load_request(a, b, &ok);
      rows = r.rows;
      start = r.start;
      tiles = r.tiles;
      groups = r.groups;
    }
    __device__ void init(const AttendArgs& a, const Share& s) {
      left = s.units;
      b = s.b0;
      head = s.head0;
      group = s.group0;
      t = s.t0;
      seg = 0;
      if (left > 0) load(a);
      skip();
    }
    __device__ __forceinline__ void skip() {      // the units before an item's tiles
      if (t < 0) {
        left += t;
        t = 0;
      }
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ int total() const { return start + rows; }
    __device__ void next(const AttendArgs& a) {
      --left;
      if (++t < tiles) return;
      t = -EXTRA;
      skip();
      ++seg;
      if (++group < groups) return;
      group = 0;
      if (++head < a.Hkv) return;
      head = 0;
      if (left <= 0) return;
      do {
        ++b;
        load(a);
      } while (rows == 0 && b + 1 < a.b.B);
      if (rows == 0) left = 0;          // the arrays changed under the kernel
    }
  };

  __device__ static __forceinline__ int group_rows(const AttendArgs& a, const Segment& s) {
    const int n = s.rows * a.G - s.group * ROWS;
    return n < ROWS ? n : ROWS;
  }

  // What the join needs of a part: the workers that share the item, from the one
  // with its first unit to that with its last.
  __device__ static __forceinline__ int4 part_of(const Segment& s, const Cut& cut) {
    const int first = cut.holder(s.item_end - s.tiles), last = cut.holder(s.item_end - 1);
    return make_int4(s.b, s.head, s.group, first | (last - first + 1) << 16);
  }
};

// The blocks of one warp in order: of every segment those t0 + warp, t0 + warp +
// warps, ...
template <class Item, int EXTRA>
struct BlockCursor {
  int b, head, group, t, end;           // end: of the segment
  int rows, start, tiles, groups;
  int64_t after;                        // units of the share after this segment
  bool more;

  __device__ void load(const AttendArgs& a) {
    bool ok;
    const typename Item::Request r = Item::load_request(a, b, &ok);
    rows = r.rows;
    start = r.start;
    tiles = r.tiles;
    groups = r.groups;
  }
  __device__ void settle(const AttendArgs& a, int warp) {     // past the ends of segments
    while (t >= end) {
      if (after <= EXTRA) {             // no more tiles in the share
        more = false;
        return;
      }
      if (++group == groups) {
        group = 0;
        if (++head == a.Hkv) {
          head = 0;
          do {
            if (++b >= a.b.B) {         // the arrays changed under the kernel
              more = false;
              return;
            }
            load(a);
          } while (rows == 0);
        }
      }
      after -= EXTRA;
      end = (int)(after < tiles ? after : tiles);
      after -= end;
      t = warp;
    }
  }
  __device__ void init(const AttendArgs& a, const Share& s, int warp) {
    more = s.units > 0;
    if (!more) return;
    b = s.b0;
    head = s.head0;
    group = s.group0;
    load(a);
    const int64_t rest = tiles - s.t0;
    const int n = (int)(rest < s.units ? rest : s.units);
    end = s.t0 + n;                     // below 0: the share ends before the tiles
    t = max(s.t0, 0) + warp;
    after = s.units - n;
    settle(a, warp);
  }
  __device__ void next(const AttendArgs& a, int warp, int warps) {
    t += warps;
    if (t >= end) settle(a, warp);
  }
};

// Draft positions 32 w .. 32 w + 31 that a node sees: its mask row (null: a
// chain) of a request with `rows` nodes.
__device__ __forceinline__ uint32_t sees_word(const uint32_t* mask_row, int rows, int node,
                                              int w) {
  const int left = rows - 32 * w;
  if (w < 0 || left <= 0) return 0u;
  const int n = node + 1 - 32 * w;
  const uint32_t m = mask_row ? __ldg(mask_row + w)
                              : n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
  return left >= 32 ? m : m & ((1u << left) - 1u);
}

// Visibility of the 32 positions from draft position j0 on (negative: context).
static __device__ __noinline__ uint32_t sees_32(const uint32_t* mask_row, int rows, int node, int j0) {
  const int w = j0 >> 5;                         // floor
  const uint32_t lo = w < 0 ? 0xffffffffu : sees_word(mask_row, rows, node, w);
  const uint32_t hi = w + 1 < 0 ? 0xffffffffu : sees_word(mask_row, rows, node, w + 1);
  return __funnelshift_r(lo, hi, j0 & 31);
}

// The magnitude's bits of the upper half of a word, a bf16; 0 where it is not finite.
__device__ __forceinline__ uint32_t finite_bits(uint32_t w) {
  const uint32_t x = w & 0x7fff0000u;
  return x >= 0x7f800000u ? 0u : x;
}

template <bool F16>
__device__ __forceinline__ bool nonfinite16(uint32_t x) {
  constexpr uint32_t e = F16 ? 0x7c00u : 0x7f80u;
  return (x & e) == e;
}

// Zeroes the non-finite elements of two packed ones; true if there were any.
template <bool F16>
__device__ __forceinline__ bool zero_nonfinite(uint32_t* w) {
  bool any = false;
  if (nonfinite16<F16>(*w)) {
    *w &= 0xffff0000u;
    any = true;
  }
  if (nonfinite16<F16>(*w >> 16)) {
    *w &= 0x0000ffffu;
    any = true;
  }
  return any;
}

template <bool F16>
__device__ __forceinline__ bool zero_nonfinite(uint4* x) {
  bool any = zero_nonfinite<F16>(&x->x);
  any |= zero_nonfinite<F16>(&x->y);
  any |= zero_nonfinite<F16>(&x->z);
  any |= zero_nonfinite<F16>(&x->w);
  return any;
}

// Four codes times any scale: through fp32, rounded and saturated as the cache
// reads back, in the order of scale_codes.
template <bool F16>
static __device__ __noinline__ uint2 scale_codes_any(uint32_t w, uint32_t byte) {
  const float s = scale_value(byte);
  const float2 x = e4m3x2_to_float2(w & 0xffffu), y = e4m3x2_to_float2(w >> 16);
  const uint2 r = make_uint2(
      pack2<F16>(saturate16<F16>(x.x * s), saturate16<F16>(x.y * s)),
      pack2<F16>(saturate16<F16>(y.x * s), saturate16<F16>(y.y * s)));
  return F16 ? r : swap_middle(r);
}

// Draft rows of V that are not finite would reach every row of the product
// (0 * NaN): their elements enter it as zeros, are noted (bad: a bit a node), and
// added here to the results that see them, which the calling thread has just
// written (columns d0 .. d1 - 1): what 0 < p times them comes to.  The result:
// 16-bit values (out), or a part's fp32 ones (column d at part[index(d)], stride
// and step given).
template <bool F16, int HELD>
__device__ __forceinline__ float bad_value(const AttendArgs& a, int b, int pos, int head, int d) {
  int64_t page;
  int slot;
  if (!locate(a.c, a.b, b, pos, &page, &slot)) return 0.f;
  const uint8_t* v = a.c.x[1].at((uint32_t)page, slot, head);
  if (HELD == k16) return to_float<F16>(reinterpret_cast<const uint16_t*>(v)[d]);
  if (HELD == kE2M1)                               // a number does not count here
    return a.c.scale[1].at((uint32_t)page, slot, head)[d / 16] > kTopScale ? __uint_as_float(0x7fffffffu) : 0.f;
  return saturate16<F16>(e4m3x2_to_float2(v[d]).x *
                         scale_value(*a.c.scale[1].at((uint32_t)page, slot, head)));
}

}  // namespace tree
}  // namespace dspark
