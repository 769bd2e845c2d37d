// tree_attend_few.cu -- attention of few drafted rows (at most 32 a cached head:
// single tokens, short chains) over a paged cache.
//
// A worker is a warp, alone with its items (16 or 32 rows by blocks of 16 keys;
// tree_items.cuh says how the work is cut, and the mathematics): no barriers,
// nothing handed between warps.  With so few rows K and V are used once from
// where they land, and the memory rate bounds the kernel; tcgen05 tiles of 128
// rows would be mostly padding, and what they need round them (rings, barriers,
// tensor memory) cost more than the products.  So the products are mma.sync
// m16n8k16, fed from registers:
//
//  - S = Q K^T: lane (g, q) = (lane / 4, lane % 4) holds B of key g and four
//    elements of it a step.  The order of the elements along the head is free as
//    long as Q has the same: lane q takes 16-byte chunks q, q + 4, ... of the row
//    as they lie, and Q's A operand is loaded by the same chunks.
//  - O = P V: P's A operand is S's accumulator, packed.  B of lane (g, q) is keys
//    2q, 2q + 1, 2q + 8, 2q + 9 at column g of every 8-column tile; the columns'
//    order is free too, so lane g takes 16-byte chunks g (and g + 8) of the four
//    rows, and pairs of keys are put together by byte permutations.
//
// So every thread reads just the 16-byte chunks that it copied itself: the ring
// in shared memory (cp.async, a stage is 16 keys of K and V) needs no barrier,
// only the thread's own wait.  e4m3 codes are converted in registers, the scale
// multiplied in (exact in bf16).
#include "tree_items.cuh"

namespace dspark {
namespace tree {
namespace {

constexpr int kBlock = 16;              // keys of a block, and of a ring stage

template <bool E4M3, int DP, int MT>
struct Few {
  static constexpr int kRows = 16 * MT;
  // as many warps as hold their O, Q and S in registers
  static constexpr int kWarps = MT == 1 ? 12 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kBytes = DP * (E4M3 ? 1 : 2);     // of a cached row
  static constexpr int kKCopies = kBytes / 64;           // 16-byte chunks a lane, of a row of K
  static constexpr int kVBytes = kBytes / 8;             // bytes a lane, of a row of V
  static constexpr int kStage = 2 * kBlock * kBytes;
  static constexpr int kVPart = kBlock * kBytes;         // V's place in a stage
  static constexpr int kStages = 16384 / kStage < 6 ? 16384 / kStage : 6;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kQ = MT == 1 ? 0 : kRows * DP * 2;        // two row tiles: Q in shared memory
  static constexpr int kScales = kRing + kQ;             // [stage][K 16, V 16]
  static constexpr int kBad = kScales + kStages * 32;
  static constexpr int kWarpBytes = kBad + DSPARK_TREE_MAX_NODES / 8;
  static constexpr int kShares = kWarps * kWarpBytes;
  static constexpr int kSums = kShares + kWarps * (int)sizeof(Share);
  static constexpr int kSmem = kSums + kWarps * 8;
};

// Column d of the result: its place in the accumulators, n = 2 q + e and tile.
template <bool E4M3, int DP>
__device__ __forceinline__ int column_n(int d) {
  return E4M3 ? d / (DP / 8) : d / 8 % 8;
}
template <bool E4M3, int DP>
__device__ __forceinline__ int column_tile(int d) {
  return E4M3 ? d % (DP / 8) : d % 8 + d / 64 * 8;
}

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if (F16) ptx::mma_16816_f16(d, a0, a1, a2, a3, b0, b1);
  else ptx::mma_16816(d, a0, a1, a2, a3, b0, b1);
}

// Four codes of two keys, as pairs of keys for four columns, any scales.
template <bool F16>
__device__ __noinline__ uint4 pair_codes_any(uint32_t wa, uint32_t byte_a, uint32_t wb,
                                             uint32_t byte_b) {
  uint2 x = scale_codes_any<F16>(wa, byte_a), y = scale_codes_any<F16>(wb, byte_b);
  if (!F16) {
    x = swap_middle(x);
    y = swap_middle(y);
  }
  return make_uint4(__byte_perm(x.x, y.x, 0x5410), __byte_perm(x.x, y.x, 0x7632),
                    __byte_perm(x.y, y.y, 0x5410), __byte_perm(x.y, y.y, 0x7632));
}

// Two codes of two keys (half 0 or 1 of words wa, wb), as two pairs of keys.
template <bool F16>
__device__ __forceinline__ uint2 pair_codes(uint32_t wa, uint32_t wb, int half, uint32_t mul2) {
  const uint32_t sel = F16 ? (half ? 0x7362 : 0x5140) : (half ? 0x7632 : 0x5410);
  return scale_codes<F16>(__byte_perm(wa, wb, sel), mul2);
}

// Adds to a row's result, written by this warp, the non-finite elements of the
// draft rows of V that it sees: 16-bit values (out), or the part's accumulators.
template <bool F16, bool E4M3, int DP>
__device__ __noinline__ void add_nonfinite(const AttendArgs& a, const uint32_t* bad,
                                           const uint32_t* mask_row, int b, int rows, int start,
                                           int head, int node, uint16_t* out, float* part,
                                           int row) {
#pragma unroll 1
  for (int j = 0; j < rows; ++j) {
    if (!(sees_word(mask_row, rows, node, j >> 5) & bad[j >> 5] & (1u << (j & 31)))) continue;
#pragma unroll 1
    for (int d = 0; d < a.D; ++d) {
      const float x = bad_value<F16, E4M3>(a, b, start + j, head, d);
      if (isfinite(x)) continue;
      if (out) {
        out[d] = (uint16_t)pack2<F16>(to_float<F16>(out[d]) + x, 0.f);
      } else {
        const int n = column_n<E4M3, DP>(d), tile = column_tile<E4M3, DP>(d);
        const int lane = row % 8 * 4 + n / 2;
        part[((row / 16 * (DP / 8) + tile) * 32 + lane) * 4 + (row / 8 % 2) * 2 + n % 2] += x;
      }
    }
  }
}

template <bool F16, bool E4M3, int DP, int MT>
__global__ void __launch_bounds__(Few<E4M3, DP, MT>::kThreads, 1)
    few_kernel(const __grid_constant__ AttendArgs a) {
  using L = Few<E4M3, DP, MT>;
  using Item = Work<kBlock, L::kRows>;
  constexpr int kTiles = DP / 8;                 // column tiles of O
  constexpr int kQChunks = DP / 32;              // 16-byte chunks of a row of Q a lane
  constexpr float kShift = F16 ? 7.f : 0.f;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, q = lane & 3;
  uint8_t* ring = smem + warp * L::kWarpBytes;
  uint4* q_mem = reinterpret_cast<uint4*>(ring + L::kRing);
  uint8_t* scales = ring + L::kScales;
  uint32_t* bad = reinterpret_cast<uint32_t*>(ring + L::kBad);
  Share* shares = reinterpret_cast<Share*>(smem + L::kShares);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int worker = warp * a.n_cta + blockIdx.x, workers = a.n_cta * L::kWarps;
  if (lane < 2) a.part_of[2 * worker + lane] = make_int4(0, 0, 0, 0);
  if (lane < DSPARK_TREE_MAX_NODES / 32) bad[lane] = 0;
  Item::template plan<L::kThreads, L::kWarps>(a, blockIdx.x, a.n_cta, workers, shares,
                                              reinterpret_cast<int64_t*>(smem + L::kSums));
  const Share& share = shares[warp];

  // ---- the copies' side: blocks in order, kStages - 1 ahead of the products
  typename Item::Cursor c;
  c.init(a, share);
  const uint32_t top_page = (uint32_t)(a.c.n_pages - 1);
  uint32_t page = 0, worst = 0;                  // lane % 16: the page of its key of the next block
  auto look = [&]() {
    if (!c.more()) return;
    const int pos = min(c.t * kBlock + lane % 16, c.total() - 1);
    page = (uint32_t)__ldg(a.b.pages + (int64_t)c.b * a.b.pages_stride + a.c.page.div(pos));
  };
  look();
  int stage_in = 0, scale_stage = -1;
  uint32_t scale_byte = 0;
  auto issue = [&]() {
    // the scales of the block before have landed: lanes 0 .. 15 K's, 16 .. 31 V's
    if (E4M3 && scale_stage >= 0) scales[scale_stage * 32 + lane] = (uint8_t)scale_byte;
    scale_stage = -1;
    if (c.more()) {
      const int pos0 = c.t * kBlock, total = c.total(), head = c.head;
      const int pos = min(pos0 + lane % 16, total - 1);
      const int slot = pos - a.c.page.div(pos) * a.c.page.d;
      worst = max(worst, page);                  // a bad page is reported at the end
      const uint32_t pg = min(page, top_page);
      if (E4M3) {
        scale_byte = __ldg(a.c.scale[lane / 16].at(pg, slot, head));
        scale_stage = stage_in;
      }
      c.next(a);
      look();
      uint8_t* dst = ring + stage_in * L::kStage + lane * 16;
      const Rows& kr = a.c.x[0];
      const uint8_t* k = kr.of_head(head) + q * 16;
#pragma unroll
      for (int kg = 0; kg < 2; ++kg) {
        const uint32_t p = __shfl_sync(0xffffffffu, pg, g + 8 * kg);
        const int s = __shfl_sync(0xffffffffu, slot, g + 8 * kg);
        const uint8_t* src = k + kr.offset(p, s);
        const bool on = pos0 + g + 8 * kg < total;
#pragma unroll
        for (int i = 0; i < L::kKCopies; ++i)
          ptx::cp_async16_or_zero(dst + (kg * L::kKCopies + i) * 512, src + i * 64,
                                  on && (4 * i + q) * 16 < a.D * (E4M3 ? 1 : 2));
      }
      const Rows& vr = a.c.x[1];
      const uint8_t* v = vr.of_head(head) + g * (L::kVBytes < 16 ? 8 : 16);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const int key = 2 * q + (kk & 1) + 8 * (kk >> 1);
        const uint32_t p = __shfl_sync(0xffffffffu, pg, key);
        const int s = __shfl_sync(0xffffffffu, slot, key);
        const uint8_t* src = v + vr.offset(p, s);
        const bool on = pos0 + key < total;
        if (L::kVBytes < 16) {                   // e4m3, 64 elements: 8 codes a lane
          ptx::cp_async8_or_zero(ring + stage_in * L::kStage + L::kVPart + (kk * 32 + lane) * 8,
                                 src, on && g * 8 < a.D);
        } else {
#pragma unroll
          for (int i = 0; i < L::kVBytes / 16; ++i)
            ptx::cp_async16_or_zero(dst + L::kVPart + (kk * (L::kVBytes / 16) + i) * 512,
                                    src + i * 128,
                                    on && (g + 8 * i) * 16 < a.D * (E4M3 ? 1 : 2));
        }
      }
    }
    ptx::cp_async_commit();
    if (++stage_in == L::kStages) stage_in = 0;
  };
#pragma unroll 1
  for (int i = 0; i < L::kStages - 1; ++i) issue();

  // ---- the products' side
  const Score sc = Score::of(a);
  const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
  typename Item::Walker w;
  typename Item::Segment s;
  w.init(a, share);
  int stage = 0;
  while (w.next(a, &s)) {
    const int rows = Item::group_rows(a, s);
    int node[MT][2];
    int64_t out_row[MT][2];
    bool valid[MT][2];
    uint4 qf[MT == 1 ? 2 : 1][MT == 1 ? kQChunks : 1];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * mt + 8 * h + g;
        valid[mt][h] = row < rows;
        const int grow = s.group * L::kRows + (valid[mt][h] ? row : 0);
        node[mt][h] = a.group.div(grow);
        const int qh = s.head * a.G + grow - node[mt][h] * a.G;
        out_row[mt][h] = (int64_t)(s.row0 + node[mt][h]) * a.Hq + qh;
        const uint8_t* src = a.q + (int64_t)(s.row0 + node[mt][h]) * a.q_row + qh * a.q_head;
#pragma unroll
        for (int j = 0; j < kQChunks; ++j) {
          // the chunk of 8 elements that meets this lane's j-th half chunk of codes, or chunk, of K
          const int chunk = E4M3 ? 8 * (j / 2) + 2 * q + j % 2 : 4 * j + q;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (valid[mt][h] && chunk * 8 < a.D) x = __ldg(reinterpret_cast<const uint4*>(src) + chunk);
          x.x ^= flip;
          x.y ^= flip;
          x.z ^= flip;
          x.w ^= flip;
          if (E4M3 && !F16) {
            const uint2 lo = swap_middle(make_uint2(x.x, x.y)), hi = swap_middle(make_uint2(x.z, x.w));
            x = make_uint4(lo.x, lo.y, hi.x, hi.y);
          }
          if (MT == 1) qf[h][j] = x;
          else q_mem[((mt * 2 + h) * kQChunks + j) * 32 + lane] = x;
        }
      }
    float o[MT][kTiles][4], mref[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      mref[mt][0] = mref[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[mt][t][k] = 0.f;
    }
    bool any_bad = false;

#pragma unroll 1
    for (int t = s.t0; t < s.t1; ++t) {
      issue();
      ptx::cp_async_wait_group<L::kStages - 1>();
      __syncwarp();
      const uint8_t* src = ring + stage * L::kStage + lane * 16;
      const uint8_t* sb = scales + stage * 32;
      const uint8_t* v_src = ring + stage * L::kStage + L::kVPart +
                             lane * (L::kVBytes < 16 ? 8 : 16);
      if (++stage == L::kStages) stage = 0;
      const int pos0 = t * kBlock;
      const bool masked = pos0 + kBlock > s.start;
      uint32_t kb[2], vb[4];                     // scale bytes of this lane's keys
      bool easy = true;
      if (E4M3) {
        kb[0] = sb[g];
        kb[1] = sb[g + 8];
        const uint32_t v01 = *reinterpret_cast<const uint16_t*>(sb + 16 + 2 * q);
        const uint32_t v23 = *reinterpret_cast<const uint16_t*>(sb + 24 + 2 * q);
        vb[0] = v01 & 0xff;
        vb[1] = v01 >> 8;
        vb[2] = v23 & 0xff;
        vb[3] = v23 >> 8;
        easy = __all_sync(0xffffffffu, easy_scale<F16>(kb[0]) && easy_scale<F16>(kb[1]) &&
                                           easy_scale<F16>(vb[0]) && easy_scale<F16>(vb[1]) &&
                                           easy_scale<F16>(vb[2]) && easy_scale<F16>(vb[3]));
      }
      // S: a lane's rows g and g + 8, keys 2q, 2q + 1 of both groups of eight
      float x[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int kg = 0; kg < 2; ++kg)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[mt][kg][k] = 0.f;
#pragma unroll
      for (int i = 0; i < L::kKCopies; ++i) {
        uint4 kc[2];
#pragma unroll
        for (int kg = 0; kg < 2; ++kg)
          kc[kg] = *reinterpret_cast<const uint4*>(src + (kg * L::kKCopies + i) * 512);
#pragma unroll
        for (int hc = 0; hc < (E4M3 ? 2 : 1); ++hc) {      // a chunk of Q: two steps
          uint4 qa[MT], qb[MT];
          const int j = E4M3 ? 2 * i + hc : i;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            qa[mt] = MT == 1 ? qf[0][MT == 1 ? j : 0] : q_mem[(mt * 2 * kQChunks + j) * 32 + lane];
            qb[mt] = MT == 1 ? qf[MT == 1 ? 1 : 0][MT == 1 ? j : 0]
                             : q_mem[((mt * 2 + 1) * kQChunks + j) * 32 + lane];
          }
#pragma unroll
          for (int kg = 0; kg < 2; ++kg) {
            uint2 b0, b1;                        // B of the two steps
            if (E4M3) {
              const uint32_t w0 = hc ? kc[kg].z : kc[kg].x, w1 = hc ? kc[kg].w : kc[kg].y;
              if (easy) {
                const uint32_t m = scale_mul2<F16>(kb[kg]);
                b0 = scale_codes<F16>(w0, m);
                b1 = scale_codes<F16>(w1, m);
              } else {
                b0 = scale_codes_any<F16>(w0, kb[kg]);
                b1 = scale_codes_any<F16>(w1, kb[kg]);
              }
            } else {
              b0 = make_uint2(kc[kg].x, kc[kg].y);
              b1 = make_uint2(kc[kg].z, kc[kg].w);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma<F16>(x[mt][kg], qa[mt].x, qb[mt].x, qa[mt].y, qb[mt].y, b0.x, b0.y);
              mma<F16>(x[mt][kg], qa[mt].z, qb[mt].z, qa[mt].w, qb[mt].w, b1.x, b1.y);
            }
          }
        }
      }
      // exponents, and whether a row's m has to move
      uint32_t see[MT][2];
      bool over = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          see[mt][h] = 0xffffffffu;
          if (masked)
            see[mt][h] = sees_32(a.mask ? a.mask + (int64_t)(s.row0 + node[mt][h]) * a.mask_stride
                                        : nullptr,
                                 s.rows, node[mt][h], pos0 - s.start) >> (2 * q);
          float mx = -INFINITY;
#pragma unroll
          for (int kg = 0; kg < 2; ++kg)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& v = x[mt][kg][2 * h + e];
              v = sc.cap2 > 0.f ? capped(sc, v) : v * sc.sl2;
              if (!masked || (see[mt][h] >> (8 * kg + e)) & 1) mx = fmaxf(mx, v);
            }
          over |= mx > mref[mt][h] + (mref[mt][h] == -INFINITY ? 0.f : kShift + 8.f);
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float mx = -INFINITY;
#pragma unroll
            for (int kg = 0; kg < 2; ++kg)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (!masked || (see[mt][h] >> (8 * kg + e)) & 1)
                  mx = fmaxf(mx, x[mt][kg][2 * h + e]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float old = mref[mt][h];
            if (mx > old + (old == -INFINITY ? 0.f : kShift + 8.f)) {
              mref[mt][h] = mx - kShift;
              const float back = old == -INFINITY ? 0.f : ex2(old - mref[mt][h]);
              l[mt][h] *= back;
#pragma unroll
              for (int c8 = 0; c8 < kTiles; ++c8) {
                o[mt][c8][2 * h] *= back;
                o[mt][c8][2 * h + 1] *= back;
              }
            }
          }
      }
      // weights, as the A operand of the second product
      uint32_t p[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float sub = mref[mt][h] == -INFINITY ? 0.f : mref[mt][h];
#pragma unroll
          for (int kg = 0; kg < 2; ++kg) {
            float w0 = ex2(x[mt][kg][2 * h] - sub), w1 = ex2(x[mt][kg][2 * h + 1] - sub);
            if (masked) {
              w0 = (see[mt][h] >> (8 * kg)) & 1 ? w0 : 0.f;
              w1 = (see[mt][h] >> (8 * kg + 1)) & 1 ? w1 : 0.f;
            }
            l[mt][h] += w0 + w1;
            p[mt][2 * kg + h] = pack2<F16>(w0, w1);
          }
        }
      // O += P V
      const int draft = s.start - pos0;          // first key of the block that is draft
      if (E4M3) {
        uint32_t vw[4][4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (L::kVBytes < 16) {
            const uint2 y = *reinterpret_cast<const uint2*>(v_src + kk * 256);
            vw[kk][0] = y.x;
            vw[kk][1] = y.y;
          } else {
            const uint4 y = *reinterpret_cast<const uint4*>(v_src + kk * 512);
            vw[kk][0] = y.x;
            vw[kk][1] = y.y;
            vw[kk][2] = y.z;
            vw[kk][3] = y.w;
          }
          const int key = 2 * q + (kk & 1) + 8 * (kk >> 1);
          if (masked && vb[kk] == 255 && key >= draft) {   // draft, or past the end
#pragma unroll
            for (int i = 0; i < L::kVBytes / 4; ++i) vw[kk][i] = 0;
            vb[kk] = 127;
            if (pos0 + key < s.start + s.rows) {
              atomicOr(&bad[(key - draft) >> 5], 1u << ((key - draft) & 31));
              any_bad = true;
            }
          }
        }
        const uint32_t m01 = (scale_mul2<F16>(vb[0]) & 0xffffu) | (scale_mul2<F16>(vb[1]) << 16);
        const uint32_t m23 = (scale_mul2<F16>(vb[2]) & 0xffffu) | (scale_mul2<F16>(vb[3]) << 16);
#pragma unroll
        for (int i = 0; i < L::kVBytes / 4; ++i) {
          uint32_t b0[4], b1[4];
          if (easy) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint2 y = pair_codes<F16>(vw[0][i], vw[1][i], h, m01);
              const uint2 z = pair_codes<F16>(vw[2][i], vw[3][i], h, m23);
              b0[2 * h] = y.x;
              b0[2 * h + 1] = y.y;
              b1[2 * h] = z.x;
              b1[2 * h + 1] = z.y;
            }
          } else {
            const uint4 y = pair_codes_any<F16>(vw[0][i], vb[0], vw[1][i], vb[1]);
            const uint4 z = pair_codes_any<F16>(vw[2][i], vb[2], vw[3][i], vb[3]);
            b0[0] = y.x;
            b0[1] = y.y;
            b0[2] = y.z;
            b0[3] = y.w;
            b1[0] = z.x;
            b1[1] = z.y;
            b1[2] = z.z;
            b1[3] = z.w;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              mma<F16>(o[mt][4 * i + k], p[mt][0], p[mt][1], p[mt][2], p[mt][3], b0[k], b1[k]);
        }
      } else {
#pragma unroll
        for (int cc = 0; cc < DP / 64; ++cc) {
          uint32_t vw[4][4];
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            uint4 y = *reinterpret_cast<const uint4*>(v_src + (kk * (DP / 64) + cc) * 512);
            if (masked) {
              const int key = 2 * q + (kk & 1) + 8 * (kk >> 1);
              if (key >= draft && pos0 + key < s.start + s.rows && zero_nonfinite<F16>(&y)) {
                atomicOr(&bad[(key - draft) >> 5], 1u << ((key - draft) & 31));
                any_bad = true;
              }
            }
            vw[kk][0] = y.x;
            vw[kk][1] = y.y;
            vw[kk][2] = y.z;
            vw[kk][3] = y.w;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t sel = h ? 0x7632 : 0x5410;
              const uint32_t b0 = __byte_perm(vw[0][i], vw[1][i], sel);
              const uint32_t b1 = __byte_perm(vw[2][i], vw[3][i], sel);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                mma<F16>(o[mt][8 * cc + 2 * i + h], p[mt][0], p[mt][1], p[mt][2], p[mt][3], b0, b1);
            }
        }
      }
    }

    // the segment's result
    const bool whole = s.whole();
    const int64_t part = 2 * worker + (s.t0 == 0 ? 1 : 0);
    float* part_o = a.part_o + part * (L::kRows * DP);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float sum = l[mt][h];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const float inv = 1.f / sum;
        if (whole && valid[mt][h]) {
          uint16_t* out = a.out + out_row[mt][h] * a.D;
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int c8 = 0; c8 < kTiles / 8; ++c8) {
              const int d = E4M3 ? (DP / 8) * (2 * q + e) + 8 * c8 : 8 * (2 * q + e) + 64 * c8;
              uint32_t y[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                y[k] = sum == 0.f ? 0u
                                  : pack2<F16>(o[mt][8 * c8 + 2 * k][2 * h + e] * inv,
                                               o[mt][8 * c8 + 2 * k + 1][2 * h + e] * inv);
              if (d < a.D) *reinterpret_cast<uint4*>(out + d) = make_uint4(y[0], y[1], y[2], y[3]);
            }
          if (q == 0 && a.lse)
            a.lse[out_row[mt][h]] = sum == 0.f ? -INFINITY : (mref[mt][h] + log2f(sum)) * kLn2;
        }
        if (!whole && q == 0)
          a.part_ml[part * L::kRows + 16 * mt + 8 * h + g] = make_float2(mref[mt][h], sum);
      }
      if (!whole) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
          reinterpret_cast<float4*>(part_o)[(mt * kTiles + t) * 32 + lane] =
              make_float4(o[mt][t][0], o[mt][t][1], o[mt][t][2], o[mt][t][3]);
      }
    }
    if (!whole && lane == 0) a.part_of[part] = Item::part_of(s, share.total, workers);
    if (__any_sync(0xffffffffu, any_bad)) {
      __syncwarp();
#pragma unroll 1
      for (int i = 0; i < 2 * MT; ++i) {         // one lane a row
        const int row = 8 * i + g;
        if (q != 0 || row >= rows) continue;
        const int grow = s.group * L::kRows + row, nd = a.group.div(grow);
        add_nonfinite<F16, E4M3, DP>(
            a, bad, a.mask ? a.mask + (int64_t)(s.row0 + nd) * a.mask_stride : nullptr, s.b, s.rows,
            s.start, s.head, nd,
            whole ? a.out + ((int64_t)(s.row0 + nd) * a.Hq + s.head * a.G + grow - nd * a.G) * a.D
                  : nullptr,
            part_o, row);
      }
      __syncwarp();
      if (lane < DSPARK_TREE_MAX_NODES / 32) bad[lane] = 0;
      __syncwarp();
    }
  }
  ptx::cp_async_wait_group<0>();
  if (worst > top_page) set_status(a.status, DSPARK_EPAGES);
}

// Joins the parts of the items that several warps share: an item of P parts has
// P blocks, which take its pieces of four accumulator tiles in turn; the eight
// warps of a block take every eighth part and are then added in order.
constexpr int kJoinThreads = 256;

template <bool F16, bool E4M3, int DP, int MT>
__global__ void __launch_bounds__(kJoinThreads) few_join_kernel(const __grid_constant__ AttendArgs a) {
  using Item = Work<kBlock, 16 * MT>;
  constexpr int kTiles = DP / 8, kRows = 16 * MT;
  __shared__ float4 sum_o[8][4][32];
  __shared__ float2 sum_ml[8][2][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 of = a.part_of[blockIdx.x];
  const int parts = of.w >> 16, first = of.w & 0xffff, head = of.y, group = of.z;
  if (parts == 0) return;
  bool ok;
  const typename Item::Request r = Item::load_request(a, of.x, &ok);
  const int rows = min(kRows, r.rows * a.G - group * kRows);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, q = lane & 3;
  for (int piece = (int)blockIdx.x / 2 - first; piece < MT * kTiles / 4; piece += parts) {
    const int mt = piece * 4 / kTiles;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float4 o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int i = warp; i < parts; i += 8) {
      const int64_t part = 2 * (first + i) + (i == 0 ? 1 : 0);
      const float4* src = reinterpret_cast<const float4*>(a.part_o + part * (kRows * DP)) +
                          piece * 4 * 32 + lane;
      float4 x[4];
      float2 ml[2];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = src[k * 32];
#pragma unroll
      for (int h = 0; h < 2; ++h) ml[h] = a.part_ml[part * kRows + 16 * mt + 8 * h + g];
      float wo[2], wx[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float m_new = fmaxf(m[h], ml[h].x), sub = m_new == -INFINITY ? 0.f : m_new;
        wo[h] = ex2(m[h] - sub);
        wx[h] = ex2(ml[h].x - sub);
        m[h] = m_new;
        l[h] = l[h] * wo[h] + ml[h].y * wx[h];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[k].x = o[k].x * wo[0] + x[k].x * wx[0];
        o[k].y = o[k].y * wo[0] + x[k].y * wx[0];
        o[k].z = o[k].z * wo[1] + x[k].z * wx[1];
        o[k].w = o[k].w * wo[1] + x[k].w * wx[1];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sum_o[warp][k][lane] = o[k];
#pragma unroll
    for (int h = 0; h < 2; ++h) sum_ml[warp][h][lane] = make_float2(m[h], l[h]);
    __syncthreads();
    if (warp < 4) {                              // warp k finishes tile k of the piece
      const int live = min(8, parts), tile = (piece * 4 + warp) % kTiles;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * mt + 8 * h + g;
        if (row >= rows) continue;
        float top = -INFINITY;
        for (int i = 0; i < live; ++i) top = fmaxf(top, sum_ml[i][h][lane].x);
        const float sub = top == -INFINITY ? 0.f : top;
        float sum = 0.f, y[2] = {0.f, 0.f};
        for (int i = 0; i < live; ++i) {
          const float w = ex2(sum_ml[i][h][lane].x - sub);
          const float4 x = sum_o[i][warp][lane];
          sum = fmaf(sum_ml[i][h][lane].y, w, sum);
          y[0] = fmaf(h ? x.z : x.x, w, y[0]);
          y[1] = fmaf(h ? x.w : x.y, w, y[1]);
        }
        const int grow = group * kRows + row, node = a.group.div(grow);
        const int64_t out_row = (int64_t)(r.row0 + node) * a.Hq + head * a.G + grow - node * a.G;
        const float inv = 1.f / sum;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int n = 2 * q + e;
          const int d = E4M3 ? (DP / 8) * n + tile : 8 * n + tile % 8 + tile / 8 * 64;
          if (d < a.D)
            a.out[out_row * a.D + d] = sum == 0.f ? 0 : (uint16_t)pack2<F16>(y[e] * inv, 0.f);
        }
        if (piece % (kTiles / 4) == 0 && warp == 0 && q == 0 && a.lse)
          a.lse[out_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
      }
    }
    __syncthreads();
  }
}

template <bool F16, bool E4M3, int DP, int MT>
cudaError_t launch(const AttendArgs& a, cudaStream_t stream) {
  using L = Few<E4M3, DP, MT>;
  few_kernel<F16, E4M3, DP, MT><<<a.n_cta, L::kThreads, L::kSmem, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the join may be set up while the main kernel runs; it waits for it itself
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * few_workers(a.n_cta, MT));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_join_kernel<F16, E4M3, DP, MT>, a);
}

template <bool F16, bool E4M3, int DP, int MT>
cudaError_t setup() {
  using L = Few<E4M3, DP, MT>;
  static_assert(L::kSmem <= 232448, "shared memory of an SM");
  cudaError_t e = cudaFuncSetAttribute(few_kernel<F16, E4M3, DP, MT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  // the main kernel's split of shared memory and L1: another would have the SMs
  // drained and set up anew between the two
  return cudaFuncSetAttribute(few_join_kernel<F16, E4M3, DP, MT>,
                              cudaFuncAttributePreferredSharedMemoryCarveout,
                              cudaSharedmemCarveoutMaxShared);
}

template <bool F16, int DP>
cudaError_t setup_all() {
  cudaError_t e = setup<F16, false, DP, 1>();
  if (e == cudaSuccess) e = setup<F16, false, DP, 2>();
  if (e == cudaSuccess) e = setup<F16, true, DP, 1>();
  if (e == cudaSuccess) e = setup<F16, true, DP, 2>();
  return e;
}

template <bool F16, bool E4M3>
cudaError_t launch_for(const AttendArgs& a, int tiles, cudaStream_t stream) {
  if (padded_dim(a.D) == 64)
    return tiles == 1 ? launch<F16, E4M3, 64, 1>(a, stream) : launch<F16, E4M3, 64, 2>(a, stream);
  return tiles == 1 ? launch<F16, E4M3, 128, 1>(a, stream) : launch<F16, E4M3, 128, 2>(a, stream);
}

}  // namespace

int few_workers(int n_cta, int tiles) {
  return n_cta * (tiles == 1 ? Few<false, 128, 1>::kWarps : Few<false, 128, 2>::kWarps);
}

cudaError_t few_setup(bool f16, int D) {
  if (padded_dim(D) == 64) return f16 ? setup_all<true, 64>() : setup_all<false, 64>();
  return f16 ? setup_all<true, 128>() : setup_all<false, 128>();
}

cudaError_t few_launch(const AttendArgs& a, int tiles, bool f16, bool e4m3, cudaStream_t stream) {
  if (f16) return e4m3 ? launch_for<true, true>(a, tiles, stream) : launch_for<true, false>(a, tiles, stream);
  return e4m3 ? launch_for<false, true>(a, tiles, stream) : launch_for<false, false>(a, tiles, stream);
}

}  // namespace tree
}  // namespace dspark
