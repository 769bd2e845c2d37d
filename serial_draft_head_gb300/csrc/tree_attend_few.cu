// tree_attend_few.cu -- attention of few drafted rows (single tokens, short
// chains: dspark_tree_attend has the rule) over a paged cache.
//
// Items are 16 rows by blocks of 16 (e4m3: 32) keys, a worker is a CTA (tree_items.cuh
// says how the work is cut, and the mathematics).  The warps of a CTA take a
// segment's blocks in turn, each with its own O, m and l, and meet at its end.
// With so few rows K and V are used once from where they land, and the memory
// rate bounds the kernel; tcgen05 tiles of 128 rows would be mostly padding, and
// what they need round them (a ring handed between warps, barriers, tensor
// memory) cost more than the products.  So the products are mma.sync m16n8k16,
// fed from registers:
//
//  - S = Q K^T: lane (g, q) = (lane / 4, lane % 4) holds B of key g and four
//    elements of it a step.  The order of the elements along the head is free as
//    long as Q has the same: lane q takes 16-byte chunks q, q + 4, ... of the row
//    as they lie, and Q's A operand is laid out by the same chunks.
//  - O = P V: P's A operand is S's accumulator, packed.  B of lane (g, q) is keys
//    2q, 2q + 1, 2q + 8, 2q + 9 at column g of every 8-column tile; the columns'
//    order is free too, so lane g takes 16-byte chunks g (and g + 8) of the four
//    rows, and pairs of keys are put together by byte permutations.
//
// So every thread reads just the 16-byte chunks that it copied itself: the ring
// in shared memory (cp.async, a stage is a block of K and V) needs no barrier,
// only the thread's own wait.
//
// e4m3: the products are f16, which holds every code, one conversion for two
// codes.  K's scale goes on the scores (fp32).  V's goes into the codes: exact in
// f16 for scales 2^-14 .. 2^7; keys with others get a product of their own in the
// handle's type, code times scale as the cache reads back (64 single tokens with such
// a key in every block: 318 us, without 173).  bf16 rows of Q are brought to f16 by a
// power of two a row (exact for elements down to 2^-32 of the row's largest, below
// that to 2^-40 of it).
//
// What bounds it.  128 single tokens of 500 to 9,000 over e4m3 (64 heads on 8):
// 317 us, 3.7 TB/s; DRAM at 1.04 times the cache's bytes, 850 warp instructions a
// block of 32 keys (conversions, the products, V's scales), issued at 34% of the
// slots by the three warps a scheduler that registers and rings leave, held by
// fixed latencies.  The same over bf16 up to 5,000 tokens: 293 us, 4.9 TB/s.  One
// token over 517: 12 us on the device, a chain of dependent steps (lengths, page,
// K, the warps' meeting, the other CTAs' parts).
#include "tree_items.cuh"

namespace dspark {
namespace tree {
namespace {

template <bool E4M3, int DP>
struct Few {
  static constexpr int kRows = 16;
  // e4m3: what a block costs beside its data is spread over twice the keys
  static constexpr int kBlock = E4M3 ? 32 : 16;
  // units an item counts beside its blocks, for Q, the first copies and the warps'
  // meeting (128 single tokens over e4m3: 1 385 us, 10 339, 20 322, 40 330, 60 345)
  static constexpr int kExtra = 20;
  static constexpr int kWarps = E4M3 ? 12 : 10;          // as many as registers and rings allow
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kBytes = DP * (E4M3 ? 1 : 2);     // of a cached row
  static constexpr int kGroups = kBlock / 8;             // of eight keys
  static constexpr int kKCopies = kBytes / 64;           // 16-byte chunks a lane, of a row of K
  static constexpr int kVBytes = kBytes / 8;             // bytes a lane, of a row of V
  static constexpr int kStage = 2 * kBlock * kBytes;
  static constexpr int kVPart = kBlock * kBytes;         // V's place in a stage
  static constexpr int kStages = kStage == 8192 ? 2 : 3;
  static constexpr int kTiles = DP / 8;                  // column tiles of O
  static constexpr int kMerge = 4;                       // of them merged at a time
  static constexpr int kRing = kStages * kStage;         // of a warp
  static constexpr int kQ = kWarps * kRing;
  static constexpr int kOut = kQ;                        // the result in Q's place: [rows][DP]
  static constexpr int kBuf = kQ + kRows * DP * 2;       // [warp][kMerge][lane] float4
  // the scales of a stage: K's as bf16, V's as f16 (0 where it is none) and as bytes
  static constexpr int kScaleBytes = E4M3 ? 5 * kBlock : 0;
  static constexpr int kScales = kBuf + kWarps * kMerge * 512;   // [warp][stage]
  static constexpr int kSmem = kScales + kWarps * kStages * kScaleBytes;
  using Item = Work<kBlock, kRows, kExtra>;
};

struct FewState {
  float2 ml[16][16];                    // [warp][row]
  float2 fin[16];                       // a row's m of all warps, and 1 / l (l = 0: 0)
  float row_mul[16];                    // a row's factor on the raw scores
  uint32_t bad[DSPARK_TREE_MAX_NODES / 32];
  int64_t sums[16];
  Share share;
  int live[2];                          // there is a segment; the next one
  int join;                             // an item to join: first worker | parts << 16
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
      const float x = bad_value<F16, E4M3 ? kE4M3 : k16>(a, b, start + j, head, d);
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

// Joins the `parts` parts of an item that several CTAs share, the first of them
// worker `first`'s: a warp has a piece of four accumulator tiles and every
// kSplit-th part; the warps of a piece are then added in order, so that the
// result does not depend on which CTA came last.
template <bool F16, bool E4M3, int DP>
__device__ __noinline__ void join_parts(const AttendArgs& a, FewState& st, float4* sum_o, int first,
                                        int parts, int row0, int head, int group, int rows) {
  using L = Few<E4M3, DP>;
  constexpr int kRows = L::kRows, kPieces = L::kTiles / 4, kSplit = L::kWarps / kPieces;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, q = lane & 3;
  const int piece = warp % kPieces, split = warp / kPieces;
  if (split < kSplit) {
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float4 o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = split; i < parts; i += kSplit) {
      const int64_t part = 2 * (first + i) + (i == 0 ? 1 : 0);
      const float4* src = reinterpret_cast<const float4*>(a.part_o + part * (kRows * DP)) +
                          piece * 4 * 32 + lane;
      float4 x[4];
      float2 ml[2];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = __ldcg(src + k * 32);
#pragma unroll
      for (int h = 0; h < 2; ++h) ml[h] = __ldcg(a.part_ml + part * kRows + 8 * h + g);
      float wo[2], wx[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (8 * h + g >= rows) ml[h] = make_float2(-INFINITY, 0.f);     // no part has the row
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
    for (int k = 0; k < 4; ++k) sum_o[(warp * 4 + k) * 32 + lane] = o[k];
    if (piece == 0 && q == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) st.ml[split][8 * h + g] = make_float2(m[h], l[h]);
    }
  }
  __syncthreads();
  const int live = min(kSplit, parts);
#pragma unroll 1
  for (int tile = warp; tile < L::kTiles; tile += L::kWarps) {
    float4 x[kSplit];
#pragma unroll
    for (int i = 0; i < kSplit; ++i)
      x[i] = sum_o[((i * kPieces + tile / 4) * 4 + tile % 4) * 32 + lane];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 8 * h + g;
      if (row >= rows) continue;
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < kSplit; ++i)
        if (i < live) top = fmaxf(top, st.ml[i][row].x);
      const float sub = top == -INFINITY ? 0.f : top;
      float sum = 0.f, y[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kSplit; ++i) {
        if (i >= live) continue;
        const float2 ml = st.ml[i][row];
        const float w = ex2(ml.x - sub);
        sum = fmaf(ml.y, w, sum);
        y[0] = fmaf(h ? x[i].z : x[i].x, w, y[0]);
        y[1] = fmaf(h ? x[i].w : x[i].y, w, y[1]);
      }
      const int grow = group * kRows + row, node = a.group.div(grow);
      const int64_t out_row = (int64_t)(row0 + node) * a.Hq + head * a.G + grow - node * a.G;
      const float inv = 1.f / sum;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int n = 2 * q + e;
        const int d = E4M3 ? (DP / 8) * n + tile : 8 * n + tile % 8 + tile / 8 * 64;
        if (d < a.D)
          a.out[out_row * a.D + d] = sum == 0.f ? 0 : (uint16_t)pack2<F16>(y[e] * inv, 0.f);
      }
      if (tile == 0 && q == 0 && a.lse)
        a.lse[out_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
  }
}

// CAP: scores are capped.  A kernel of its own, for the capped form's code in the loop
// costs other calls: 64 single tokens of 500 to 6,800 over a 16-bit cache, no cap, 210
// us with it, 196 without; capped 222 (scores all far from the cap), 228 (near it).
template <bool F16, bool E4M3, int DP, bool CAP>
__global__ void __launch_bounds__(Few<E4M3, DP>::kThreads, 1)
    few_kernel(const __grid_constant__ AttendArgs a) {
  using L = Few<E4M3, DP>;
  using Item = typename L::Item;
  using Segment = typename Item::Segment;
  constexpr bool kHalf = F16 || E4M3;            // the products' type is f16
  constexpr int kTiles = L::kTiles, kGroups = L::kGroups, kBlock = L::kBlock;
  constexpr int kQChunks = DP / 32;              // 16-byte chunks of a row of Q a lane
  constexpr int kQWarp = L::kWarps - 2;          // the two warps that bring Q, eight rows each
  constexpr float kShift = kHalf ? 7.f : 0.f;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ FewState st;
  __shared__ typename Item::Walker walker;
  __shared__ Segment segments[2];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, q = lane & 3;
  uint8_t* ring = smem + warp * L::kRing;
  uint4* q_mem = reinterpret_cast<uint4*>(smem + L::kQ);
  uint8_t* scales = smem + L::kScales + warp * L::kStages * L::kScaleBytes;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x < DSPARK_TREE_MAX_NODES / 32) st.bad[threadIdx.x] = 0;
  Item::template plan<L::kThreads>(a, &st.share, st.sums);

  // ---- the copies' side: the warp's blocks in order, kStages - 1 ahead of the products
  BlockCursor<Item, L::kExtra> c;
  c.init(a, st.share, warp);
  const uint32_t top_page = (uint32_t)(a.c.n_pages - 1);
  const bool even = a.c.page.d % kBlock == 0;    // a block lies in one page
  uint32_t page = 0, worst = 0;                  // of the next block: its page, or that of key lane
  auto look = [&]() {
    if (!c.more) return;
    const int pos = c.t * kBlock + (even ? 0 : lane % kBlock);
    page = (uint32_t)__ldg(a.b.pages + (int64_t)c.b * a.b.pages_stride +
                           a.c.page.div(min(pos, c.start + c.rows - 1)));
  };
  look();
  int stage_in = 0, scale_stage = -1;
  uint32_t k_byte = 0, v_byte = 0, easy_stages = 0;     // bit: all of V's scales in the stage are easy
  auto issue = [&]() {
    // the scales of the block before have landed: lane = key
    if (E4M3 && scale_stage >= 0) {
      uint8_t* sb = scales + scale_stage * L::kScaleBytes;
      // 2^(byte - 127), of byte 0 a subnormal number
      reinterpret_cast<uint16_t*>(sb)[lane] = (uint16_t)(k_byte == 0 ? 0x40u : k_byte << 7);
      const bool easy = easy_scale<true>(v_byte);
      reinterpret_cast<uint16_t*>(sb + 2 * kBlock)[lane] =
          (uint16_t)(easy ? scale_mul2<true>(v_byte) : 0u);
      sb[4 * kBlock + lane] = (uint8_t)v_byte;
      easy_stages = easy_stages & ~(1u << scale_stage) |
                    (__all_sync(0xffffffffu, easy) ? 1u << scale_stage : 0u);
    }
    scale_stage = -1;
    if (c.more) {
      const int pos0 = c.t * kBlock, total = c.start + c.rows, head = c.head;
      const bool full = pos0 + kBlock <= total;
      worst = max(worst, page);                  // a bad page is reported at the end
      const uint32_t pg = min(page, top_page);
      const int pos = even ? pos0 : min(pos0 + lane % kBlock, total - 1);
      const int slot = pos - a.c.page.div(pos) * a.c.page.d;   // of the block, or of key lane
      if (E4M3) {
        const int key_slot = even ? slot + lane : slot;
        k_byte = __ldg(a.c.scale[0].at(pg, key_slot, head));
        v_byte = __ldg(a.c.scale[1].at(pg, key_slot, head));
        // a slot past the end holds anything: its codes are zeros here, its scale is 1
        // (one token over 600, the rest of its page not written: 16.4 to 12.2 us)
        if (!full && pos0 + lane >= total) v_byte = 127;
        scale_stage = stage_in;
      }
      c.next(a, warp, L::kWarps);
      look();
      uint8_t* dst = ring + stage_in * L::kStage + lane * 16;
      const Rows &kr = a.c.x[0], &vr = a.c.x[1];
      const uint8_t* k = kr.of_head(head) + q * 16;
      const uint8_t* v = vr.of_head(head) + g * (L::kVBytes < 16 ? 8 : 16);
      if (even) {
        k += kr.offset(pg, slot + g);
        v += vr.offset(pg, slot + 2 * q);
      }
      if (even && full && a.D == DP && L::kVBytes >= 16) {       // the common case, no predicates
#pragma unroll
        for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
          for (int i = 0; i < L::kKCopies; ++i)
            ptx::cp_async16(dst + (kg * L::kKCopies + i) * 512,
                            k + (uint64_t)(8 * kg) * kr.slot + i * 64);
#pragma unroll
        for (int kk = 0; kk < kBlock / 4; ++kk)
#pragma unroll
          for (int i = 0; i < L::kVBytes / 16; ++i)
            ptx::cp_async16(dst + L::kVPart + (kk * (L::kVBytes / 16) + i) * 512,
                            v + (uint64_t)((kk & 1) + 8 * (kk >> 1)) * vr.slot + i * 128);
      } else {
#pragma unroll
      for (int kg = 0; kg < kGroups; ++kg) {
        const uint8_t* src;
        if (even) {
          src = k + (uint64_t)(8 * kg) * kr.slot;
        } else {
          const uint32_t p = __shfl_sync(0xffffffffu, pg, g + 8 * kg);
          src = k + kr.offset(p, __shfl_sync(0xffffffffu, slot, g + 8 * kg));
        }
        const bool on = full || pos0 + g + 8 * kg < total;
#pragma unroll
        for (int i = 0; i < L::kKCopies; ++i)
          ptx::cp_async16_or_zero(dst + (kg * L::kKCopies + i) * 512, src + i * 64,
                                  on && (4 * i + q) * 16 < a.D * (E4M3 ? 1 : 2));
      }
#pragma unroll
      for (int kk = 0; kk < kBlock / 4; ++kk) {
        const int off = (kk & 1) + 8 * (kk >> 1), key = 2 * q + off;
        const uint8_t* src;
        if (even) {
          src = v + (uint64_t)off * vr.slot;
        } else {
          const uint32_t p = __shfl_sync(0xffffffffu, pg, key);
          src = v + vr.offset(p, __shfl_sync(0xffffffffu, slot, key));
        }
        const bool on = full || pos0 + key < total;
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
    }
    ptx::cp_async_commit();
    if (++stage_in == L::kStages) stage_in = 0;
  };

  // ---- Q of a segment: lane (g, q) of two warps the chunks that meet its K
  const Score sc = Score::of(a);
  const int q_row = 8 * (warp - kQWarp) + g;
  uint4 qx[kQChunks];
  auto load_q = [&](const Segment& s) {
    const int rows = Item::group_rows(a, s);
    const int grow = s.group * L::kRows + (q_row < rows ? q_row : 0), nd = a.group.div(grow);
    const uint8_t* src = a.q + (int64_t)(s.row0 + nd) * a.q_row +
                         (int64_t)(s.head * a.G + grow - nd * a.G) * a.q_head;
#pragma unroll
    for (int j = 0; j < kQChunks; ++j) {
      const int chunk = E4M3 ? 8 * (j / 2) + 2 * q + j % 2 : 4 * j + q;
      qx[j] = make_uint4(0, 0, 0, 0);
      if (q_row < rows && chunk * 8 < a.D)
        qx[j] = __ldg(reinterpret_cast<const uint4*>(src) + chunk);
    }
  };
  auto store_q = [&]() {
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
    float row_mul = CAP ? 1.f : sc.sl2, r = 1.f;
    if (E4M3 && !F16) {
      // the row's largest finite magnitude to [2^14, 2^15): r a power of two, exact
      uint32_t big = 0;
#pragma unroll
      for (int j = 0; j < kQChunks; ++j) {
        const uint32_t w[4] = {qx[j].x, qx[j].y, qx[j].z, qx[j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) big = max(big, max(finite_bits(w[k] << 16), finite_bits(w[k])));
      }
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      const int e = (int)(big >> 23);
      const int up = big == 0 ? 0 : min(127 + 14 - e, 126);
      r = __uint_as_float((uint32_t)(127 + up) << 23);
      // finite, so that a score of zero stays one
      row_mul = fminf(row_mul * __uint_as_float((uint32_t)(127 - up) << 23), 3.40282347e38f);
    }
    if (q == 0) st.row_mul[q_row] = row_mul;
#pragma unroll
    for (int j = 0; j < kQChunks; ++j) {
      uint32_t w[4] = {qx[j].x ^ flip, qx[j].y ^ flip, qx[j].z ^ flip, qx[j].w ^ flip};
      if (E4M3 && !F16) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = pack2<true>(to_float<false>((uint16_t)w[k]) * r,
                             to_float<false>((uint16_t)(w[k] >> 16)) * r);
      }
      q_mem[((warp - kQWarp) * kQChunks + j) * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  };
  if (threadIdx.x == 0) {
    walker.init(a, st.share);
    st.live[0] = walker.next(a, &segments[0]);
  }
#pragma unroll 1
  for (int i = 0; i < L::kStages - 1; ++i) issue();
  __syncthreads();
  if (st.live[0] && warp >= kQWarp) {
    load_q(segments[0]);
    store_q();
  }
  __syncthreads();

  // ---- the products' side
  int stage = 0, cur = 0;
  while (st.live[cur]) {
    const Segment& s = segments[cur];
    const int rows = Item::group_rows(a, s), t1 = s.t1, start = s.start;
    float o[kTiles][4], mref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    const float row_mul[2] = {st.row_mul[g], st.row_mul[g + 8]};
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[t][k] = 0.f;
    // the segment after this one, meanwhile
    if (threadIdx.x == L::kThreads - 1) st.live[cur ^ 1] = walker.next(a, &segments[cur ^ 1]);
#pragma unroll 1
    for (int t = s.t0 + warp; t < t1; t += L::kWarps) {
      issue();
      ptx::cp_async_wait_group<L::kStages - 1>();
      __syncwarp();
      const uint8_t* src = ring + stage * L::kStage + lane * 16;
      const uint8_t* sb = scales + stage * L::kScaleBytes;
      const bool easy = !E4M3 || easy_stages >> stage & 1;
      const uint8_t* v_src = ring + stage * L::kStage + L::kVPart +
                             lane * (L::kVBytes < 16 ? 8 : 16);
      if (++stage == L::kStages) stage = 0;
      const int pos0 = t * kBlock;
      const bool masked = pos0 + kBlock > start;
      // S: a lane's rows g and g + 8, keys 2q, 2q + 1 of every group of eight
      float x[kGroups][4];
#pragma unroll
      for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[kg][k] = 0.f;
#pragma unroll
      for (int i = 0; i < L::kKCopies; ++i) {
        uint4 kc[kGroups];
#pragma unroll
        for (int kg = 0; kg < kGroups; ++kg)
          kc[kg] = *reinterpret_cast<const uint4*>(src + (kg * L::kKCopies + i) * 512);
#pragma unroll
        for (int hc = 0; hc < (E4M3 ? 2 : 1); ++hc) {      // a chunk of Q: two steps
          const int j = E4M3 ? 2 * i + hc : i;
          const uint4 qa = q_mem[j * 32 + lane], qb = q_mem[(kQChunks + j) * 32 + lane];
          uint2 b0[kGroups], b1[kGroups];                  // B of the two steps
#pragma unroll
          for (int kg = 0; kg < kGroups; ++kg) {
            if (E4M3) {
              b0[kg] = e4m3x4_to_f16(hc ? kc[kg].z : kc[kg].x);
              b1[kg] = e4m3x4_to_f16(hc ? kc[kg].w : kc[kg].y);
            } else {
              b0[kg] = make_uint2(kc[kg].x, kc[kg].y);
              b1[kg] = make_uint2(kc[kg].z, kc[kg].w);
            }
          }
#pragma unroll
          for (int kg = 0; kg < kGroups; ++kg)
            mma<kHalf>(x[kg], qa.x, qb.x, qa.y, qb.y, b0[kg].x, b0[kg].y);
#pragma unroll
          for (int kg = 0; kg < kGroups; ++kg)
            mma<kHalf>(x[kg], qa.z, qb.z, qa.w, qb.w, b1[kg].x, b1[kg].y);
        }
      }
      // scores by K's scales (x times row_mul is the exponent), invisible ones -infinity
      if (E4M3) {
#pragma unroll
        for (int kg = 0; kg < kGroups; ++kg) {
          const uint32_t k01 = reinterpret_cast<const uint32_t*>(sb)[4 * kg + q];
          const float s0 = __uint_as_float(k01 << 16), s1 = __uint_as_float(k01 & 0xffff0000u);
          x[kg][0] *= s0;
          x[kg][1] *= s1;
          x[kg][2] *= s0;
          x[kg][3] *= s1;
        }
      }
      uint32_t see[2] = {~0u, ~0u};              // bit 8 kg + e: rows g and g + 8 see the key
      if (masked) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = 8 * h + g;
          const int nd = a.group.div(s.group * L::kRows + (row < rows ? row : 0));
          see[h] = sees_32(a.mask ? a.mask + (int64_t)(s.row0 + nd) * a.mask_stride : nullptr, s.rows,
                           nd, pos0 - start) >> (2 * q);
#pragma unroll
          for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!((see[h] >> (8 * kg + e)) & 1)) x[kg][2 * h + e] = -INFINITY;
        }
      }
      float mx[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(x[0][2 * h], x[0][2 * h + 1]);
#pragma unroll
        for (int kg = 1; kg < kGroups; ++kg)
          mx[h] = fmaxf(mx[h], fmaxf(x[kg][2 * h], x[kg][2 * h + 1]));
        mx[h] = mx[h] == -INFINITY ? -INFINITY : mx[h] * row_mul[h];
        // a visible score of -infinity is the cap's negative, an invisible one nothing
        constexpr uint32_t kMine = kGroups == 4 ? 0x03030303u : 0x0303u;
        if (CAP && (see[h] & kMine) != 0) mx[h] = capped(sc, mx[h], 0.f);
      }
      // the first visible key sets a row's m, later ones when the maximum has grown enough
      const bool over = mx[0] > mref[0] + (mref[0] == -INFINITY ? 0.f : kShift + 8.f) ||
                        mx[1] > mref[1] + (mref[1] == -INFINITY ? 0.f : kShift + 8.f);
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
          const float old = mref[h];
          if (mx[h] > old + (old == -INFINITY ? 0.f : kShift + 8.f)) {
            mref[h] = mx[h] - kShift;
            const float back = old == -INFINITY ? 0.f : ex2(old - mref[h]);
            l[h] *= back;
#pragma unroll
            for (int t8 = 0; t8 < kTiles; ++t8) {
              o[t8][2 * h] *= back;
              o[t8][2 * h + 1] *= back;
            }
          }
        }
      }
      // weights, as the A operand of the second product
      const float sub[2] = {mref[0] == -INFINITY ? 0.f : mref[0],
                            mref[1] == -INFINITY ? 0.f : mref[1]};
      if (!CAP) {
#pragma unroll
        for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[kg][k] = fmaf(x[kg][k], row_mul[k / 2], -sub[k / 2]);
      } else {
#pragma unroll
        for (int kg = 0; kg < kGroups; ++kg) {
          float raw[4], big = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            raw[k] = x[kg][k] * row_mul[k / 2];
            big = fmaxf(big, fabsf(raw[k]));
            x[kg][k] = capped_near(sc, raw[k], sub[k / 2]);
          }
          if (__any_sync(0xffffffffu, past_near(sc, big))) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float past = capped_past(sc, raw[k], sub[k / 2]);
              if (past_near(sc, raw[k])) x[kg][k] = past;
            }
          }
        }
      }
      uint32_t p[kGroups / 2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
          for (int e = 0; e < 2; ++e) x[kg][2 * h + e] = ex2(x[kg][2 * h + e]);
        // by the bits: an invisible key's exponent can be anything (-infinity times a
        // scale of zero)
        if (masked) {
#pragma unroll
          for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!((see[h] >> (8 * kg + e)) & 1)) x[kg][2 * h + e] = 0.f;
        }
#pragma unroll
        for (int kg = 0; kg < kGroups; ++kg) {
          const float w0 = x[kg][2 * h], w1 = x[kg][2 * h + 1];
          l[h] += w0 + w1;
          p[kg / 2][2 * (kg % 2) + h] = pack2<kHalf>(w0, w1);
        }
      }
      // O += P V, 16 keys at a time
      const int draft = start - pos0, last = start + s.rows - pos0;   // in the block
#pragma unroll
      for (int ks = 0; ks < kGroups / 2; ++ks) {
        if (E4M3) {
          uint32_t vw[4][4];
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (L::kVBytes < 16) {
              const uint2 y = *reinterpret_cast<const uint2*>(v_src + (4 * ks + kk) * 256);
              vw[kk][0] = y.x;
              vw[kk][1] = y.y;
            } else {
              const uint4 y = *reinterpret_cast<const uint4*>(v_src + (4 * ks + kk) * 512);
              vw[kk][0] = y.x;
              vw[kk][1] = y.y;
              vw[kk][2] = y.z;
              vw[kk][3] = y.w;
            }
          }
          auto product = [&]() {                 // by f16 scales
            const uint32_t* sv = reinterpret_cast<const uint32_t*>(sb + 2 * kBlock) + 8 * ks + q;
            const uint32_t m01 = sv[0], m23 = sv[4];
#pragma unroll
            for (int i = 0; i < L::kVBytes / 4; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t sel = h ? 0x7362 : 0x5140;  // two codes of two keys, key by key
                const uint2 y = scale_codes<true>(__byte_perm(vw[0][i], vw[1][i], sel), m01);
                const uint2 z = scale_codes<true>(__byte_perm(vw[2][i], vw[3][i], sel), m23);
                mma<true>(o[4 * i + 2 * h], p[ks][0], p[ks][1], p[ks][2], p[ks][3], y.x, z.x);
                mma<true>(o[4 * i + 2 * h + 1], p[ks][0], p[ks][1], p[ks][2], p[ks][3], y.y, z.y);
              }
          };
          if (easy) {
            product();
          } else {
            // keys whose scale is not easy count nothing in this product (their f16 scale
            // is 0) and alone in one more, in the handle's type: how a row's weights are
            // rounded does not go by keys that it does not see
            uint32_t vb[4];
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const int key = 16 * ks + 2 * q + (kk & 1) + 8 * (kk >> 1);
              vb[kk] = sb[4 * kBlock + key];
              if (masked && vb[kk] == 255 && key >= draft) {   // draft, or past the end
#pragma unroll
                for (int i = 0; i < L::kVBytes / 4; ++i) vw[kk][i] = 0;
                vb[kk] = 127;
                if (key < last) atomicOr(&st.bad[(key - draft) >> 5], 1u << ((key - draft) & 31));
              }
            }
            product();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (!easy_scale<true>(vb[kk])) continue;
#pragma unroll
              for (int i = 0; i < L::kVBytes / 4; ++i) vw[kk][i] = 0;
            }
            if (!F16) {                          // weights in the handle's type
#pragma unroll
              for (int k = 0; k < 4; ++k)
                p[ks][k] = pack2<false>(x[2 * ks + k / 2][2 * (k % 2)],
                                        x[2 * ks + k / 2][2 * (k % 2) + 1]);
            }
#pragma unroll
            for (int i = 0; i < L::kVBytes / 4; ++i) {
              const uint4 y = pair_codes_any<F16>(vw[0][i], vb[0], vw[1][i], vb[1]);
              const uint4 z = pair_codes_any<F16>(vw[2][i], vb[2], vw[3][i], vb[3]);
              const uint32_t b0[4] = {y.x, y.y, y.z, y.w}, b1[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma<F16>(o[4 * i + k], p[ks][0], p[ks][1], p[ks][2], p[ks][3], b0[k], b1[k]);
            }
          }
        } else {
#pragma unroll
          for (int cc = 0; cc < DP / 64; ++cc) {
            uint32_t vw[4][4];
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              uint4 y = *reinterpret_cast<const uint4*>(v_src + ((4 * ks + kk) * (DP / 64) + cc) * 512);
              if (masked) {
                const int key = 16 * ks + 2 * q + (kk & 1) + 8 * (kk >> 1);
                if (key >= draft && key < last && zero_nonfinite<F16>(&y))
                  atomicOr(&st.bad[(key - draft) >> 5], 1u << ((key - draft) & 31));
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
                mma<F16>(o[8 * cc + 2 * i + h], p[ks][0], p[ks][1], p[ks][2], p[ks][3],
                         __byte_perm(vw[0][i], vw[1][i], sel), __byte_perm(vw[2][i], vw[3][i], sel));
              }
          }
        }
      }
    }

    // the warps meet: O, m and l of the segment
    const bool whole = s.whole();
    const int64_t part = 2 * blockIdx.x + (s.t0 == 0 ? 1 : 0);
    const int live = min(L::kWarps, s.t1 - s.t0);          // warps that had a block
    float4* buf = reinterpret_cast<float4*>(smem + L::kBuf);
    uint16_t* out = reinterpret_cast<uint16_t*>(smem + L::kOut);
    auto out_row = [&](int row) {
      const int grow = s.group * L::kRows + row, nd = a.group.div(grow);
      return (int64_t)(s.row0 + nd) * a.Hq + s.head * a.G + grow - nd * a.G;
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float sum = l[h];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (q == 0) st.ml[warp][8 * h + g] = make_float2(mref[h], sum);
    }
    __syncthreads();
    const bool next_live = st.live[cur ^ 1];
    if (warp == 0 && lane < L::kRows) {          // a row a lane: m and l of all warps
      float top = -INFINITY, sum = 0.f;
      for (int i = 0; i < live; ++i) top = fmaxf(top, st.ml[i][lane].x);
      const float sub = top == -INFINITY ? 0.f : top;
      for (int i = 0; i < live; ++i) sum = fmaf(st.ml[i][lane].y, ex2(st.ml[i][lane].x - sub), sum);
      st.fin[lane] = make_float2(sub, sum == 0.f ? 0.f : 1.f / sum);
      if (lane < rows) {
        if (!whole) a.part_ml[part * L::kRows + lane] = make_float2(top, sum);
        else if (a.lse) a.lse[out_row(lane)] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
      }
    }
    if (next_live && warp >= kQWarp) load_q(segments[cur ^ 1]);
    __syncthreads();
    // every warp's O by its weight, kMerge accumulator tiles at a time
    const float w0 = ex2(mref[0] - st.fin[g].x), w1 = ex2(mref[1] - st.fin[g + 8].x);
#pragma unroll
    for (int pass = 0; pass < kTiles / L::kMerge; ++pass) {
      if (warp < live) {
#pragma unroll
        for (int k = 0; k < L::kMerge; ++k) {
          const float* v = o[pass * L::kMerge + k];
          buf[(warp * L::kMerge + k) * 32 + lane] =
              make_float4(v[0] * w0, v[1] * w0, v[2] * w1, v[3] * w1);
        }
      }
      __syncthreads();
      if (warp < L::kMerge) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < live; ++i) {
          const float4 v = buf[(i * L::kMerge + warp) * 32 + lane];
          y.x += v.x;
          y.y += v.y;
          y.z += v.z;
          y.w += v.w;
        }
        const int tile = pass * L::kMerge + warp;
        if (!whole) {
          reinterpret_cast<float4*>(a.part_o + part * (L::kRows * DP))[tile * 32 + lane] = y;
        } else {
          // l = 0: every weight was 0, and so is O
          const float i0 = st.fin[g].y, i1 = st.fin[g + 8].y;
          const int d0 = E4M3 ? (DP / 8) * 2 * q + tile : 16 * q + tile % 8 + tile / 8 * 64;
          const int d1 = d0 + (E4M3 ? DP / 8 : 8);
          out[g * DP + d0] = (uint16_t)pack2<F16>(y.x * i0, 0.f);
          out[g * DP + d1] = (uint16_t)pack2<F16>(y.y * i0, 0.f);
          out[(g + 8) * DP + d0] = (uint16_t)pack2<F16>(y.z * i1, 0.f);
          out[(g + 8) * DP + d1] = (uint16_t)pack2<F16>(y.w * i1, 0.f);
        }
      }
      __syncthreads();
    }
    if (whole) {
      for (int i = threadIdx.x; i < rows * (DP / 8); i += L::kThreads) {
        const int row = i / (DP / 8), chunk = i % (DP / 8);
        if (chunk * 8 < a.D)
          reinterpret_cast<uint4*>(a.out + out_row(row) * a.D)[chunk] =
              reinterpret_cast<const uint4*>(out)[i];
      }
    }
    uint32_t any_bad = 0;
#pragma unroll
    for (int k = 0; k < DSPARK_TREE_MAX_NODES / 32; ++k) any_bad |= st.bad[k];
    __syncthreads();
    if (next_live && warp >= kQWarp) store_q();
    if (any_bad != 0) {
      if (threadIdx.x < L::kRows && (int)threadIdx.x < rows) {
        const int nd = a.group.div(s.group * L::kRows + threadIdx.x);
        add_nonfinite<F16, E4M3, DP>(
            a, st.bad, a.mask ? a.mask + (int64_t)(s.row0 + nd) * a.mask_stride : nullptr, s.b, s.rows,
            s.start, s.head, nd, whole ? a.out + out_row(threadIdx.x) * a.D : nullptr,
            a.part_o + part * (L::kRows * DP), threadIdx.x);
      }
      __syncthreads();
      if (threadIdx.x < DSPARK_TREE_MAX_NODES / 32) st.bad[threadIdx.x] = 0;
    }
    if (!whole) {
      // the last CTA to leave its part of the item joins them all
      if (threadIdx.x == 0) {
        const int w = Item::part_of(s, st.share.cut).w;
        int* count = a.arrived + (w & 0xffff);
        __threadfence();
        const bool last = atomicAdd(count, 1) == (w >> 16) - 1;
        if (last) *count = 0;
        __threadfence();
        st.join = last ? w : 0;
      }
      __syncthreads();
      if (st.join)
        join_parts<F16, E4M3, DP>(a, st, buf, st.join & 0xffff, st.join >> 16, s.row0, s.head,
                                  s.group, rows);
    }
    __syncthreads();
    cur ^= 1;
  }
  ptx::cp_async_wait_group<0>();
  if (worst > top_page) set_status(a.status, DSPARK_EPAGES);
}

template <bool F16, bool E4M3, int DP, bool CAP>
cudaError_t launch(const AttendArgs& a, cudaStream_t stream) {
  using L = Few<E4M3, DP>;
  // launched while the kernel before it in the stream ends, which it waits for before
  // anything else (calls in a row: 14.3 to 12.3 us for 1 token)
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.n_cta);
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_kernel<F16, E4M3, DP, CAP>, a);
}

template <bool F16, bool E4M3, int DP>
cudaError_t setup() {
  using L = Few<E4M3, DP>;
  static_assert(L::kSmem + sizeof(FewState) + 512 <= 232448, "shared memory of an SM");
  const cudaError_t e = cudaFuncSetAttribute(
      few_kernel<F16, E4M3, DP, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(few_kernel<F16, E4M3, DP, true>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
}

template <bool F16, int DP>
cudaError_t setup_both() {
  const cudaError_t e = setup<F16, false, DP>();
  return e != cudaSuccess ? e : setup<F16, true, DP>();
}

template <bool F16, bool E4M3, int DP>
cudaError_t launch_cap(const AttendArgs& a, cudaStream_t stream) {
  return a.softcap > 0.f ? launch<F16, E4M3, DP, true>(a, stream)
                         : launch<F16, E4M3, DP, false>(a, stream);
}

template <bool F16, bool E4M3>
cudaError_t launch_for(const AttendArgs& a, cudaStream_t stream) {
  return padded_dim(a.D) == 64 ? launch_cap<F16, E4M3, 64>(a, stream)
                               : launch_cap<F16, E4M3, 128>(a, stream);
}

}  // namespace

cudaError_t few_setup(bool f16, int D) {
  if (padded_dim(D) == 64) return f16 ? setup_both<true, 64>() : setup_both<false, 64>();
  return f16 ? setup_both<true, 128>() : setup_both<false, 128>();
}

cudaError_t few_launch(const AttendArgs& a, bool f16, bool e4m3, cudaStream_t stream) {
  if (f16) return e4m3 ? launch_for<true, true>(a, stream) : launch_for<true, false>(a, stream);
  return e4m3 ? launch_for<false, true>(a, stream) : launch_for<false, false>(a, stream);
}

}  // namespace tree
}  // namespace dspark
