// tree_attend_few4.cuh -- attention of few drafted rows (single tokens, short chains:
// dspark_tree_attend has the rule) over a paged cache in 4 bits.
//
// Items are 8, 16 or 32 rows by blocks of 32 keys, a worker is a group of warps, four or a
// CTA's (tree_items.cuh says how the work is cut, and the mathematics).  The warps of a
// group take a segment's blocks in turn, each with its own O, m and l, and meet at its
// end; with four to a group the others of the SM go on meanwhile.
//
// Each warp has a ring of two blocks, which it fills itself by copies of 16 bytes a lane,
// so that nothing is handed between warps.  Where a page holds a head's slots and their
// scales next to each other (KVCache.zeros lays them so: RUNS), a block is a run of memory
// and a copy an address and an immediate offset.  (Bulk copies: by a warp for all others
// 340 cycles a block, more than the others need for it; by each warp for itself about 60
// instructions a block more than these.)
//
// A cached row of 128 elements is 72 bytes, so what bounds the kernel is less the memory
// than what is done to every element on the way to the products (f16 mma.sync
// m16n8k16): one conversion for two codes, one multiplication by their scales, exact.
// The products stand the other way round than those of tree_attend_few.cu: keys (for S)
// and columns of V (for O) are the 16 rows of A, the drafted rows the 8 columns of B, so
// that eight rows (a single token of a group of eight heads) fill a tile and O takes half
// the registers.
//
//  - S^T = K Q^T: lane (g, q) = (lane / 4, lane % 4) holds keys g and g + 8 of A.  The
//    order of the elements along the head is free as long as Q has the same: lane q takes
//    the q-th quarter of a row, two blocks under a scale each, as it lies.
//  - P^T's B operand is S^T's accumulator, packed and transposed by movmatrix.
//  - O^T = V^T P^T: A of lane (g, q) is column g and g + 8 of keys 2q, 2q + 1, 2q + 8,
//    2q + 9; the columns' order is free too, so lane g takes the g-th eighth of the rows,
//    one block, puts two keys' codes into bytes by four logic operations for 16, and
//    multiplies by the two keys' scales, which are a pair as ldmatrix hands them out
//    transposed.
//
// Keys stand in the products' rows in the order `row_key`, so that the rows that lanes
// read together lie in different banks.  Rows of Q are brought to f16 by a power of two
// a row.
//
// What bounds it.  128 single tokens of 500 to 9,000 (64 heads on 8): 147 us, 4.9 TB/s;
// 700 warp instructions a block, issued at 64% of the slots, held by fixed latencies and
// the pipes of the conversions and 16-bit products (without the products: 125).  19
// requests of 32,767: 128 us, 5.6 TB/s.  Items of 32 rows (16 chains of 8 over 300 to 6,000
// with 4 heads on one: 66 us of 56,874 keys, 72 of 64,643): two warps a scheduler, issued at 28%.
#pragma once

#include "tree_items.cuh"

namespace dspark {
namespace tree {
namespace {

// DP: head dimension as laid out, 64 or 128; NT: tiles of eight rows; GROUP: warps of a
// worker; RUNS: slots and scales lie next to each other.
template <int DP, int NT, int GROUP, bool RUNS>
struct Few4 {
  static constexpr int kRows = 8 * NT;
  static constexpr int kBlock = 32;
  static constexpr int kParts = kBlock / 8;              // of eight keys
  // units an item counts beside its blocks, for Q, the first copies and the warps'
  // meeting
  static constexpr int kExtra = GROUP == 4 ? 10 : 20;
  // as many as leave O, m and l in registers; with heads of 128 what a segment needs now and
  // then is spilled: 136 bytes at most (NT 1), 356 (2), 388 (4)
  static constexpr int kWarps = NT == 1 ? 16 : NT == 2 ? 12 : 8;
  static constexpr int kWorkers = kWarps / GROUP;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kBytes = DP / 2;                  // of a row of codes
  static constexpr int kScaleBytes = DP / 16;            // of its scales (RUNS)
  static constexpr int kChunks = kBytes / 16;            // 16-byte copies of a row
  static constexpr int kRowsAtOnce = 32 / kChunks;       // rows of one copy instruction
  static constexpr int kCopies = kBlock / kRowsAtOnce;
  static constexpr int kWords = kBytes / 16;             // 32-bit words a lane, of a row of K
  static constexpr int kVPart = kBlock * kBytes;         // V's place in a stage
  static constexpr int kScales = 2 * kVPart;             // and the scales' bytes
  static constexpr int kStage = kScales + (RUNS ? 2 * kBlock * kScaleBytes : 0);
  static constexpr int kStages = 2;
  static constexpr int kTiles = DP / 16;                 // of O^T
  static constexpr int kScale = kStages * kStage;        // a block's scales as f16: [K, V][key][8]
  static constexpr int kRing = kScale + 2 * kBlock * 16; // of a warp
  static constexpr int kQ = kWarps * kRing;              // [worker][NT][DP / 32][lane] 16 bytes
  static constexpr int kQBytes = kRows * DP * 2;
  static constexpr int kMerge = kQ + kWorkers * kQBytes; // [warp][row][kCols + 4] floats
  // columns merged at a time: all where there is room
  static constexpr int kPasses = kMerge + kWarps * kRows * (DP + 4) * 4 <= 232448 - 6144 ? 1 : 2;
  static constexpr int kCols = DP / kPasses;
  static constexpr int kMergeRow = kCols + 4;
  static constexpr int kMergeWarp = kRows * kMergeRow * 4;
  static constexpr int kSmem = kMerge + kWarps * kMergeWarp;
  using Item = Work<kBlock, kRows, kExtra>;
};

// A part of an item that others share, and what its join needs.
struct Left {
  int item;                             // first worker | parts << 16; 0: none
  int row0, head, group, rows;
};

template <int GROUP, int ROWS>
struct WorkerState {
  float2 ml[GROUP][ROWS];               // [warp][row]
  float2 fin[ROWS];                     // a row's m of all warps, and 1 / l (l = 0: 0)
  float2 row_mul[ROWS / 2];             // two rows' factors on the raw scores
  uint32_t bad[DSPARK_TREE_MAX_NODES / 32];
  int live[2];                          // there is a segment; the next one
  Left left[2];                         // the parts that the worker leaves: of its first item and its last
  int join[2];                          // whether all parts of theirs are there
};

// The warps of worker w meet.
template <int GROUP>
__device__ __forceinline__ void meet(int w) {
  asm volatile("bar.sync %0, %1;" ::"r"(w + 1), "n"(GROUP * 32) : "memory");
}

// The key of eight that stands in row r of a product.
__device__ __forceinline__ int row_key(int r) { return r ^ (r >> 1 & 1); }

__device__ __forceinline__ uint32_t pack_out(bool f16, float lo, float hi) {
  return f16 ? pack2<true>(lo, hi) : pack2<false>(lo, hi);
}

// The 8x8 matrix of 16-bit elements that a warp holds, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t saddr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}

// The scale bytes of a row, as many as its elements have blocks.
__device__ __forceinline__ uint2 load_scales(const uint8_t* p, int D) {
  uint2 r = make_uint2(0u, 0u);
  if (D == 128) {
    r = __ldg(reinterpret_cast<const uint2*>(p));
  } else if (D == 64) {
    r.x = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
    r.x = __ldg(h);
    if (D == 96) {
      r.x |= (uint32_t)__ldg(h + 1) << 16;
      r.y = __ldg(h + 2);
    }
  }
  return r;
}

// Eight f16 scales for the eight 16-byte-eighths of a row of 128 elements (64: each of
// four blocks twice).
template <int DP>
__device__ __forceinline__ uint4 spread_scales(uint2 b) {
  if (DP == 128)
    return make_uint4(__byte_perm(b.x, 0, 0x4140) << 7, __byte_perm(b.x, 0, 0x4342) << 7,
                      __byte_perm(b.y, 0, 0x4140) << 7, __byte_perm(b.y, 0, 0x4342) << 7);
  return make_uint4(__byte_perm(b.x, 0, 0x4040) << 7, __byte_perm(b.x, 0, 0x4141) << 7,
                    __byte_perm(b.x, 0, 0x4242) << 7, __byte_perm(b.x, 0, 0x4343) << 7);
}

// Whether one of a row's scale bytes is past those of numbers; and those, as 0.
__device__ __forceinline__ bool zero_nonnumbers(uint32_t* w) {
  const uint32_t over = __vcmpgtu4(*w, kTopScale * 0x01010101u);
  *w &= ~over;
  return over != 0;
}

// Overwrites a row's result, written by this CTA, with NaN where a draft row of V that
// it sees has a block that is none: 16-bit values (out), or the part's floats.
__device__ __noinline__ void add_nan(const AttendArgs& a, const uint32_t* bad,
                                     const uint32_t* mask_row, int b, int rows, int start, int head,
                                     int node, uint16_t* out, float* part) {
#pragma unroll 1
  for (int j = 0; j < rows; ++j) {
    if (!(sees_word(mask_row, rows, node, j >> 5) & bad[j >> 5] & (1u << (j & 31)))) continue;
    int64_t page;
    int slot;
    if (!locate(a.c, a.b, b, start + j, &page, &slot)) continue;
    const uint8_t* s = a.c.scale[1].at((uint32_t)page, slot, head);
#pragma unroll 1
    for (int d = 0; d < a.D; ++d) {
      if (s[d / 16] <= kTopScale) continue;
      if (out) out[d] = 0x7fffu;                 // NaN in f16 and in bf16
      else part[d] = __uint_as_float(0x7fffffffu);
    }
  }
}

// Joins the parts of an item that several workers share, in their order, so that the result
// does not depend on which came last.  A thread has four columns of a row and eight parts'
// loads in flight.
template <class L, int GROUP>
__device__ __noinline__ void join_parts(const AttendArgs& a, const Left& of, int tid) {
  constexpr int kRows = L::kRows, DP = L::kBytes * 2, kAtOnce = 8;
  const int first = of.item & 0xffff, parts = of.item >> 16;
  auto part_at = [&](int i) { return (int64_t)2 * (first + i) + (i == 0 ? 1 : 0); };
#pragma unroll 1
  for (int i = tid; i < of.rows * (DP / 4); i += GROUP * 32) {
    const int row = i / (DP / 4), c = i % (DP / 4);
    if (4 * c >= a.D) continue;
    float m = -INFINITY, l = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < parts; k0 += kAtOnce) {
      float4 x[kAtOnce];
      float2 ml[kAtOnce];
      float top = m;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + k < parts) {
          ml[k] = __ldcg(a.part_ml + part_at(k0 + k) * kRows + row);
          x[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + part_at(k0 + k) * (kRows * DP)) + i);
        }
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, ml[k].x);
      const float base = top == -INFINITY ? 0.f : top, old = ex2(m - base);
      m = top;
      l *= old;
      y.x *= old;
      y.y *= old;
      y.z *= old;
      y.w *= old;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const float w = ex2(ml[k].x - base);
        l = fmaf(ml[k].y, w, l);
        y.x = fmaf(x[k].x, w, y.x);
        y.y = fmaf(x[k].y, w, y.y);
        y.z = fmaf(x[k].z, w, y.z);
        y.w = fmaf(x[k].w, w, y.w);
      }
    }
    // l = 0: every weight was 0, and so is O
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int grow = of.group * kRows + row, node = a.group.div(grow);
    const int64_t to = (int64_t)(of.row0 + node) * a.Hq + of.head * a.G + grow - node * a.G;
    *reinterpret_cast<uint2*>(a.out + to * a.D + 4 * c) =
        make_uint2(pack_out(a.f16, y.x * inv, y.y * inv), pack_out(a.f16, y.z * inv, y.w * inv));
    if (c == 0 && a.lse) a.lse[to] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

template <int DP, int NT, int GROUP, bool RUNS, bool CAP>
__global__ void __launch_bounds__(Few4<DP, NT, GROUP, RUNS>::kThreads, 1)
    few4_kernel(const __grid_constant__ AttendArgs a) {
  using L = Few4<DP, NT, GROUP, RUNS>;
  using Item = typename L::Item;
  using Segment = typename Item::Segment;
  constexpr int kParts = L::kParts, kBlock = L::kBlock, kTiles = L::kTiles;
  constexpr int kWorkerThreads = GROUP * 32;
  constexpr float kShift = 7.f;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ WorkerState<GROUP, L::kRows> states[L::kWorkers];
  __shared__ Share shares[L::kWorkers];
  __shared__ int64_t sums[L::kThreads / 32];
  __shared__ typename Item::Walker walkers[L::kWorkers];
  __shared__ Segment all_segments[L::kWorkers][2];
  const int cta_warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, q = lane & 3;
  const int worker = cta_warp / GROUP, warp = cta_warp % GROUP;
  const int tid = threadIdx.x % kWorkerThreads;  // in the worker
  const int gk = row_key(g);
  WorkerState<GROUP, L::kRows>& st = states[worker];
  uint8_t* ring = smem + cta_warp * L::kRing;
  uint4* q_mem = reinterpret_cast<uint4*>(smem + L::kQ + worker * L::kQBytes);
  const uint32_t scale_mem = ptx::smem_u32(ring + L::kScale) +
                             (lane / 8 * 8 + row_key(lane % 8)) * 16;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid < DSPARK_TREE_MAX_NODES / 32) st.bad[tid] = 0;
  if (tid < 2) st.left[tid].item = 0;
  Item::template plan<L::kThreads, L::kWorkers>(a, shares, sums);
  const Share& share = shares[worker];
  Segment* segments = all_segments[worker];

  // ---- the copies' side: the warp's blocks in order, one ahead of the products
  BlockCursor<Item, L::kExtra> c;
  c.init(a, share, warp);
  const uint32_t top_page = (uint32_t)(a.c.n_pages - 1);
  const bool even = RUNS || a.c.page.d % 16 == 0;          // half a block lies in one page
  const bool in_two = RUNS && a.c.page.d % kBlock != 0;    // a block can lie in two
  // of the next block: the pages of its halves and (RUNS) their first slots, or that of key `lane`
  uint32_t page[2] = {0, 0}, worst = 0;
  int slots[2] = {0, 0};
  // RUNS: what changes with the request and with the head alone is kept from block to block:
  // the request's row of the table; this lane's places in the head's codes of K and V, and
  // in the scales, lanes 0 .. K's, as many after them V's
  constexpr int kScaleLanes = kBlock * L::kScaleBytes / 16;
  const int32_t* table = nullptr;
  const uint8_t *k_head = nullptr, *v_head = nullptr, *s_head = nullptr;
  int at_b = -1, at_head = -1;
  const Rows scale_rows = a.c.scale[lane / kScaleLanes % 2];
  auto look = [&]() {
    if (!c.more) return;
    if (RUNS) {
      if (c.b != at_b) {
        at_b = c.b;
        table = a.b.pages + (int64_t)c.b * a.b.pages_stride;
      }
      const int pos = c.t * kBlock, i = a.c.page.div(pos);
      slots[0] = pos - i * a.c.page.d;
      page[0] = (uint32_t)__ldg(table + i);
      if (in_two) {                              // its second half may lie past the end
        const int pos1 = pos + 16, j = a.c.page.div(pos1);
        slots[1] = pos1 - j * a.c.page.d;
        page[1] = (uint32_t)__ldg(table + (pos1 < c.start + c.rows ? j : i));
      }
      return;
    }
    const int32_t* row = a.b.pages + (int64_t)c.b * a.b.pages_stride;
    const int pos = c.t * kBlock + (even ? 0 : lane), last = c.start + c.rows - 1;
    page[0] = (uint32_t)__ldg(row + a.c.page.div(min(pos, last)));
    if (even) page[1] = (uint32_t)__ldg(row + a.c.page.div(min(pos + 16, last)));
  };
  look();
  // this lane's place in a copy: its row of the rows at once, and its chunk
  const int copy_row = lane / L::kChunks, copy_chunk = lane % L::kChunks;
  const bool chunk_in = copy_chunk * 32 < a.D;
  int stage_in = 0;
  uint2 k_scale = make_uint2(0u, 0u), v_scale = make_uint2(0u, 0u);   // of key `lane` in the block in flight
  auto issue = [&]() {
    if (RUNS) {
      if (c.more) {
        constexpr int kCodes = kBlock * L::kBytes, kHalfRun = kCodes / 2;
        if (c.head != at_head) {
          at_head = c.head;
          k_head = a.c.x[0].of_head(at_head) + lane * 16;
          v_head = a.c.x[1].of_head(at_head) + lane * 16;
          s_head = scale_rows.of_head(at_head) + lane % kScaleLanes * 16;
        }
        worst = max(worst, page[0]);             // a bad page is reported at the end
        const uint32_t pg = min(page[0], top_page);
        uint8_t* dst = ring + stage_in * L::kStage + lane * 16;
        const uint8_t* k = k_head + a.c.x[0].offset(pg, 0) + slots[0] * L::kBytes;
        const uint8_t* v = v_head + a.c.x[1].offset(pg, 0) + slots[0] * L::kBytes;
        if (!in_two) {
#pragma unroll
          for (int i = 0; i < kCodes; i += 512) ptx::cp_async16(dst + i, k + i);
#pragma unroll
          for (int i = 0; i < kCodes; i += 512) ptx::cp_async16(dst + kCodes + i, v + i);
          if (lane < 2 * kScaleLanes)
            ptx::cp_async16(dst + L::kScales, s_head + scale_rows.offset(pg, 0) + slots[0] * L::kScaleBytes);
        } else {
          worst = max(worst, page[1]);
          const uint32_t pg1 = min(page[1], top_page);
          const uint8_t* k1 = k_head + a.c.x[0].offset(pg1, 0) + slots[1] * L::kBytes - kHalfRun;
          const uint8_t* v1 = v_head + a.c.x[1].offset(pg1, 0) + slots[1] * L::kBytes - kHalfRun;
#pragma unroll
          for (int i = 0; i < kCodes; i += 512) {
            ptx::cp_async16(dst + i, (i < kHalfRun ? k : k1) + i);
            ptx::cp_async16(dst + kCodes + i, (i < kHalfRun ? v : v1) + i);
          }
          const bool first = lane % kScaleLanes < kScaleLanes / 2;
          if (lane < 2 * kScaleLanes)
            ptx::cp_async16(dst + L::kScales,
                            s_head + scale_rows.offset(first ? pg : pg1, 0) +
                                (first ? slots[0] : slots[1] - 16) * L::kScaleBytes);
        }
        c.next(a, warp, GROUP);
        look();
      }
      ptx::cp_async_commit();
      stage_in ^= 1;
      return;
    }
    if (c.more) {
      const int pos0 = c.t * kBlock, last = c.start + c.rows - 1, head = c.head;
      worst = max(worst, max(page[0], page[1])); // a bad page is reported at the end
      const uint32_t pg0 = min(page[0], top_page), pg1 = min(page[1], top_page);
      // slots of the halves' first keys, or of key `lane`
      const int pos = even ? pos0 : min(pos0 + lane, last);
      const int slot0 = pos - a.c.page.div(pos) * a.c.page.d;
      const int slot1 = pos + 16 - a.c.page.div(pos + 16) * a.c.page.d;
      const bool upper = lane >= 16 && even;
      const uint32_t my_page = upper ? pg1 : pg0;
      const int my_slot = !even ? slot0 : upper ? slot1 + lane - 16 : slot0 + lane;
      k_scale = load_scales(a.c.scale[0].at(my_page, my_slot, head), a.D);
      v_scale = load_scales(a.c.scale[1].at(my_page, my_slot, head), a.D);
      c.next(a, warp, GROUP);
      look();
      uint8_t* dst = ring + stage_in * L::kStage;
      const Rows &kr = a.c.x[0], &vr = a.c.x[1];
      const uint8_t* k = kr.of_head(head) + copy_chunk * 16;
      const uint8_t* v = vr.of_head(head) + copy_chunk * 16;
#pragma unroll
      for (int i = 0; i < L::kCopies; ++i) {
        const int key = i * L::kRowsAtOnce + copy_row;
        uint32_t p;
        int s;
        if (even) {
          const bool second = i * L::kRowsAtOnce >= 16;
          p = second ? pg1 : pg0;
          s = (second ? slot1 : slot0) + key % 16;
        } else {
          p = __shfl_sync(0xffffffffu, my_page, key);
          s = __shfl_sync(0xffffffffu, my_slot, key);
        }
        ptx::cp_async16_or_zero(dst + i * 512 + lane * 16, k + kr.offset(p, s), chunk_in);
        ptx::cp_async16_or_zero(dst + L::kVPart + i * 512 + lane * 16, v + vr.offset(p, s), chunk_in);
      }
    }
    ptx::cp_async_commit();
    stage_in ^= 1;
  };

  // ---- Q of a segment, warp nt of the worker the rows 8 nt ..: lane (g, q) the q-th quarter of row g
  const Score sc = Score::of(a);
  constexpr int kQChunks = DP / 32;              // 16-byte chunks of a row of Q a lane
  uint4 qx[kQChunks];
  auto load_q = [&](const Segment& s) {
    const int rows = Item::group_rows(a, s), row = 8 * warp + g;
    const int grow = s.group * L::kRows + (row < rows ? row : 0), nd = a.group.div(grow);
    const uint4* src = reinterpret_cast<const uint4*>(
        a.q + (int64_t)(s.row0 + nd) * a.q_row + (int64_t)(s.head * a.G + grow - nd * a.G) * a.q_head);
#pragma unroll
    for (int j = 0; j < kQChunks; ++j) {
      qx[j] = make_uint4(0, 0, 0, 0);
      if (row < rows && (q * kQChunks + j) * 8 < a.D) qx[j] = __ldg(src + q * kQChunks + j);
    }
  };
  auto store_q = [&]() {
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
    float row_mul = CAP ? 1.f : sc.sl2, r = 1.f;
    if (!a.f16) {
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
    if (q == 0) reinterpret_cast<float*>(st.row_mul)[8 * warp + g] = row_mul;
#pragma unroll
    for (int j = 0; j < kQChunks; ++j) {
      uint32_t w[4] = {qx[j].x ^ flip, qx[j].y ^ flip, qx[j].z ^ flip, qx[j].w ^ flip};
      if (!a.f16) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = pack2<true>(to_float<false>((uint16_t)w[k]) * r,
                             to_float<false>((uint16_t)(w[k] >> 16)) * r);
      }
      q_mem[(warp * kQChunks + j) * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  };
  typename Item::Walker& walker = walkers[worker];
  if (tid == 0) {
    walker.init(a, share);
    st.live[0] = walker.next(a, &segments[0]);
  }
  issue();
  meet<GROUP>(worker);
  if (st.live[0] && warp < NT) {
    load_q(segments[0]);
    store_q();
  }
  meet<GROUP>(worker);

  // ---- the products' side
  int stage = 0, cur = 0;
  while (st.live[cur]) {
    const Segment& s = segments[cur];
    const int rows = Item::group_rows(a, s), t1 = s.t1, start = s.start;
    // O^T: tile t of row tile nt has columns (DP / 8) g + 2 t, + 1 of rows 8 nt + 2q, + 1
    float o[NT][kTiles][4], mref[NT][2], l[NT][2];
    // kept in registers where there are some left, else worked out each time: a row's
    // factor, what an exponent has to pass to move m, and m, or 0 before the first visible key
    constexpr int kKept = NT <= 2 ? NT : 1;
    float kept_mul[kKept][2], kept_limit[kKept][2], kept_sub[kKept][2];
    auto row_mul = [&](int nt, int e) {
      if (NT <= 2) return kept_mul[nt % kKept][e];
      const float2 y = st.row_mul[4 * nt + q];
      return e ? y.y : y.x;
    };
    auto limit = [&](int nt, int e) {
      return NT <= 2 ? kept_limit[nt % kKept][e]
                     : mref[nt][e] == -INFINITY ? -INFINITY : mref[nt][e] + (kShift + 8.f);
    };
    auto sub = [&](int nt, int e) {
      return NT <= 2 ? kept_sub[nt % kKept][e] : mref[nt][e] == -INFINITY ? 0.f : mref[nt][e];
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mref[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
        if (NT <= 2) {
          kept_limit[nt % kKept][e] = -INFINITY;
          kept_sub[nt % kKept][e] = 0.f;
          kept_mul[nt % kKept][e] = e ? st.row_mul[4 * nt + q].y : st.row_mul[4 * nt + q].x;
        }
      }
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nt][t][k] = 0.f;
    }
    // the segment after this one, meanwhile
    if (tid == kWorkerThreads - 1) st.live[cur ^ 1] = walker.next(a, &segments[cur ^ 1]);
#pragma unroll 1
    for (int t = s.t0 + warp; t < t1; t += GROUP) {
      const int pos0 = t * kBlock;
      const bool masked = pos0 + kBlock > start;
      const uint8_t* src = ring + stage * L::kStage;
      __syncwarp();                              // the block before has been read
      if (RUNS) {
        issue();
        ptx::cp_async_wait_group<1>();
        __syncwarp();
        const uint8_t* raw = src + L::kScales + lane * L::kScaleBytes;
        if (DP == 128) {
          k_scale = *reinterpret_cast<const uint2*>(raw);
          v_scale = *reinterpret_cast<const uint2*>(raw + kBlock * L::kScaleBytes);
        } else {
          k_scale.x = *reinterpret_cast<const uint32_t*>(raw);
          v_scale.x = *reinterpret_cast<const uint32_t*>(raw + kBlock * L::kScaleBytes);
        }
      }
      // the block's scales as f16, by lane = key
      {
        uint2 vs = v_scale;
        if (masked) {
          const int j = pos0 + lane - start;     // place in the draft
          if (j >= s.rows) {                     // past the end: anything may stand there
            vs = make_uint2(0u, 0u);
          } else if (j >= 0) {
            const bool x = zero_nonnumbers(&vs.x), y = zero_nonnumbers(&vs.y);
            if (x || y) atomicOr(&st.bad[j >> 5], 1u << (j & 31));
          }
        }
        uint4* to = reinterpret_cast<uint4*>(ring + L::kScale);
        to[lane] = spread_scales<DP>(k_scale);
        to[32 + lane] = spread_scales<DP>(vs);
      }
      if (!RUNS) {
        issue();
        ptx::cp_async_wait_group<1>();
      }
      __syncwarp();
      // S^T: keys row_key(g), + 8, .. of rows 8 nt + 2q, + 1
      uint32_t ks[4];
      ptx::ldmatrix_x4(scale_mem, ks[0], ks[1], ks[2], ks[3]);
      float x[NT][kParts][2];
      // with eight rows both tiles of 16 keys side by side, for the products of one follow
      // each other; with more there are others to go between
      constexpr int kSide = NT == 1 ? 2 : 1;
#pragma unroll
      for (int m0 = 0; m0 < kParts / 2; m0 += kSide) {
        uint32_t kw[2 * kSide][L::kWords];
#pragma unroll
        for (int h = 0; h < 2 * kSide; ++h) {
          const uint8_t* row = src + ((2 * m0 + h) * 8 + gk) * L::kBytes + q * (L::kBytes / 4);
          if (DP == 128) {
            const uint4 y = *reinterpret_cast<const uint4*>(row);
            kw[h][0] = y.x, kw[h][1] = y.y, kw[h][2 % L::kWords] = y.z, kw[h][3 % L::kWords] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(row);
            kw[h][0] = y.x, kw[h][1] = y.y;
          }
        }
        float acc[kSide][NT][4];
#pragma unroll
        for (int mt = 0; mt < kSide; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[mt][nt][k] = 0.f;
#pragma unroll
        for (int i = 0; i < L::kWords; ++i) {    // a word: two steps
          uint4 b[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) b[nt] = q_mem[(nt * kQChunks + i) * 32 + lane];
#pragma unroll
          for (int mt = 0; mt < kSide; ++mt) {
            // 128 elements: the lane's first two words are under one scale, the others under the next
            const uint32_t sel = i < 2 ? 0x1010 : 0x3232;
            const uint32_t s0 = __byte_perm(ks[2 * (m0 + mt)], 0, sel);
            const uint32_t s1 = __byte_perm(ks[2 * (m0 + mt) + 1], 0, sel);
            uint4 ka = e2m1x8_to_f16(kw[2 * mt][i]), kb = e2m1x8_to_f16(kw[2 * mt + 1][i]);
            ka = make_uint4(mul_f16x2(ka.x, s0), mul_f16x2(ka.y, s0), mul_f16x2(ka.z, s0), mul_f16x2(ka.w, s0));
            kb = make_uint4(mul_f16x2(kb.x, s1), mul_f16x2(kb.y, s1), mul_f16x2(kb.z, s1), mul_f16x2(kb.w, s1));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) ptx::mma_16816_f16(acc[mt][nt], ka.x, kb.x, ka.y, kb.y, b[nt].x, b[nt].y);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) ptx::mma_16816_f16(acc[mt][nt], ka.z, kb.z, ka.w, kb.w, b[nt].z, b[nt].w);
          }
        }
#pragma unroll
        for (int mt = 0; mt < kSide; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) x[nt][2 * (m0 + mt) + k / 2][k % 2] = acc[mt][nt][k];
      }
      // invisible scores -infinity; see: bit 8 i, the row sees key 8 i + row_key(g)
      uint32_t see[NT][2], of_row = ~0u;         // of row `lane`, all 32 keys
      if (masked) {
        const int row = lane % L::kRows, nd = a.group.div(s.group * L::kRows + (row < rows ? row : 0));
        of_row = sees_32(a.mask ? a.mask + (int64_t)(s.row0 + nd) * a.mask_stride : nullptr, s.rows, nd,
                         pos0 - start);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          see[nt][e] = 0x01010101u;
          if (masked) {
            see[nt][e] = __shfl_sync(0xffffffffu, of_row, 8 * nt + 2 * q + e) >> gk & 0x01010101u;
#pragma unroll
            for (int i = 0; i < kParts; ++i)
              if (!(see[nt][e] >> (8 * i) & 1)) x[nt][i][e] = -INFINITY;
          }
        }
      float mx[NT][2];
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = fmaxf(fmaxf(x[nt][0][e], x[nt][1][e]), fmaxf(x[nt][2][e], x[nt][3][e]));
          y = y == -INFINITY ? -INFINITY : y * row_mul(nt, e);
          // a visible score of -infinity is the cap's negative, an invisible one nothing
          if (CAP && see[nt][e] != 0) y = capped(sc, y, 0.f);
          mx[nt][e] = y;
          over |= y > limit(nt, e);
        }
      // the first visible key sets a row's m, later ones when the maximum has grown enough
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = mx[nt][e];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, off));
            const float old = mref[nt][e];
            if (y > limit(nt, e)) {
              mref[nt][e] = y - kShift;
              if (NT <= 2) {
                kept_sub[nt % kKept][e] = mref[nt][e];
                kept_limit[nt % kKept][e] = y + 8.f;
              }
              if (t >= s.t0 + GROUP) {           // not the warp's first block: O and l are zeros there
                const float back = old == -INFINITY ? 0.f : ex2(old - mref[nt][e]);
                l[nt][e] *= back;
#pragma unroll
                for (int t8 = 0; t8 < kTiles; ++t8) {
                  o[nt][t8][e] *= back;
                  o[nt][t8][2 + e] *= back;
                }
              }
            }
          }
      }
      // weights, as the B operand of the second product
      uint32_t p[NT][kParts];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[kParts][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (!CAP) {
#pragma unroll
            for (int i = 0; i < kParts; ++i) w[i][e] = fmaf(x[nt][i][e], row_mul(nt, e), -sub(nt, e));
          } else {
            float raw[kParts], big = 0.f;
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
              raw[i] = x[nt][i][e] * row_mul(nt, e);
              big = fmaxf(big, fabsf(raw[i]));
              w[i][e] = capped_near(sc, raw[i], sub(nt, e));
            }
            if (__any_sync(0xffffffffu, past_near(sc, big))) {
#pragma unroll
              for (int i = 0; i < kParts; ++i) {
                const float past = capped_past(sc, raw[i], sub(nt, e));
                if (past_near(sc, raw[i])) w[i][e] = past;
              }
            }
          }
#pragma unroll
          for (int i = 0; i < kParts; ++i) w[i][e] = ex2(w[i][e]);
          // by the bits: an invisible key's exponent can be anything (-infinity times a
          // scale of zero)
          if (masked) {
#pragma unroll
            for (int i = 0; i < kParts; ++i)
              if (!(see[nt][e] >> (8 * i) & 1)) w[i][e] = 0.f;
          }
          l[nt][e] += (w[0][e] + w[1][e]) + (w[2][e] + w[3][e]);
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i) p[nt][i] = transpose8x8(pack2<true>(w[i][0], w[i][1]));
      }
      // O^T += V^T P^T, 16 keys at a time
      uint32_t vs[4];
      ldmatrix_x4_trans(scale_mem + kBlock * 16, vs);
#pragma unroll
      for (int mt = 0; mt < kParts / 2; ++mt) {
        // the lane's codes of the keys of rows 16 mt + 2q, + 1, + 8, + 9
        constexpr int kV = DP / 64;              // words a key
        uint32_t vw[4][kV];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = 16 * mt + 8 * (k >> 1) + (2 * q + ((k ^ q) & 1));      // row_key(2 q + k % 2)
          const uint8_t* row = src + L::kVPart + key * L::kBytes + g * (4 * kV);
          if (DP == 128) {
            const uint2 y = *reinterpret_cast<const uint2*>(row);
            vw[k][0] = y.x, vw[k][kV - 1] = y.y;
          } else {
            vw[k][0] = *reinterpret_cast<const uint32_t*>(row);
          }
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          // even elements of the pairs of keys, and odd ones: a byte a column
          uint4 even2[2], odd2[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t wa = vw[2 * h][i], wb = vw[2 * h + 1][i], sv = vs[2 * mt + h];
            uint4 y = e2m1x8_to_f16((wa & 0x0f0f0f0fu) | (wb << 4 & 0xf0f0f0f0u));
            even2[h] = make_uint4(mul_f16x2(y.x, sv), mul_f16x2(y.y, sv), mul_f16x2(y.z, sv), mul_f16x2(y.w, sv));
            y = e2m1x8_to_f16((wa >> 4 & 0x0f0f0f0fu) | (wb & 0xf0f0f0f0u));
            odd2[h] = make_uint4(mul_f16x2(y.x, sv), mul_f16x2(y.y, sv), mul_f16x2(y.z, sv), mul_f16x2(y.w, sv));
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t b0 = p[nt][2 * mt], b1 = p[nt][2 * mt + 1];
            ptx::mma_16816_f16(o[nt][4 * i], even2[0].x, odd2[0].x, even2[1].x, odd2[1].x, b0, b1);
            ptx::mma_16816_f16(o[nt][4 * i + 1], even2[0].y, odd2[0].y, even2[1].y, odd2[1].y, b0, b1);
            ptx::mma_16816_f16(o[nt][4 * i + 2], even2[0].z, odd2[0].z, even2[1].z, odd2[1].z, b0, b1);
            ptx::mma_16816_f16(o[nt][4 * i + 3], even2[0].w, odd2[0].w, even2[1].w, odd2[1].w, b0, b1);
          }
        }
      }
      stage ^= 1;
    }

    // the warps meet: O, m and l of the segment
    const bool whole = s.whole();
    const int64_t part = 2 * (blockIdx.x * L::kWorkers + worker) + (s.t0 == 0 ? 1 : 0);
    const int live = min(GROUP, s.t1 - s.t0);  // warps that had a block
    float* merge = reinterpret_cast<float*>(smem + L::kMerge + worker * GROUP * L::kMergeWarp);
    auto out_row = [&](int row) {
      const int grow = s.group * L::kRows + row, nd = a.group.div(grow);
      return (int64_t)(s.row0 + nd) * a.Hq + s.head * a.G + grow - nd * a.G;
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nt][e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (g == 0) st.ml[warp][8 * nt + 2 * q + e] = make_float2(mref[nt][e], sum);
      }
    // every warp's O, some columns at a time, and by which weight is for those to see who add
    // them up
    constexpr int kT = kTiles / L::kPasses, kCols = L::kCols;
    bool next_live = false;
    uint32_t any_bad = 0;
#pragma unroll
    for (int pass = 0; pass < L::kPasses; ++pass) {
      if (warp < live) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* dst = merge + (warp * L::kRows + 8 * nt + 2 * q + e) * L::kMergeRow + g * (2 * kT);
#pragma unroll
            for (int k = 0; k < kT; k += 2) {
              const float* y = o[nt][pass * kT + k];
              const float* z = o[nt][pass * kT + k + 1];
              *reinterpret_cast<float4*>(dst + 2 * k) = make_float4(y[e], y[2 + e], z[e], z[2 + e]);
            }
          }
      }
      meet<GROUP>(worker);
      if (pass == 0) {
        next_live = st.live[cur ^ 1];
        if (next_live && warp < NT) load_q(segments[cur ^ 1]);
#pragma unroll
        for (int k = 0; k < DSPARK_TREE_MAX_NODES / 32; ++k) any_bad |= st.bad[k];
      }
      for (int i = tid; i < rows * (kCols / 4); i += kWorkerThreads) {
        const int row = i / (kCols / 4), n = i % (kCols / 4) * 4;
        float top = -INFINITY, sum = 0.f;
#pragma unroll 4
        for (int k = 0; k < live; ++k) top = fmaxf(top, st.ml[k][row].x);
        const float base = top == -INFINITY ? 0.f : top;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < live; ++k) {
          const float2 ml = st.ml[k][row];
          const float4 v = *reinterpret_cast<const float4*>(merge + (k * L::kRows + row) * L::kMergeRow + n);
          const float w = ex2(ml.x - base);
          sum = fmaf(ml.y, w, sum);
          y.x = fmaf(v.x, w, y.x);
          y.y = fmaf(v.y, w, y.y);
          y.z = fmaf(v.z, w, y.z);
          y.w = fmaf(v.w, w, y.w);
        }
        const int d = n / (2 * kT) * (DP / 8) + pass * (2 * kT) + n % (2 * kT);
        if (!whole) {
          *reinterpret_cast<float4*>(a.part_o + (part * L::kRows + row) * DP + d) = y;
          if (pass == 0 && n == 0) a.part_ml[part * L::kRows + row] = make_float2(top, sum);
        } else {
          // l = 0: every weight was 0, and so is O
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          const int64_t to = out_row(row);
          if (d < a.D)
            *reinterpret_cast<uint2*>(a.out + to * a.D + d) =
                make_uint2(pack_out(a.f16, y.x * inv, y.y * inv), pack_out(a.f16, y.z * inv, y.w * inv));
          if (pass == 0 && n == 0 && a.lse) a.lse[to] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
        }
      }
      if (pass + 1 < L::kPasses) meet<GROUP>(worker);
    }
    if (next_live && warp < NT) store_q();       // all are past the segment's products
    if (any_bad != 0) {
      meet<GROUP>(worker);
      if ((int)tid < rows) {
        const int nd = a.group.div(s.group * L::kRows + tid);
        add_nan(a, st.bad, a.mask ? a.mask + (int64_t)(s.row0 + nd) * a.mask_stride : nullptr, s.b, s.rows,
                s.start, s.head, nd, whole ? a.out + out_row(tid) * a.D : nullptr,
                a.part_o + (part * L::kRows + tid) * DP);
      }
      meet<GROUP>(worker);
      if (tid < DSPARK_TREE_MAX_NODES / 32) st.bad[tid] = 0;
    }
    if (!whole && tid == 0)
      st.left[s.t0 == 0 ? 1 : 0] = {Item::part_of(s, share.cut).w, s.row0, s.head, s.group, rows};
    meet<GROUP>(worker);
    cur ^= 1;
  }
  // items whose parts are all there now are joined by this worker, at its end: in between,
  // what makes a part seen by others would have held up all of its warps (20 requests of
  // 1,000 tokens: 22.9 us, with no item shared 12.2)
  if (st.left[0].item | st.left[1].item) {
    __threadfence();
    meet<GROUP>(worker);
    if (tid < 2) {
      const int item = st.left[tid].item;
      bool last = false;
      if (item != 0) {
        int* count = a.arrived + (item & 0xffff);
        last = atomicAdd(count, 1) == (item >> 16) - 1;
        if (last) *count = 0;
        __threadfence();
      }
      st.join[tid] = last;
    }
    meet<GROUP>(worker);
#pragma unroll 1
    for (int k = 0; k < 2; ++k)
      if (st.join[k]) join_parts<L, GROUP>(a, st.left[k], tid);
  }
  ptx::cp_async_wait_group<0>();
  if (worst > top_page) set_status(a.status, DSPARK_EPAGES);
}

template <int DP, int NT, int GROUP, bool RUNS, bool CAP>
cudaError_t launch(AttendArgs a, uint32_t* ready, cudaStream_t stream) {
  using L = Few4<DP, NT, GROUP, RUNS>;
  static_assert(L::kSmem + L::kWorkers * (sizeof(WorkerState<GROUP, L::kRows>) + 300) + 1024 <= 232448,
                "shared memory of an SM");
  static_assert(L::kWorkers <= kFew4Workers && 2 * L::kWorkers * L::kRows <= kFew4PartRows, "the parts' place");
  constexpr uint32_t kBit = 1u << (NT / 2 * 5 + (GROUP == 4 ? 4 : 2 * RUNS + CAP));
  static_assert(kBit < kReadyMany, "a bit of its own");
  if (!(*ready & kBit)) {
    const cudaError_t e = cudaFuncSetAttribute(few4_kernel<DP, NT, GROUP, RUNS, CAP>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    if (e != cudaSuccess) return e;
    *ready |= kBit;
  }
  // launched while the kernel before it in the stream ends, which it waits for before
  // anything else
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
  a.n_cta *= L::kWorkers;
  return cudaLaunchKernelEx(&cfg, few4_kernel<DP, NT, GROUP, RUNS, CAP>, a);
}

// alone: a worker a CTA; else of four warps, where slots lie in runs and scores are not
// capped (those, and slots that are no runs, go with a worker a CTA: 128 tokens as above 147 us,
// capped 223, a slot's heads next to each other 280).
template <int DP, int NT, int WARPS>
cudaError_t launch_all(const AttendArgs& a, bool alone, bool runs, uint32_t* ready, cudaStream_t stream) {
  const bool cap = a.softcap > 0.f;
  if (!runs)
    return cap ? launch<DP, NT, WARPS, false, true>(a, ready, stream)
               : launch<DP, NT, WARPS, false, false>(a, ready, stream);
  if (cap) return launch<DP, NT, WARPS, true, true>(a, ready, stream);
  return alone ? launch<DP, NT, WARPS, true, false>(a, ready, stream)
               : launch<DP, NT, 4, true, false>(a, ready, stream);
}

}  // namespace

// A source file each.
template <int DP, int NT>
cudaError_t few4_launch_of(const AttendArgs& a, bool alone, bool runs, uint32_t* ready, cudaStream_t stream);

}  // namespace tree
}  // namespace dspark
