// tree_attend.cuh -- attention of drafted rows over a paged cache on tcgen05, for
// more rows a cached head than tree_attend_few.cu and tree_attend_few4.cu take.  Items are 256 rows by
// tiles of 128 keys, a worker is a CTA, one a SM (tree_items.cuh says how the
// work is cut, and the mathematics).
//
// Warps: 8 of softmax in two groups of 128 threads (thread = row = tensor-memory
// lane), then the producers (4 for a 16-bit cache, 8 for e4m3), then a group of 4
// of which two issue products, one a stream, and a third works out where the
// parts lie.  Two streams share the ring of key and value tiles: with more than
// 128 rows (a pair) each stream owns a row tile and both read every key tile;
// with fewer, the streams take alternate key tiles of the one row tile and are
// joined at the end.  Per stream: S = Q K^T (both operands in shared memory) into
// tensor memory, softmax there, P written over S, O += P V with P read from
// tensor memory.
//
// S and P share columns and tensor memory is full, so the next S cannot be made
// before P has been used.  A pair therefore goes by halves of 64 keys: one half's
// S is made while the softmax is at the other (64 requests of 64 nodes, 4,096 to
// 8,192 tokens: 402 us at the time, 426 with whole tiles).  Alternate tiles stay whole: with
// few rows the copies bound, and halves hold their slots longer (64 us against 75
// for 16 requests of 8 nodes).
//
// Tensor memory (512 columns): S/P of the streams at 0 and 128, O at 256 and
// 384.  Shared memory: two Q tiles (the result leaves through their place, a row
// at a time) and the ring, rows of 64 elements (128 bytes) swizzled in atoms of 8
// rows; K is read K-major, V (same layout) N-major.  A 16-bit cache comes by
// tiled copies where pages allow (make_maps), else by 16-byte copies of any
// strides and page size; e4m3 through registers, the scale multiplied in (exact
// in bf16), so everything after the ring is the same; e2m1 too, whose values are exact in
// both types.
//
// Keys past the end are zero rows and masked; draft rows of V that are not
// finite would reach every row of the product (0 * NaN), so such elements are
// zeroed in the ring and noted, and added at the end to the rows that see them.
//
// What bounds it.  64 x 64 as above (414 GFLOP, 1.7 GB): 407 to 422 us, 1.0 PFLOP/s, the
// tensor pipe active 50% of the time and the issue slots 50%: the rest is the
// chain softmax - product - next S of two streams, and 15 us an item for Q, the
// masked tiles and the result.  17 nodes over 131,000 tokens: 99 us, 5.4 TB/s.
// 16 requests of 8 nodes: 60 us, 2.9 TB/s, the ring's five slots against the
// copies' latency (long scoreboard 7.2 of 15 warp cycles an issue).  64 x 64 over e2m1: 462
// us (at 495: without the producers' loads 427, without their conversions too 390).
#pragma once

#include "tree_items.cuh"

namespace dspark {
namespace tree {
namespace {

constexpr int kKeys = 128;              // keys of a tile
constexpr int kHalf = 64;               // of them in one step of the softmax
constexpr int kSoftWarps = 8;

// Warps and registers.  The softmax groups take registers from the others: for
// a 16-bit cache enough to hold a row of scores; for codes the producers need
// theirs to convert in, and the softmax reads its scores in two halves.
template <int HELD>
struct Roles {
  static constexpr bool kCodes = HELD != k16;
  static constexpr int kProdWarps = kCodes ? 8 : 4;
  static constexpr int kMmaWarp = kSoftWarps + kProdWarps;
  static constexpr int kThreads = (kMmaWarp + 4) * 32;
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
  static constexpr int kSoftRegs = kCodes ? 120 : 184;
  // e2m1, 64 x 64: producers 88 and products 64 477 us, 96 and 48 519, while the latter
  // had registers to spill
  static constexpr int kProdRegs = HELD == kE4M3 ? 96 : 88;
  static constexpr int kMmaRegs = HELD == kE4M3 ? 48 : HELD == kE2M1 ? 64 : 56;
  static constexpr int kSplit =
      kSoftWarps * kSoftRegs + kProdWarps * kProdRegs + 4 * kMmaRegs;   // times 32
  static_assert(kSplit * 32 <= kThreads * kLaunchRegs, "the split asks for more than there is");
};

constexpr int kLag = 2;                 // slots a producer issues ahead of the one it completes
constexpr int kBadSets = 8;             // segments the producers can be ahead, rounded up
constexpr uint64_t kWaitLimitNs = 1000000000ull;
// An item's Q, result and way into the loop take as long as about three tiles (16
// requests of 8 nodes: 1 65 us, 3 63, 6 68; 13 trees over e4m3: 49.7, 49.6, 55.6).
using Item = Work<kKeys, kGroupRows, 3>;
using Segment = Item::Segment;
using Walker = Item::Walker;
using Cursor = Item::Cursor;

template <int DP>
struct Layout {
  static constexpr int kTile = kKeys * DP * 2;                  // bytes of a Q, K or V tile
  static constexpr int kSlots = DP == 128 ? 5 : 8;
  static constexpr int kRing = 2 * kTile;
  static constexpr int kTail = kRing + kSlots * kTile;
};

// A place in the ring and the parity of its fills.
template <int SLOTS>
struct RingPos {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == SLOTS) {
      slot = 0;
      phase ^= 1;
    }
  }
};

struct Tail {
  uint64_t full[8], empty[8], q_full, q_empty;
  uint64_t s_full[2][2], p_full[2][2], o_done[2][2];      // [stream][half of the tile]
  float2 ml[2][kKeys];
  uint32_t bad[kBadSets][DSPARK_TREE_MAX_NODES / 32];
  Share share;
  int64_t warp_sum[20];
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ uint64_t globaltimer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// Every wait ends: past the limit the CTA's abort flag makes all its waits
// return at once, the loops run on without starting copies or products (all
// accesses stay in bounds), and the status says so.
//
// A parity wait tells a phase from the next one only.  So whoever waits on a
// barrier waits for each of its phases in order (or knows that the one before is
// over), and no phase can end before all lanes that wait for the one before it
// have seen that: what ends it depends on an arrival of theirs.
__device__ __forceinline__ void wait_long(Tail* s, uint64_t* bar, uint32_t parity, int* status) {
  const uint64_t t0 = globaltimer_ns();
  uint32_t spins = 0;
  while (!ptx::mbar_try_wait(bar, parity)) {
    if ((++spins & 63u) != 0u) continue;
    if (*(const volatile int*)&s->abort) return;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      *(volatile int*)&s->abort = 1;
      set_status(status, DSPARK_ETIMEOUT);
      return;
    }
  }
}

__device__ __forceinline__ void wait(Tail* s, uint64_t* bar, uint32_t parity, int* status) {
  if (!ptx::mbar_try_wait(bar, parity)) wait_long(s, bar, parity, status);
}

__device__ __forceinline__ bool aborted(const Tail* s) {
  return *(const volatile int*)&s->abort != 0;
}

// Visibility of the 128 positions from draft position j0 on (negative: context).
__device__ __noinline__ uint4 sees_128(const uint32_t* mask_row, int rows, int node, int j0) {
  const int w = j0 >> 5;                         // floor
  uint32_t x[5];
#pragma unroll
  for (int k = 0; k < 5; ++k) x[k] = w + k < 0 ? 0xffffffffu : sees_word(mask_row, rows, node, w + k);
  return make_uint4(__funnelshift_r(x[0], x[1], j0 & 31), __funnelshift_r(x[1], x[2], j0 & 31),
                    __funnelshift_r(x[2], x[3], j0 & 31), __funnelshift_r(x[3], x[4], j0 & 31));
}

using ptx::add_f32x2;
using ptx::fma_f32x2;
using ptx::mul_f32x2;
using ptx::pack_f32x2;
using ptx::sub_f32x2;
using ptx::unpack_f32x2;

// ------------------------------------------------------------- producers --

// Byte offset of (row, 16-byte chunk) in a tile: 64-element blocks of 128 rows.
__device__ __forceinline__ uint32_t tile_offset(int row, int chunk) {
  return (uint32_t)(chunk >> 3) * (kKeys * 128) + (uint32_t)row * 128 +
         (uint32_t)((chunk ^ row) & 7) * 16;
}

// 16-bit cache.  With a map (see make_maps for when), tiles of context go by
// tiled copies, lane 0 of every warp issuing its share of the boxes; tiles that
// reach into the draft (the last of a request), and all tiles without a map, by
// 16-byte copies, completed two slots later, so that rows past the end are zero
// and draft rows of V can be looked through.  A warp copies 32 rows of the
// tile; each lane looks one row's page up, a tile ahead, and hands it round.
template <bool F16, int DP>
__device__ __forceinline__ void produce16(const AttendArgs& a, const TileMaps& maps, uint8_t* smem,
                                          Tail* sh) {
  using L = Layout<DP>;
  constexpr int kWarps = Roles<k16>::kProdWarps;
  constexpr int kChunks = DP / 8;                // 16-byte chunks of a row
  constexpr int kSub = 32 / kChunks;             // rows of one copy instruction
  static_assert(kWarps * 32 == kKeys, "32 rows a warp");
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32 - kSoftWarps;
  const int chunk = lane % kChunks, sub = lane / kChunks;
  const bool in_dim = chunk * 8 < a.D;
  const int pieces = maps.rows > 0 ? kKeys / maps.rows : 0;      // boxes along a tile's keys
  const int boxes = pieces * (DP / 64);          // of a tile; warp w issues w, w + 4, ...
  uint8_t* ring = smem + L::kRing;
  Cursor c;
  c.init(a, sh->share);
  if (!c.more()) return;
  // the page of this lane's row (tiled: of the warp's box) of the tile at the cursor
  int page_next = 0;
  auto fetch_page = [&]() {
    if (!c.more()) return;
    const bool tiled = maps.rows > 0 && (c.t + 1) * kKeys <= c.start;
    const int row = tiled ? warp % pieces * maps.rows : warp * 32 + lane;
    const int pos = min(c.t * kKeys + row, c.total() - 1);
    page_next = __ldg(a.b.pages + (int64_t)c.b * a.b.pages_stride + a.c.page.div(pos));
  };
  fetch_page();
  RingPos<L::kSlots> at;
  uint32_t copied = 0;                           // bit i: the slot i + 1 before went by 16-byte copies
  // the V tile in flight: where it is and which of its positions are draft
  int prev_pos = 0, prev_start = 0, prev_total = 0, prev_seg = 0;
  auto complete = [&](int back, bool v) {        // this thread's copies `back` slots ago have landed
    const uint32_t slot = at.slot >= (uint32_t)back ? at.slot - back : at.slot + L::kSlots - back;
    if (v && prev_pos + kKeys > prev_start) {
#pragma unroll 1
      for (int i = sub; i < 32; i += kSub) {
        const int row = warp * 32 + i, pos = prev_pos + row;
        if (pos < prev_start || pos >= prev_total) continue;
        uint4* p = reinterpret_cast<uint4*>(ring + slot * L::kTile + tile_offset(row, chunk));
        uint4 x = *p;
        if (zero_nonfinite<F16>(&x)) {
          *p = x;
          const int j = pos - prev_start;
          atomicOr(&sh->bad[prev_seg % kBadSets][j >> 5], 1u << (j & 31));
        }
      }
      __syncwarp();
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&sh->full[slot]);
  };
  while (c.more()) {
    const int head = c.head, start = c.start, total = c.total(), seg = c.seg;
    const int pos0 = c.t * kKeys;
    const bool tiled = maps.rows > 0 && pos0 + kKeys <= start;
    int page = page_next;
    if ((uint32_t)page >= (uint64_t)a.c.n_pages) {
      set_status(a.status, DSPARK_EPAGES);
      page = -1;
    }
    c.next(a);
    fetch_page();
    const int my_pos = pos0 + (tiled ? warp % pieces * maps.rows : warp * 32 + lane);
    const int my_slot = my_pos - a.c.page.div(my_pos) * a.c.page.d;
    if (my_pos >= total) page = -1;
#pragma unroll 1
    for (int v = 0; v < 2; ++v) {
      uint64_t* full = &sh->full[at.slot];
      uint8_t* dst = ring + at.slot * L::kTile;
      wait(sh, &sh->empty[at.slot], at.phase ^ 1, a.status);
      if (tiled) {
        __syncwarp();                            // every lane's wait is over
        if (lane == 0) {
          // after an abort no copy may outlive the CTA: none is started
          if (warp < boxes && !aborted(sh)) {
            ptx::mbar_expect_tx(full, maps.rows * 128);
            const int block = warp / pieces;
            ptx::tma_load_4d(dst + block * (kKeys * 128) + warp % pieces * maps.rows * 128,
                             v ? &maps.v : &maps.k, block * 64, my_slot, head,
                             page < 0 ? (int)a.c.n_pages : page, full);   // past the end: zeros
          } else {
            ptx::mbar_arrive(full);
          }
        }
        __syncwarp();
      } else {
        const Rows rows = a.c.x[v];
        const uint8_t* src = rows.of_head(head) + chunk * 16;
#pragma unroll
        for (int i = 0; i < 32; i += kSub) {
          const int p = __shfl_sync(0xffffffffu, page, i + sub);
          const int s = __shfl_sync(0xffffffffu, my_slot, i + sub);
          const bool on = in_dim && p >= 0;
          ptx::cp_async16_or_zero(dst + tile_offset(warp * 32 + i + sub, chunk),
                                  on ? src + rows.offset(p, s) : rows.p, on);
        }
      }
      ptx::cp_async_commit();
      if (copied >> (kLag - 1) & 1) {
        ptx::cp_async_wait_group<kLag>();
        complete(kLag, v);
      }
      copied = copied << 1 | (tiled ? 0u : 1u);
      at.next();
    }
    prev_pos = pos0;
    prev_start = start;
    prev_total = total;
    prev_seg = seg;
  }
  ptx::cp_async_wait_group<0>();
  if (copied & 1) {
    complete(2, false);
    complete(1, true);
  }
}

// A chunk of 16 codes whose scale is not easy, stored at p0 and p1.  Non-finite
// elements of a draft row of V are zeroed and noted (bad: its bit's word).
template <bool F16>
__device__ __noinline__ void store_any(uint4 x, uint32_t byte, uint8_t* p0, uint8_t* p1,
                                       uint32_t* bad, uint32_t bit) {
  const uint2 c0 = scale_codes_any<F16>(x.x, byte), c1 = scale_codes_any<F16>(x.y, byte);
  const uint2 c2 = scale_codes_any<F16>(x.z, byte), c3 = scale_codes_any<F16>(x.w, byte);
  uint4 y0 = make_uint4(c0.x, c0.y, c1.x, c1.y), y1 = make_uint4(c2.x, c2.y, c3.x, c3.y);
  if (bad) {
    const bool b0 = zero_nonfinite<F16>(&y0), b1 = zero_nonfinite<F16>(&y1);
    if (b0 || b1) atomicOr(bad, bit);
  }
  *reinterpret_cast<uint4*>(p0) = y0;
  *reinterpret_cast<uint4*>(p1) = y1;
}

// e4m3 cache, through registers.  A half tile (K or V) is converted while the
// next is in flight in registers; pages are looked up two half tiles earlier,
// and the rows kAhead tiles on are asked for in L2, one row of K or V a thread.
// The loop is one half tile: unrolled over register sets it outgrew the
// instruction cache.
template <bool F16, int DP>
__device__ __forceinline__ void produce8(const AttendArgs& a, uint8_t* smem, Tail* sh) {
  using L = Layout<DP>;
  constexpr int kWarps = Roles<kE4M3>::kProdWarps;
  constexpr int kChunks = DP / 16;               // 16-code chunks of a row
  constexpr int kWarpRows = 32 / kChunks;
  constexpr int kRows = kWarps * kWarpRows;      // rows a pass
  constexpr int kPasses = kKeys / kRows;
  constexpr int kAhead = 4;
  static_assert(kWarps * 32 == 2 * kKeys, "one row of K or V a thread");
  const int tid = threadIdx.x - kSoftWarps * 32, lane = tid % 32, warp = tid / 32;
  // eight lanes store to two neighbouring rows, four 32-byte chunks of one
  // 64-element block each: all banks once
  const int chunk = (lane & 3) | (DP == 128 ? (lane >> 1) & 4 : 0);
  const int r0 = warp * kWarpRows +
                 (DP == 128 ? ((lane >> 2) & 1) | ((lane >> 3) & 2) : lane >> 2);
  const bool in_dim = chunk * 16 < a.D;
  const uint32_t to0 = tile_offset(r0, 2 * chunk), to1 = tile_offset(r0, 2 * chunk + 1);
  uint8_t* ring = smem + L::kRing;
  Cursor c;                                      // the tile after the one in `page`
  c.init(a, sh->share);
  if (!c.more()) return;
  struct Tile {
    int head, rows, draft, seg;                  // rows that exist; the first of the draft
  };
  auto tile_at = [&]() {
    return Tile{c.head, min(kKeys, c.total() - c.t * kKeys), c.start - c.t * kKeys, c.seg};
  };
  uint32_t page[kPasses], worst = 0;
  int slot[kPasses];
  auto fetch_pages = [&]() {
    const int32_t* table = a.b.pages + (int64_t)c.b * a.b.pages_stride;
    const int last = c.total() - 1;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int pos = min(c.t * kKeys + r0 + i * kRows, last), at = a.c.page.div(pos);
      page[i] = (uint32_t)__ldg(table + at);
      slot[i] = pos - at * a.c.page.d;
    }
  };
  RingPos<L::kSlots> at;
  // rows of the same request kAhead tiles on, across a head's end
  auto ask = [&]() {
    int t = c.t + kAhead, head = c.head;
    if (t >= c.tiles) {
      t -= c.tiles;
      ++head;
    }
    if (head >= a.Hkv || t >= c.tiles) return;
    const int pos = min(t * kKeys + tid % kKeys, c.total() - 1), at = a.c.page.div(pos);
    const uint32_t p = (uint32_t)__ldg(a.b.pages + (int64_t)c.b * a.b.pages_stride + at);
    if (p >= (uint64_t)a.c.n_pages) return;
    ptx::prefetch_l2(a.c.x[tid >= kKeys].at(p, pos - at * a.c.page.d, head));
  };
  uint4 x[kPasses], x_next[kPasses];
  uint32_t byte[kPasses], byte_next[kPasses];
  const uint32_t top_page = (uint32_t)(a.c.n_pages - 1);
  auto load = [&](bool v, int head) {
    const Rows rows = a.c.x[v], scales = a.c.scale[v];
    const uint8_t* src = rows.of_head(head) + (in_dim ? chunk * 16 : 0);
    const uint8_t* sc = scales.of_head(head);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if (!v) {                                  // a bad page is reported at the end
        worst = max(worst, page[i]);
        page[i] = min(page[i], top_page);
      }
      x_next[i] = ptx::ldg_nc_na(src + rows.offset(page[i], slot[i]));
      byte_next[i] = __ldg(sc + scales.offset(page[i], slot[i]));
    }
  };
  fetch_pages();
  Tile cur = tile_at();
  load(false, cur.head);
  bool more = true;                              // another half tile after the one in x_next
#pragma unroll 1
  for (bool v = false; more; v = !v, at.next()) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      x[i] = x_next[i];
      byte[i] = byte_next[i];
    }
    const Tile tile = cur;
    if (!v) {
      load(true, cur.head);                      // V of the same tile, then the next tile's pages
      c.next(a);
      if (c.more()) {
        fetch_pages();
        ask();
      }
    } else {
      more = c.more();
      if (more) {
        cur = tile_at();
        load(false, cur.head);
      }
    }
    wait(sh, &sh->empty[at.slot], at.phase ^ 1, a.status);
    uint8_t* dst = ring + at.slot * L::kTile;
    if (tile.rows < kKeys || a.D < DP) {         // rows and elements past the end are zeros
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
        if (!in_dim || r0 + i * kRows >= tile.rows) {
          x[i] = make_uint4(0, 0, 0, 0);
          byte[i] = 127;
        }
    }
    bool easy = true;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) easy &= easy_scale<F16>(byte[i]);
    if (easy) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const uint32_t m = scale_mul2<F16>(byte[i]);
        const uint2 c0 = scale_codes<F16>(x[i].x, m), c1 = scale_codes<F16>(x[i].y, m);
        const uint2 c2 = scale_codes<F16>(x[i].z, m), c3 = scale_codes<F16>(x[i].w, m);
        *reinterpret_cast<uint4*>(dst + to0 + i * kRows * 128) = make_uint4(c0.x, c0.y, c1.x, c1.y);
        *reinterpret_cast<uint4*>(dst + to1 + i * kRows * 128) = make_uint4(c2.x, c2.y, c3.x, c3.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int j = r0 + i * kRows - tile.draft;
        const bool draft = v && j >= 0;
        store_any<F16>(x[i], byte[i], dst + to0 + i * kRows * 128, dst + to1 + i * kRows * 128,
                       draft ? &sh->bad[tile.seg % kBadSets][j >> 5] : nullptr, 1u << (j & 31));
      }
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&sh->full[at.slot]);
  }
  if (worst > top_page) set_status(a.status, DSPARK_EPAGES);
}

// e2m1 cache, through registers, as e4m3: a lane has 32 codes, two blocks, of one or two
// rows and multiplies them by their scales, exactly.  A warp has 16 rows of the tile; two
// lanes look a row's page up, ask for half of its scales each, and hand both round.  K and
// V have registers of their own, so that what is asked for is used a whole tile later.
template <bool F16, int DP>
__device__ __forceinline__ void produce4(const AttendArgs& a, uint8_t* smem, Tail* sh) {
  using L = Layout<DP>;
  constexpr int kWarps = Roles<kE2M1>::kProdWarps;
  constexpr int kLanes = DP / 32;                // of a row
  constexpr int kWarpRows = 32 / kLanes;
  constexpr int kRows = kWarps * kWarpRows;      // rows a pass
  constexpr int kPasses = kKeys / kRows;
  constexpr int kAhead = 4;
  static_assert(kWarps * 32 == 2 * kKeys, "one row of K or V a thread");
  static_assert(kPasses * kWarpRows == 16, "16 rows a warp");
  const int tid = threadIdx.x - kSoftWarps * 32, lane = tid % 32, warp = tid / 32;
  // Eight lanes store to all banks once: of 128 elements two rows whose numbers differ by two,
  // and in their second 64 elements, which lie behind the same banks, each pair of 16-byte
  // chunks the other way round.
  const int part = lane % kLanes, i0 = lane / kLanes;
  const int w0 = DP == 128 ? (i0 & 4) | (i0 & 1) << 1 | (i0 >> 1 & 1) : i0;
  const int r0 = warp * kWarpRows + w0, turn = DP == 128 ? part >> 1 : 0;
  const bool in_dim = part * 32 < a.D;
  uint32_t to[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) to[k] = tile_offset(r0, 4 * part + (k ^ turn));
  // row lane / 2 of the warp's, and which half of its scales
  const int own = lane / 2, half = lane & 1;
  const int own_row = own / kWarpRows * kRows + warp * kWarpRows + own % kWarpRows;
  const bool own_in = half * 64 < a.D;
  uint8_t* ring = smem + L::kRing;
  Cursor c;                                      // the tile whose loads come next
  c.init(a, sh->share);
  if (!c.more()) return;
  struct Tile {
    int head, rows, draft, seg;                  // rows that exist; the first of the draft
  };
  auto tile_at = [&]() {
    return Tile{c.head, min(kKeys, c.total() - c.t * kKeys), c.start - c.t * kKeys, c.seg};
  };
  const uint32_t top_page = (uint32_t)(a.c.n_pages - 1);
  uint32_t page = 0, worst = 0;
  int slot = 0;
  auto fetch_page = [&]() {
    const int pos = min(c.t * kKeys + own_row, c.total() - 1), at = a.c.page.div(pos);
    page = (uint32_t)__ldg(a.b.pages + (int64_t)c.b * a.b.pages_stride + at);
    slot = pos - at * a.c.page.d;
  };
  // rows of the same request kAhead tiles on, across a head's end, are asked for in L2, a
  // tile after their pages have been looked up
  uint32_t ask_page = ~0u;
  int ask_slot = 0, ask_head = 0;
  auto ask = [&]() {
    if (ask_page <= top_page) {
      ptx::prefetch_l2(a.c.x[tid >= kKeys].at(ask_page, ask_slot, ask_head));
      ptx::prefetch_l2(a.c.scale[tid >= kKeys].at(ask_page, ask_slot, ask_head));
    }
    ask_page = ~0u;
    int t = c.t + kAhead;
    ask_head = c.head;
    if (t >= c.tiles) {
      t -= c.tiles;
      ++ask_head;
    }
    if (ask_head >= a.Hkv || t >= c.tiles) return;
    const int pos = min(t * kKeys + tid % kKeys, c.total() - 1), at = a.c.page.div(pos);
    ask_page = (uint32_t)__ldg(a.b.pages + (int64_t)c.b * a.b.pages_stride + at);
    ask_slot = pos - at * a.c.page.d;
  };
  struct Part {
    uint4 x[kPasses];
    uint32_t scales;                             // four bytes of row `own`
  };
  auto load = [&](Part& half_tile, int v, int head) {
    const Rows rows = a.c.x[v];
    const uint8_t* src = rows.of_head(head) + (in_dim ? part * 16 : 0);
    const uint8_t* sc = a.c.scale[v].at(page, slot, head) + (own_in ? half * 4 : 0);
    if (a.D % 64 == 0) {
      half_tile.scales = __ldg(reinterpret_cast<const uint32_t*>(sc));
    } else {                                     // heads of 32 and 96: two bytes at their end
      half_tile.scales = __ldg(reinterpret_cast<const uint16_t*>(sc));
      if (half * 64 + 32 < a.D)
        half_tile.scales |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(sc) + 1) << 16;
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int from = 2 * (i * kWarpRows + w0);
      const uint32_t p = __shfl_sync(0xffffffffu, page, from);
      const int s = __shfl_sync(0xffffffffu, slot, from);
      half_tile.x[i] = ptx::ldg_nc_na(src + rows.offset(p, s));
    }
  };
  RingPos<L::kSlots> at;
  auto convert = [&](const Part& half_tile, bool v, const Tile& tile) {
    uint32_t scales = half_tile.scales;
    if (own_row >= tile.rows) scales = 0;        // rows past the end are zeros
    if (v && tile.draft < kKeys) {               // draft rows: zeros for blocks that are no numbers
      const uint32_t over = __vcmpgtu4(scales, kTopScale * 0x01010101u);
      const int j = own_row - tile.draft;
      if (j >= 0 && over != 0) {
        scales &= ~over;
        atomicOr(&sh->bad[tile.seg % kBadSets][j >> 5], 1u << (j & 31));
      }
    }
    wait(sh, &sh->empty[at.slot], at.phase ^ 1, a.status);
    uint8_t* dst = ring + at.slot * L::kTile;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const uint32_t four = __shfl_sync(0xffffffffu, scales, 2 * (i * kWarpRows + w0) + part / 2);
      const uint32_t two = in_dim ? four >> (part % 2 * 16) : 0u;
      const uint4 x = half_tile.x[i];
      const uint32_t w[4] = {turn ? x.y : x.x, turn ? x.x : x.y, turn ? x.w : x.z, turn ? x.z : x.w};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t s = e2m1_mul2<F16>(two >> (8 * h) & 0xffu);
#pragma unroll
        for (int k = 2 * h; k < 2 * h + 2; ++k)
          *reinterpret_cast<uint4*>(dst + to[k] + i * kRows * 128) = e2m1x8_times<F16>(w[k], s);
      }
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&sh->full[at.slot]);
    at.next();
  };
  Part k, v;
  auto clamp_page = [&]() {                      // a bad page is reported at the end
    worst = max(worst, page);
    page = min(page, top_page);
  };
  fetch_page();
  clamp_page();
  Tile cur = tile_at();
  load(k, 0, cur.head);
  load(v, 1, cur.head);
  c.next(a);
  bool more = c.more();
  if (more) fetch_page();
#pragma unroll 1
  while (true) {
    Tile next = cur;
    if (more) {
      next = tile_at();
      ask();
    }
    convert(k, false, cur);
    if (more) {
      clamp_page();
      load(k, 0, next.head);
    }
    convert(v, true, cur);
    if (!more) break;
    load(v, 1, next.head);
    cur = next;
    c.next(a);
    more = c.more();
    if (more) fetch_page();
  }
  if (worst > top_page) set_status(a.status, DSPARK_EPAGES);
}

// ------------------------------------------------------------------- MMA --

// One warp a stream; all lanes run the loop and one issues, so that descriptors
// stay in uniform registers.
template <bool F16, int DP>
__device__ __forceinline__ void issue(const AttendArgs& a, uint8_t* smem, Tail* sh, int stream) {
  using L = Layout<DP>;
  constexpr uint32_t kTypes = F16 ? (1u << 7) | (1u << 10) : 0u;   // bf16 fields, cleared for f16
  constexpr uint32_t kQK = ptx::idesc_bf16_f32(128, kKeys) & ~kTypes;
  constexpr uint32_t kQKHalf = ptx::idesc_bf16_f32(128, kHalf) & ~kTypes;
  constexpr uint32_t kPV = (ptx::idesc_bf16_f32(128, DP) & ~kTypes) | (1u << 16);  // B N-major
  const uint32_t tm_s = sh->tmem + stream * 128, tm_o = sh->tmem + 256 + stream * 128;
  const uint32_t ring = ptx::smem_u32(smem + L::kRing);
  Walker w;
  Segment s;
  w.init(a, sh->share);
  RingPos<L::kSlots> at;
  uint32_t count[2] = {0, 0};                    // products so far, of h
  bool pair = false;
  uint64_t q_desc = 0;
  // the next slot of the ring, filled; also those that are only passed: every phase
  // is waited for in order
  auto take = [&]() {
    const uint32_t slot = at.slot;
    wait(sh, &sh->full[slot], at.phase, a.status);
    at.next();
    return slot;
  };
  auto filled = [&]() {                          // whether the next slot is
    return __any_sync(0xffffffffu, ptx::mbar_test_wait(&sh->full[at.slot], at.phase)) != 0;
  };
  // a slot is free when both streams have let go of it: by the products that read
  // it, or, for one that is only passed, by this warp after its wait.  So no slot
  // is refilled, and no phase runs on, before both have seen it filled.
  auto release = [&](uint32_t slot) { ptx::tc_commit(&sh->empty[slot]); };
  auto pass = [&](uint32_t slot) {
    __syncwarp();                                // every lane's wait is over
    if (threadIdx.x % 32 == 0) ptx::mbar_arrive(&sh->empty[slot]);
  };
  auto scores = [&](uint32_t slot, int h, bool all) {      // S of half a tile, or of all of it
    if (!aborted(sh)) {
      ptx::tc_fence_after();
      const uint64_t k_desc =
          ptx::smem_desc_swizzle128(ring + slot * L::kTile + h * (kHalf * 128), 16, 1024);
      const uint32_t type = all ? kQK : kQKHalf;
      if (ptx::elect_one()) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
          ptx::tc_mma_smem(tm_s + h * kHalf, q_desc + (k / 4) * (kKeys * 128 / 16) + (k % 4) * 2,
                           k_desc + (k / 4) * (kKeys * 128 / 16) + (k % 4) * 2, type, k > 0);
        ptx::tc_commit(&sh->s_full[stream][h]);
        if (all && pair) ptx::tc_commit(&sh->s_full[stream][1]);
        if (all || h == 1) release(slot);
      }
      __syncwarp();
    }
  };
  // O += P V of half a tile, or of all of it (h = 0), and the wait for it
  auto values = [&](uint32_t slot, int h, bool add) {
    const uint32_t phase = count[h]++ & 1;
    wait(sh, &sh->p_full[stream][h], phase, a.status);
    if (!aborted(sh)) {
      ptx::tc_fence_after();
      const uint64_t v_desc =
          ptx::smem_desc_swizzle128(ring + slot * L::kTile + h * (kHalf * 128), kKeys * 128, 1024);
      if (ptx::elect_one()) {
#pragma unroll
        for (int k = 0; k < kHalf / 16; ++k)
          ptx::tc_mma_tmem_a(tm_o, tm_s + h * kHalf + 8 * k, v_desc + k * (2048 / 16), kPV,
                             add || k > 0);
        if (!pair) {
#pragma unroll
          for (int k = kHalf / 16; k < kKeys / 16; ++k)
            ptx::tc_mma_tmem_a(tm_o, tm_s + 8 * k, v_desc + k * (2048 / 16), kPV, true);
        }
        ptx::tc_commit(&sh->o_done[stream][h]);
        if (!pair || h == 1) release(slot);
      }
      __syncwarp();
    }
    wait(sh, &sh->o_done[stream][h], phase, a.status);
  };
  for (uint32_t seg = 0; w.next(a, &s); ++seg) {
    pair = Item::group_rows(a, s) > kKeys;
    const int n = s.t1 - s.t0;
    q_desc = ptx::smem_desc_swizzle128(ptx::smem_u32(smem) + (pair ? stream * L::kTile : 0), 16,
                                       1024);
    wait(sh, &sh->q_full, seg & 1, a.status);
    if (pair) {
      // S and P share columns, so the next S of a half follows the product that read
      // its P: made while the softmax works on the other half, unless K has not come
      // (the producers may need this tile's V slot to get there)
      uint32_t k_slot = take();
      scores(k_slot, 0, true);
      for (int i = 0;; ++i) {
        const uint32_t v_slot = take();
        values(v_slot, 0, i > 0);
        const bool early = i + 1 < n && filled();
        if (early) {
          k_slot = take();
          scores(k_slot, 0, false);
        }
        values(v_slot, 1, true);
        if (i + 1 == n) break;
        if (!early) k_slot = take();
        scores(k_slot, early ? 1 : 0, !early);
      }
    } else {
      // a tile at a time: nothing but V's slot is held, and the ring's depth, which
      // is what counts with few rows, is the copies'
      for (int i = 0; i < n; ++i) {
        const uint32_t k_slot = take();
        const bool own = (i & 1) == stream;
        if (own) scores(k_slot, 0, true);
        else pass(k_slot);
        const uint32_t v_slot = take();
        if (own) values(v_slot, 0, i > 1);
        else pass(v_slot);
      }
    }
    if (threadIdx.x % 32 == 0) ptx::mbar_arrive(&sh->q_empty);
  }
}

// The parts' places for the join, by a warp that has nothing else to do (1.1 us of
// divisions).
__device__ __forceinline__ void place_parts(const AttendArgs& a, Tail* sh) {
  Walker w;
  Segment s;
  w.init(a, sh->share);
  while (w.next(a, &s))
    if (threadIdx.x % 32 == 0 && !s.whole())
      a.part_of[2 * blockIdx.x + (s.t0 == 0 ? 1 : 0)] = Item::part_of(s, sh->share.cut);
}

// --------------------------------------------------------------- softmax --

// Adds to a row's result, which the calling thread has just written (columns d0
// .. d1 - 1), the non-finite elements of the draft rows of V that it sees: what
// 0 < p times them comes to.  The result: 16-bit values (out), or the part's fp32
// ones (column d at part[(d / 4) * stride + d % 4]).
template <bool F16, int HELD>
__device__ __noinline__ void add_nonfinite(const AttendArgs& a, const uint32_t* bad,
                                           const uint32_t* mask_row, int b, int rows, int start,
                                           int head, int node, int d0, int d1, uint16_t* out,
                                           float* part, int64_t stride) {
#pragma unroll 1
  for (int j = 0; j < rows; ++j) {
    if (!(sees_word(mask_row, rows, node, j >> 5) & bad[j >> 5] & (1u << (j & 31)))) continue;
#pragma unroll 1
    for (int d = d0; d < d1; ++d) {
      const float x = bad_value<F16, HELD>(a, b, start + j, head, d);
      if (isfinite(x)) continue;
      if (out) out[d] = (uint16_t)pack2<F16>(to_float<F16>(out[d]) + x, 0.f);
      else part[(d >> 2) * stride + (d & 3)] += x;
    }
  }
}

// Two values of at most 2^100 rounded to eight significant bits (Veltkamp's splitting):
// upper halves that are theirs as bf16, without the conversion pipe and with their floats
// at hand.
__device__ __forceinline__ uint64_t round8_f32x2(uint64_t x) {
  // the product rounded by itself: as a fused one with the zero, which is fused no further
  const uint64_t t = fma_f32x2(x, pack_f32x2(65537.f, 65537.f), pack_f32x2(0.f, 0.f));
  return sub_f32x2(t, sub_f32x2(t, x));
}
// O of this row times `back`.
template <int DP>
__device__ __forceinline__ void scale_row(uint32_t tm_o, float back) {
#pragma unroll 1
  for (int c = 0; c < DP / 32; ++c) {
    uint32_t v[32];
    ptx::tmem_ld32(tm_o + 32 * c, v);
    ptx::tmem_wait_ld32(v);
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * back);
    ptx::tmem_st32(tm_o + 32 * c, v);
  }
}

// How far a row's maximum may grow past the one that set m before m moves.  Over e2m1
// codes in bf16 as far as O and l in fp32 bear (2^64 times 2^16 times 2^31 keys): a weight
// has bf16's relative precision whatever its size, and what moves m costs (64 x 64 with
// a key in 50 eight times the others: 8 607 us, 64 495).  In f16 no further than f16 goes.
template <bool F16, int HELD>
constexpr bool far_growth() {
  return HELD == kE2M1 && !F16;
}
template <bool F16, int HELD>
constexpr float grow_limit() {
  return far_growth<F16, HELD>() ? 64.f : 8.f;
}

// A row's sum of weights, and, where m need not be near the maximum, of the weights as
// they are rounded.  There a row's largest weights are no powers of two (next to a m that
// is the maximum the largest is 1), and divided by the sum that is not rounded their
// error would be that of a row with few large ones (2.2e-3 of the result in all, bf16's own
// rounding 1.6e-3); divided by the rounded sum it is not.
template <bool FAR>
struct Sum {
  float l = 0.f, rounded = 0.f;
  __device__ __forceinline__ void times(float x) {
    l *= x;
    rounded *= x;
  }
};
template <>
struct Sum<false> {                              // any other row's
  float l = 0.f;
  __device__ __forceinline__ void times(float x) { l *= x; }
};
template <bool F16, int HELD>
using SumOf = Sum<far_growth<F16, HELD>()>;

// What two packed bf16 weights come to.
__device__ __forceinline__ void add_rounded(uint32_t pk, float* even, float* odd) {
  *even += __uint_as_float(pk << 16);
  *odd += __uint_as_float(pk & 0xffff0000u);
}

// The row's m after keys whose largest exponent is x_max; l and O follow if it
// moves: the first visible key sets it, later ones when it has grown enough.  O
// is free to scale once the last product is done (o_done, null before the first).
template <bool F16, int HELD, int DP>
__device__ __forceinline__ float move_reference(float x_max, Tail* sh, uint64_t* o_done,
                                                uint32_t parity, int* status, uint32_t tm_o,
                                                float mref, SumOf<F16, HELD>* l) {
  constexpr float kShift = F16 ? 7.f : 0.f;
  const bool move = x_max > mref + (mref == -INFINITY ? 0.f : kShift + grow_limit<F16, HELD>());
  const float m_new = move ? x_max - kShift : mref;
  if (o_done && __any_sync(0xffffffffu, move)) {
    wait(sh, o_done, parity, status);
    ptx::tc_fence_after();
    const float back = mref == -INFINITY ? 0.f : ex2(mref - m_new);
    l->times(back);
    scale_row<DP>(tm_o, back);
  }
  return m_new;
}

// KEYS keys (a tile or half) of one row that are all visible, scores not capped, m
// set: P over S, and l.  The weights go by m as it stands while the maximum is
// taken beside them, so nothing waits for it; if it has outgrown m in any row of
// the warp, S is still there and they are done again (false; x_max is the row's largest
// exponent).  A 16-bit cache: the next 32 scores are loaded while these are worked on.
template <bool F16, int HELD, int KEYS>
__device__ __forceinline__ bool softmax_plain(float sl2, uint32_t tm_s, float mref,
                                              SumOf<F16, HELD>* l, float* x_max) {
  constexpr float kShift = F16 ? 7.f : 0.f;
  constexpr bool WIDE = HELD == k16;
  constexpr int kBuf = WIDE ? 2 : 1, kChunks = KEYS / 32;
  uint32_t v[kBuf][32], pk[kChunks][16];
  float mx[2] = {-INFINITY, -INFINITY}, sum[4] = {0.f, 0.f, 0.f, 0.f};
  uint64_t sum2[2] = {0, 0}, rounded2[2] = {0, 0};         // pairs of zeros
  const uint64_t mul = pack_f32x2(sl2, sl2), neg = pack_f32x2(-mref, -mref);
  ptx::tmem_ld32(tm_s, v[0]);
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    uint32_t (&x)[32] = v[c % kBuf];
    ptx::tmem_wait_ld32(x);
    if (WIDE && c < kChunks - 1) ptx::tmem_ld32(tm_s + 32 * (c + 1), v[(c + 1) % kBuf]);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float r0 = __uint_as_float(x[2 * k]), r1 = __uint_as_float(x[2 * k + 1]);
      mx[k & 1] = fmaxf(mx[k & 1], fmaxf(r0, r1));
      float p0, p1;
      unpack_f32x2(fma_f32x2(pack_f32x2(r0, r1), mul, neg), &p0, &p1);
      p0 = ex2(p0);
      p1 = ex2(p1);
      if constexpr (far_growth<F16, HELD>()) {
        const uint64_t p = pack_f32x2(p0, p1), near = round8_f32x2(p);
        sum2[k & 1] = add_f32x2(sum2[k & 1], p);
        rounded2[k & 1] = add_f32x2(rounded2[k & 1], near);
        unpack_f32x2(near, &p0, &p1);
        pk[c][k] = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
      } else {
        sum[2 * k & 3] += p0;
        sum[(2 * k + 1) & 3] += p1;
        pk[c][k] = pack2<F16>(p0, p1);
      }
    }
    if (!WIDE && c < kChunks - 1) ptx::tmem_ld32(tm_s + 32 * (c + 1), v[0]);
  }
  *x_max = fmaxf(mx[0], mx[1]) * sl2;
  if (__any_sync(0xffffffffu, *x_max > mref + (kShift + grow_limit<F16, HELD>()))) return false;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) ptx::tmem_st16(tm_s + 16 * c, pk[c]);
  if constexpr (far_growth<F16, HELD>()) {
    unpack_f32x2(add_f32x2(sum2[0], sum2[1]), &sum[0], &sum[1]);
    float r0, r1;
    unpack_f32x2(add_f32x2(rounded2[0], rounded2[1]), &r0, &r1);
    l->rounded += r0 + r1;
  }
  l->l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
  ptx::tmem_wait_st();
  return true;
}

// 64 or 128 keys of one row, also with invisible keys (see: a bit a key), capped
// scores, or a maximum that moves m; 32 keys at a time.  Returns m and the sums.
template <bool FAR>
struct Softened {
  float m;
  Sum<FAR> l;
};
template <bool F16, int HELD, int DP>
__device__ __noinline__ Softened<far_growth<F16, HELD>()> softmax_any(
    Score sc, Tail* sh, uint64_t* o_done, uint32_t parity, int* status, uint32_t tm_s, uint32_t tm_o,
    int keys, uint4 see, float mref, SumOf<F16, HELD> l) {
  const bool cap = sc.cap2 > 0.f;
  uint32_t any = 0;                              // whether the row sees one of the keys
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
  for (int c = 0; c < keys / 32; ++c) {
    const uint32_t m = c == 0 ? see.x : c == 1 ? see.y : c == 2 ? see.z : see.w;
    uint32_t v[32];
    ptx::tmem_ld32(tm_s + 32 * c, v);
    ptx::tmem_wait_ld32(v);
    any |= m;
#pragma unroll
    for (int k = 0; k < 32; ++k)
      mx[k & 3] = fmaxf(mx[k & 3], (m >> k) & 1 ? __uint_as_float(v[k]) : -INFINITY);
  }
  const float raw_max = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
  float x_max = raw_max == -INFINITY ? -INFINITY : raw_max * sc.sl2;
  // a visible score of -infinity is the cap's negative, an invisible one nothing
  if (cap && any != 0) x_max = capped(sc, raw_max, 0.f);
  mref = move_reference<F16, HELD, DP>(x_max, sh, o_done, parity, status, tm_o, mref, &l);
  const float sub = mref == -INFINITY ? 0.f : mref;
  // coefficients of capped_near.  No special functions but the weight's own where all
  // of 8 keys are far from the cap in all rows of the warp; 16 requests of 64 nodes, 300
  // to 6,000 tokens, 16-bit: 130 us where all are, 168 where in all groups some are not
  // (no cap 84).
  uint64_t coef[6];
#pragma unroll
  for (int i = 0; i < 6; ++i)
    coef[i] = pack_f32x2(sc.cap2 * tanh_coef(i), sc.cap2 * tanh_coef(i));
  const uint64_t neg = pack_f32x2(-sub, -sub);
  const float past0 = sc.cap2 - sub;
  // scores k0 .. k0 + n - 1 to exponents, two at once, by capped_near; `both`: those
  // past it by capped_past
  auto cap_pairs = [&](uint32_t (&v)[32], int k0, int n, bool both) {
#pragma unroll
    for (int k = k0; k < k0 + n; k += 2) {
      const uint64_t raw = pack_f32x2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
      const uint64_t y = mul_f32x2(raw, pack_f32x2(sc.cap_y, sc.cap_y));
      const uint64_t u = mul_f32x2(y, y);
      uint64_t t = coef[5];
#pragma unroll
      for (int i = 4; i >= 0; --i) t = fma_f32x2(t, u, coef[i]);
      float x[2];
      unpack_f32x2(fma_f32x2(y, t, neg), &x[0], &x[1]);
      if (both) {
        float z[2], yy[2], r[2];
        unpack_f32x2(mul_f32x2(raw, pack_f32x2(sc.cap_in, sc.cap_in)), &z[0], &z[1]);
        unpack_f32x2(y, &yy[0], &yy[1]);
        const uint64_t d = pack_f32x2(rcp(ex2(z[0]) + 1.f), rcp(ex2(z[1]) + 1.f));
        unpack_f32x2(fma_f32x2(d, pack_f32x2(-2.f * sc.cap2, -2.f * sc.cap2),
                               pack_f32x2(past0, past0)), &r[0], &r[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) x[e] = fabsf(yy[e]) > kNearCap ? r[e] : x[e];
      }
      v[k] = __float_as_uint(x[0]);
      v[k + 1] = __float_as_uint(x[1]);
    }
  };
  float sum[2] = {0.f, 0.f}, rounded[2] = {0.f, 0.f};
#pragma unroll 1
  for (int c = 0; c < keys / 32; ++c) {
    const uint32_t m = c == 0 ? see.x : c == 1 ? see.y : c == 2 ? see.z : see.w;
    uint32_t v[32], pk[16];
    ptx::tmem_ld32(tm_s + 32 * c, v);
    ptx::tmem_wait_ld32(v);
    if (cap) {
      float big[4] = {0.f, 0.f, 0.f, 0.f};       // of 8 keys each
#pragma unroll
      for (int k = 0; k < 32; ++k) big[k / 8] = fmaxf(big[k / 8], fabsf(__uint_as_float(v[k])));
      if (!__any_sync(0xffffffffu, past_near(sc, fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3]))))) {
        cap_pairs(v, 0, 32, false);
      } else {
#pragma unroll
        for (int k0 = 0; k0 < 32; k0 += 8) {
          if (__any_sync(0xffffffffu, past_near(sc, big[k0 / 8]))) cap_pairs(v, k0, 8, true);
          else cap_pairs(v, k0, 8, false);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        v[k] = __float_as_uint(fmaf(__uint_as_float(v[k]), sc.sl2, -sub));
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float p0 = (m >> (2 * k)) & 1 ? ex2(__uint_as_float(v[2 * k])) : 0.f;
      const float p1 = (m >> (2 * k + 1)) & 1 ? ex2(__uint_as_float(v[2 * k + 1])) : 0.f;
      sum[0] += p0;
      sum[1] += p1;
      pk[k] = pack2<F16>(p0, p1);
      if (far_growth<F16, HELD>()) add_rounded(pk[k], &rounded[0], &rounded[1]);
    }
    ptx::tmem_st16(tm_s + 16 * c, pk);
  }
  ptx::tmem_wait_st();
  l.l += sum[0] + sum[1];
  if constexpr (far_growth<F16, HELD>()) l.rounded += rounded[0] + rounded[1];
  return {mref, l};
}

template <bool F16, int HELD, int DP>
__device__ __forceinline__ void softmax(const AttendArgs& a, uint8_t* smem, Tail* sh) {
  using L = Layout<DP>;
  constexpr bool kSwapped = !F16 && HELD == kE4M3;       // the codes' order (scale_codes)
  const int wg = threadIdx.x / 128, lane_row = threadIdx.x % 128;
  const int warp = threadIdx.x / 32 % 4;
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  const uint32_t tm_s = sh->tmem + lanes + wg * 128;
  const uint32_t tm_o = sh->tmem + lanes + 256;
  const Score sc = Score::of(a);
  const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
  Walker w;
  Segment s;
  w.init(a, sh->share);
  uint32_t count0 = 0, count1 = 0;               // steps of this stream so far, of h
  for (uint32_t seg = 0; w.next(a, &s); ++seg) {
    const int rows = Item::group_rows(a, s);
    const bool pair = rows > kKeys;
    const int n = s.t1 - s.t0;
    // Q into shared memory, all 256 threads
    {
      constexpr int kChunks = DP / 8, kStep = 256 / kChunks;
      const int q_rows = pair ? kGroupRows : kKeys, chunk = threadIdx.x % kChunks;
      const bool in_dim = chunk * 8 < a.D;
      auto place = [&](int r) {
        return reinterpret_cast<uint4*>(smem + (r / kKeys) * L::kTile +
                                        tile_offset(r % kKeys, chunk));
      };
#pragma unroll 2
      for (int r = threadIdx.x / kChunks; r < q_rows; r += kStep) {
        const bool on = in_dim && r < rows;
        const int gr = s.group * kGroupRows + (on ? r : 0), nd = a.group.div(gr);
        const uint8_t* src = a.q + (int64_t)(s.row0 + nd) * a.q_row +
                             (int64_t)(s.head * a.G + gr - nd * a.G) * a.q_head;
        ptx::cp_async16_or_zero(place(r), on ? src + chunk * 16 : src, on);
      }
      ptx::cp_async_commit();
      ptx::cp_async_wait_group<0>();
      if (kSwapped || flip) {                    // each thread the chunks that it copied
#pragma unroll 1
        for (int r = threadIdx.x / kChunks; r < q_rows; r += kStep) {
          uint4 x = *place(r);
          x.x ^= flip;
          x.y ^= flip;
          x.z ^= flip;
          x.w ^= flip;
          if (kSwapped) {
            const uint2 lo = swap_middle(make_uint2(x.x, x.y)), hi = swap_middle(make_uint2(x.z, x.w));
            x = make_uint4(lo.x, lo.y, hi.x, hi.y);
          }
          *place(r) = x;
        }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (threadIdx.x % 32 == 0) ptx::mbar_arrive(&sh->q_full);
    }
    const int local = (pair ? wg * kKeys : 0) + lane_row;        // row of the group
    const bool valid = local < rows;
    const bool warp_valid = local - threadIdx.x % 32 < rows;
    const int grow = s.group * kGroupRows + (valid ? local : 0);
    const int node = a.group.div(grow);
    const uint32_t* mask_row =
        a.mask ? a.mask + (int64_t)(s.row0 + node) * a.mask_stride : nullptr;
    float mref = -INFINITY, l = 0.f;
    SumOf<F16, HELD> sums;
    const int step = pair ? 1 : 2;
    const int keys = pair ? kHalf : kKeys;       // of one step
    for (int i = pair ? 0 : wg; i < n; i += step) {
#pragma unroll 1
      for (int h = 0; h < (pair ? 2 : 1); ++h) {
        wait(sh, &sh->s_full[wg][h], (h ? count1 : count0) & 1, a.status);
        ptx::tc_fence_after();
        if (warp_valid) {
          const int pos0 = (s.t0 + i) * kKeys + h * kHalf;
          const bool masked = pos0 + keys > s.start;
          bool done = !masked && sc.cap2 == 0.f && !__any_sync(0xffffffffu, mref == -INFINITY);
          // the product before this one
          const int before = pair ? h ^ 1 : 0;
          auto phase = [&]() { return ((before ? count1 : count0) - 1) & 1; };
          auto o_done = [&]() { return h == 1 || i >= step ? &sh->o_done[wg][before] : nullptr; };
          if (done) {
            float x_max;
            auto plain = [&]() {
              return pair ? softmax_plain<F16, HELD, kHalf>(sc.sl2, tm_s + h * kHalf, mref, &sums, &x_max)
                          : softmax_plain<F16, HELD, kKeys>(sc.sl2, tm_s, mref, &sums, &x_max);
            };
            done = plain();
            if (HELD == kE2M1 && !done) {        // as long as m follows, the second time it fits
              mref = move_reference<F16, HELD, DP>(x_max, sh, o_done(), phase(), a.status, tm_o + wg * 128,
                                                   mref, &sums);
              done = plain();
            }
          }
          if (!done) {
            const auto r = softmax_any<F16, HELD, DP>(
                sc, sh, o_done(), phase(), a.status, tm_s + h * kHalf, tm_o + wg * 128, keys,
                masked ? sees_128(mask_row, s.rows, node, pos0 - s.start)
                       : make_uint4(~0u, ~0u, ~0u, ~0u),
                mref, sums);
            mref = r.m;
            sums = r.l;
          }
          ptx::tc_fence_before();
        }
        __syncwarp();
        if (threadIdx.x % 32 == 0) ptx::mbar_arrive(&sh->p_full[wg][h]);
        if (h == 0) ++count0;
        else ++count1;
      }
    }

    // as O's weights add up to the rounded sum, m stands so much higher that the sum is the
    // same: from here on m and l are any row's
    l = sums.l;
    if constexpr (far_growth<F16, HELD>()) {
      if (sums.rounded > 0.f) {
        mref += log2f(sums.l / sums.rounded);
        l = sums.rounded;
      }
    }
    // the segment's result
    const int n1 = n / 2;                        // the second stream's tiles, not in pairs
    if (pair || wg < n) wait(sh, &sh->o_done[wg][0], (count0 - 1) & 1, a.status);
    if (pair) wait(sh, &sh->o_done[wg][1], (count1 - 1) & 1, a.status);
    if (!pair) sh->ml[wg][lane_row] = make_float2(mref, l);
    ptx::tc_fence_before();
    asm volatile("bar.sync 1, 256;" ::: "memory");
    ptx::tc_fence_after();
    float w0 = 1.f, w1 = 0.f;                    // weights of the two streams' O
    if (!pair) {
      const float2 x0 = sh->ml[0][lane_row], x1 = sh->ml[1][lane_row];
      mref = fmaxf(x0.x, x1.x);
      const float sub = mref == -INFINITY ? 0.f : mref;
      w0 = ex2(x0.x - sub);
      w1 = n1 > 0 ? ex2(x1.x - sub) : 0.f;
      l = w0 * x0.y + (n1 > 0 ? w1 * x1.y : 0.f);
    }
    wait(sh, &sh->q_empty, seg & 1, a.status);   // both MMA warps are past it
    const bool whole = s.whole();
    const int part = 2 * blockIdx.x + (s.t0 == 0 ? 1 : 0);
    const uint32_t* bad = sh->bad[seg % kBadSets];
    uint32_t any_bad = 0;
#pragma unroll
    for (int k = 0; k < DSPARK_TREE_MAX_NODES / 32; ++k) any_bad |= bad[k];
    if (warp_valid) {
      const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
      const int64_t out_row = (int64_t)(s.row0 + node) * a.Hq + s.head * a.G + grow - node * a.G;
      // pair: a group its own row tile, all columns; else both tiles, half the columns
      const int c0 = pair ? 0 : wg * (DP / 64), c1 = pair ? DP / 32 : c0 + DP / 64;
      // 16-byte chunks of a row here: kPer places, of which not in pairs half is used
      constexpr int kPer = DP / 8;
      const int lane = threadIdx.x % 32;
      uint4* q_rows = reinterpret_cast<uint4*>(smem) + (threadIdx.x / 32) * 32 * kPer;
#pragma unroll 1
      for (int c = c0; c < c1; ++c) {
        uint32_t v[32];
        float o[32];
        ptx::tmem_ld32(tm_o + (pair ? wg * 128 : 0) + 32 * c, v);
        ptx::tmem_wait_ld32(v);
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = __uint_as_float(v[k]) * w0;
        if (!pair && n1 > 0) {
          ptx::tmem_ld32(tm_o + 128 + 32 * c, v);
          ptx::tmem_wait_ld32(v);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = fmaf(__uint_as_float(v[k]), w1, o[k]);
        }
        if (kSwapped) {
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float y = o[k + 1];
            o[k + 1] = o[k + 2];
            o[k + 2] = y;
          }
        }
        if (whole) {                             // to the warp's rows in Q's place
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = l == 0.f ? 0u : pack2<F16>(o[8 * k + 2 * e] * inv, o[8 * k + 2 * e + 1] * inv);
            q_rows[lane * kPer + (4 * (c - c0) + k ^ lane % kPer)] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        } else if (valid) {
          float4* dst = reinterpret_cast<float4*>(a.part_o) +
                        ((int64_t)part * (DP / 4) + 8 * c) * a.part_rows + local;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[(int64_t)k * a.part_rows] =
                make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
        __syncwarp();
      }
      if (whole) {                               // whole rows at a time to memory
        const int per = 4 * (c1 - c0), n_chunks = per * min(32, rows - (local - lane));
#pragma unroll 4
        for (int k = lane; k < 32 * per; k += 32) {
          const int r = k / per, chunk = k % per;
          const int64_t to = __shfl_sync(0xffffffffu, out_row, r);
          if (k < n_chunks && (4 * c0 + chunk) * 8 < a.D)
            reinterpret_cast<uint4*>(a.out + to * a.D)[4 * c0 + chunk] =
                q_rows[r * kPer + (chunk ^ r % kPer)];
        }
        __syncwarp();
      }
      if (valid && any_bad != 0)
        add_nonfinite<F16, HELD>(
            a, bad, mask_row, s.b, s.rows, s.start, s.head, node, 32 * c0, min(32 * c1, a.D),
            whole ? a.out + out_row * a.D : nullptr,
            a.part_o + ((int64_t)part * (DP / 4) * a.part_rows + local) * 4,
            (int64_t)a.part_rows * 4);
      __syncwarp();
      if (valid && (pair || wg == 0)) {
        if (!whole) a.part_ml[(int64_t)part * a.part_rows + local] = make_float2(mref, l);
        else if (a.lse) a.lse[out_row] = l == 0.f ? -INFINITY : (mref + log2f(l)) * kLn2;
      }
    }
    ptx::tc_fence_before();
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (any_bad != 0 && threadIdx.x < DSPARK_TREE_MAX_NODES / 32)
      sh->bad[seg % kBadSets][threadIdx.x] = 0;
  }
}

// REGS: the registers a thread that the roles' split counts on at launch.  In the
// kernel's name, where the build checks it against what the compiler gave.
template <bool F16, int HELD, int DP, int REGS>
__global__ void __launch_bounds__(Roles<HELD>::kThreads, 1)
    attend_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ TileMaps maps) {
  using R = Roles<HELD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Tail* sh = reinterpret_cast<Tail*>(smem + Layout<DP>::kTail);
  const int warp = threadIdx.x / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == R::kMmaWarp) {
    ptx::tmem_alloc(&sh->tmem, 512);
    ptx::tmem_relinquish();
  }
  if (HELD == k16 && threadIdx.x == kSoftWarps * 32 && maps.rows > 0) {
    ptx::prefetch_tensormap(&maps.k);
    ptx::prefetch_tensormap(&maps.v);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      ptx::mbar_init(&sh->full[i], R::kProdWarps);
      ptx::mbar_init(&sh->empty[i], 2);
    }
    ptx::mbar_init(&sh->q_full, kSoftWarps);
    ptx::mbar_init(&sh->q_empty, 2);
    for (int i = 0; i < 2; ++i) {
      for (int h = 0; h < 2; ++h) {
        ptx::mbar_init(&sh->s_full[i][h], 1);
        ptx::mbar_init(&sh->p_full[i][h], 4);
        ptx::mbar_init(&sh->o_done[i][h], 1);
      }
    }
    ptx::fence_mbar_init();
    sh->abort = 0;
    a.part_of[2 * blockIdx.x] = a.part_of[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
  }
  for (int i = threadIdx.x; i < kBadSets * (DSPARK_TREE_MAX_NODES / 32); i += R::kThreads)
    (&sh->bad[0][0])[i] = 0;
  Item::plan<R::kThreads>(a, &sh->share, sh->warp_sum);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp < kSoftWarps) {
    ptx::set_registers<REGS, R::kSoftRegs>();
    softmax<F16, HELD, DP>(a, smem, sh);
  } else if (warp < R::kMmaWarp) {
    ptx::set_registers<REGS, R::kProdRegs>();
    if (HELD == kE2M1) produce4<F16, DP>(a, smem, sh);
    else if (HELD == kE4M3) produce8<F16, DP>(a, smem, sh);
    else produce16<F16, DP>(a, maps, smem, sh);
  } else {
    ptx::set_registers<REGS, R::kMmaRegs>();
    if (warp < R::kMmaWarp + 2)
      issue<F16, DP>(a, smem, sh, warp - R::kMmaWarp);
    else if (warp == R::kMmaWarp + 2) place_parts(a, sh);
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (aborted(sh)) {                              // let what was started land
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
  }
  __syncwarp();
  if (warp == R::kMmaWarp) ptx::tmem_dealloc(sh->tmem, 512);
}

// Joins the parts of the items that several CTAs share, in pieces of 32 rows (lane
// = row) by 16 columns.  An item of P parts has P x kJoinSplit blocks: block (p, y)
// of a part's slot p takes every (P x kJoinSplit)-th of its pieces, or of groups of
// eight where one warp joins a piece alone (up to kJoinAlone parts).  With more
// parts the warps of a block take every eighth one and are then added in order:
// the result does not depend on timing.  Alone for none / 4 / 8 / any number: 13
// trees 58.8 / 49.8 / 47.9 / 48.2 us, 64 x 64 431 / 404 / 405 / 397 (up to 3 parts),
// 17 nodes over 131,000 tokens (20 parts) 106 / 102.7 / 102.7 / 114.3.
constexpr int kJoinThreads = 256;
constexpr int kJoinSplit = 4;
constexpr int kJoinAlone = 8;

struct JoinSum {
  float m = -INFINITY, l = 0.f;
  float4 o[4] = {};

  // adds parts first + i, first + i + step, ... below `parts`
  template <int DP, int UNROLL>
  __device__ __forceinline__ void add(const AttendArgs& a, int first, int parts, int i, int step,
                                      int c4, int local) {
#pragma unroll UNROLL
    for (; i < parts; i += step) {
      const int64_t part = 2 * (first + i) + (i == 0 ? 1 : 0);
      const float2 ml = a.part_ml[part * a.part_rows + local];
      const float4* src = reinterpret_cast<const float4*>(a.part_o) +
                          (part * (DP / 4) + c4) * a.part_rows + local;
      float4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = src[(int64_t)k * a.part_rows];
      const float m_new = fmaxf(m, ml.x), sub = m_new == -INFINITY ? 0.f : m_new;
      const float wo = ex2(m - sub), wx = ex2(ml.x - sub);
      m = m_new;
      l = l * wo + ml.y * wx;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[k].x = o[k].x * wo + x[k].x * wx;
        o[k].y = o[k].y * wo + x[k].y * wx;
        o[k].z = o[k].z * wo + x[k].z * wx;
        o[k].w = o[k].w * wo + x[k].w * wx;
      }
    }
  }
};

template <bool F16>
__device__ __forceinline__ uint2 join_pack(float4 s, float l) {
  if (l == 0.f) return make_uint2(0u, 0u);
  const float inv = 1.f / l;
  return make_uint2(pack2<F16>(s.x * inv, s.y * inv), pack2<F16>(s.z * inv, s.w * inv));
}

template <bool F16, int DP>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttendArgs a) {
  __shared__ float4 part_sum[8][4][32];
  __shared__ float2 part_ml[8][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 of = a.part_of[blockIdx.x];
  const int parts = of.w >> 16, first = of.w & 0xffff, head = of.y, group = of.z;
  if (parts == 0) return;
  bool ok;
  const Item::Request r = Item::load_request(a, of.x, &ok);
  const int rows = min(kGroupRows, r.rows * a.G - group * kGroupRows);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int pieces = (rows + 31) / 32 * (DP / 16);
  // this block's place among the item's: which part's slot, and y
  const int mine = ((int)blockIdx.x / 2 - first) * kJoinSplit + blockIdx.y;
  const bool alone = parts <= kJoinAlone;
  const int step = parts * kJoinSplit * (alone ? 8 : 1);
  for (int piece = alone ? mine * 8 + warp : mine; piece < pieces; piece += step) {
    const int c4 = piece % (DP / 16) * 4, local = piece / (DP / 16) * 32 + lane;   // float4 column
    const int grow = group * kGroupRows + local, node = a.group.div(grow);
    const int64_t out_row = (int64_t)(r.row0 + node) * a.Hq + head * a.G + grow - node * a.G;
    JoinSum s;
    if (alone) {
      s.add<DP, 2>(a, first, parts, 0, 1, c4, local);
      if (local >= rows) continue;
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const uint2 x = join_pack<F16>(s.o[k], s.l), y = join_pack<F16>(s.o[k + 1], s.l);
        if (4 * (c4 + k) < a.D)
          *reinterpret_cast<uint4*>(a.out + out_row * a.D + 4 * (c4 + k)) =
              make_uint4(x.x, x.y, y.x, y.y);
      }
      if (c4 == 0 && a.lse) a.lse[out_row] = s.l == 0.f ? -INFINITY : (s.m + log2f(s.l)) * kLn2;
      continue;
    }
    s.add<DP, 1>(a, first, parts, warp, 8, c4, local);
#pragma unroll
    for (int k = 0; k < 4; ++k) part_sum[warp][k][lane] = s.o[k];
    part_ml[warp][lane] = make_float2(s.m, s.l);
    __syncthreads();
    if (warp < 4 && local < rows) {              // warp k finishes float4 column c4 + k
      const int live = min(8, parts);
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < live; ++i) m = fmaxf(m, part_ml[i][lane].x);
      const float sub = m == -INFINITY ? 0.f : m;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = 0; i < live; ++i) {
        const float w = ex2(part_ml[i][lane].x - sub);
        const float4 x = part_sum[i][warp][lane];
        l = fmaf(part_ml[i][lane].y, w, l);
        y.x = fmaf(x.x, w, y.x);
        y.y = fmaf(x.y, w, y.y);
        y.z = fmaf(x.z, w, y.z);
        y.w = fmaf(x.w, w, y.w);
      }
      const int d = 4 * (c4 + warp);
      if (d < a.D) *reinterpret_cast<uint2*>(a.out + out_row * a.D + d) = join_pack<F16>(y, l);
      if (d == 0 && a.lse) a.lse[out_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
    __syncthreads();
  }
}

template <int DP>
constexpr size_t smem_bytes() {
  return Layout<DP>::kTail + sizeof(Tail);
}

template <bool F16, int HELD, int DP>
cudaError_t launch(const AttendArgs& a, const TileMaps& maps, cudaStream_t stream) {
  using R = Roles<HELD>;
  // either kernel is launched while the one before it ends (the join: runs), and waits
  // for it itself before anything else
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.n_cta);
  cfg.blockDim = dim3(R::kThreads);
  cfg.dynamicSmemBytes = smem_bytes<DP>();
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, attend_kernel<F16, HELD, DP, R::kLaunchRegs>, a, maps);
  if (e != cudaSuccess) return e;
  cfg.dynamicSmemBytes = 0;
  cfg.gridDim = dim3(2 * a.n_cta, kJoinSplit);
  cfg.blockDim = dim3(kJoinThreads);
  return cudaLaunchKernelEx(&cfg, join_kernel<F16, DP>, a);
}

template <bool F16, int HELD, int DP>
cudaError_t setup() {
  static_assert(smem_bytes<DP>() <= 232448, "shared memory of an SM");
  return cudaFuncSetAttribute(attend_kernel<F16, HELD, DP, Roles<HELD>::kLaunchRegs>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<DP>());
}

// The join keeps the main kernel's split of shared memory and L1: another would
// have the SMs drained and set up anew between the two.
template <bool F16, int DP>
cudaError_t setup_join() {
  return cudaFuncSetAttribute(join_kernel<F16, DP>, cudaFuncAttributePreferredSharedMemoryCarveout,
                              cudaSharedmemCarveoutMaxShared);
}

}  // namespace
}  // namespace tree
}  // namespace dspark
