// tree_attend_few4.cu -- the choice among the forms of tree_attend_few4.cuh.
#include "tree_attend_few4.cuh"

namespace dspark {
namespace tree {

template <>
cudaError_t few4_launch_of<64, 1>(const AttendArgs& a, bool alone, bool runs, uint32_t* ready,
                                   cudaStream_t stream);
template <>
cudaError_t few4_launch_of<64, 2>(const AttendArgs& a, bool alone, bool runs, uint32_t* ready,
                                   cudaStream_t stream);
template <>
cudaError_t few4_launch_of<64, 4>(const AttendArgs& a, bool alone, bool runs, uint32_t* ready,
                                   cudaStream_t stream);
template <>
cudaError_t few4_launch_of<128, 1>(const AttendArgs& a, bool alone, bool runs, uint32_t* ready,
                                   cudaStream_t stream);
template <>
cudaError_t few4_launch_of<128, 2>(const AttendArgs& a, bool alone, bool runs, uint32_t* ready,
                                   cudaStream_t stream);
template <>
cudaError_t few4_launch_of<128, 4>(const AttendArgs& a, bool alone, bool runs, uint32_t* ready,
                                   cudaStream_t stream);

namespace {

// Whether a page holds each head's slots, and their scales, next to each other, in pieces
// that 16-byte copies take.
bool in_runs(const AttendArgs& a) {
  if (a.c.page.d % 16 != 0 || a.D % 64 != 0) return false;
  for (int v = 0; v < 2; ++v) {
    const Rows &x = a.c.x[v], &s = a.c.scale[v];
    if (x.slot != (uint32_t)a.D / 2 || s.slot != (uint32_t)a.D / 16) return false;
    if ((reinterpret_cast<uintptr_t>(s.p) | (uint64_t)s.head | s.page) % 16 != 0) return false;
  }
  return true;
}

template <int DP>
cudaError_t launch_for(const AttendArgs& a, int tiles, bool alone, bool runs, uint32_t* ready,
                       cudaStream_t stream) {
  if (tiles == 1) return few4_launch_of<DP, 1>(a, alone, runs, ready, stream);
  return tiles == 2 ? few4_launch_of<DP, 2>(a, alone, runs, ready, stream)
                    : few4_launch_of<DP, 4>(a, alone, runs, ready, stream);
}

}  // namespace

cudaError_t few4_launch(const AttendArgs& a, uint32_t* ready, cudaStream_t stream) {
  // rows of an item: what the requests have on average, in whole tiles of eight
  const int64_t rows = (int64_t)a.b.N * a.G;
  const int tiles = rows <= (int64_t)8 * a.b.B ? 1 : rows <= (int64_t)16 * a.b.B ? 2 : 4;
  // Workers of four warps where there are two items a SM (64 heads on 8, 500 to 9,000
  // tokens, us with four / with a CTA's: 48 requests 69 / 87, 128 146 / 195; 16 requests 36 /
  // 35, 1 of 5,000 28 / 14, 19 of 32,767 135 / 128).  Items of 16 and 32 rows (32 heads on 8):
  // 128 requests of 100 to 300 tokens 46 / 55 and 81 / 90, of 300 to 6,000 272 / 269 and 400 / 381,
  // with heads of 64 elements 107 / 124 and 200 / 205; the lengths are not known here.
  const int64_t items = (rows + 8 * tiles - 1) / (8 * tiles) * a.Hkv;
  const bool alone = items < (int64_t)2 * a.n_cta;
  const bool runs = in_runs(a);
  return padded_dim(a.D) == 64 ? launch_for<64>(a, tiles, alone, runs, ready, stream)
                               : launch_for<128>(a, tiles, alone, runs, ready, stream);
}

}  // namespace tree
}  // namespace dspark
