// tree_attend.cu -- tree_attend.cuh over caches of 16 bits and of e4m3 codes.
#include "tree_attend.cuh"

namespace dspark {
namespace tree {
namespace {

template <bool F16, int DP>
cudaError_t setup_both() {
  cudaError_t e = setup<F16, k16, DP>();
  if (e == cudaSuccess) e = setup<F16, kE4M3, DP>();
  return e == cudaSuccess ? setup_join<F16, DP>() : e;
}

}  // namespace

cudaError_t attend_setup(bool f16, int D) {
  if (padded_dim(D) == 64) return f16 ? setup_both<true, 64>() : setup_both<false, 64>();
  return f16 ? setup_both<true, 128>() : setup_both<false, 128>();
}

cudaError_t attend_launch(const AttendArgs& a, const TileMaps& maps, bool f16, bool e4m3,
                          cudaStream_t stream) {
  const int sel = (f16 ? 4 : 0) + (e4m3 ? 2 : 0) + (padded_dim(a.D) == 128 ? 1 : 0);
  switch (sel) {
    case 0: return launch<false, k16, 64>(a, maps, stream);
    case 1: return launch<false, k16, 128>(a, maps, stream);
    case 2: return launch<false, kE4M3, 64>(a, maps, stream);
    case 3: return launch<false, kE4M3, 128>(a, maps, stream);
    case 4: return launch<true, k16, 64>(a, maps, stream);
    case 5: return launch<true, k16, 128>(a, maps, stream);
    case 6: return launch<true, kE4M3, 64>(a, maps, stream);
    default: return launch<true, kE4M3, 128>(a, maps, stream);
  }
}

}  // namespace tree
}  // namespace dspark
