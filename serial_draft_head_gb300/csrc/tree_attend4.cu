// tree_attend4.cu -- tree_attend.cuh over a cache of e2m1 codes.
#include "tree_attend.cuh"

namespace dspark {
namespace tree {
namespace {

template <bool F16, int DP>
cudaError_t setup_both() {
  const cudaError_t e = setup<F16, kE2M1, DP>();
  return e == cudaSuccess ? setup_join<F16, DP>() : e;
}

}  // namespace

cudaError_t attend4_setup(bool f16, int D) {
  if (padded_dim(D) == 64) return f16 ? setup_both<true, 64>() : setup_both<false, 64>();
  return f16 ? setup_both<true, 128>() : setup_both<false, 128>();
}

cudaError_t attend4_launch(const AttendArgs& a, bool f16, cudaStream_t stream) {
  TileMaps maps{};
  if (padded_dim(a.D) == 64)
    return f16 ? launch<true, kE2M1, 64>(a, maps, stream) : launch<false, kE2M1, 64>(a, maps, stream);
  return f16 ? launch<true, kE2M1, 128>(a, maps, stream) : launch<false, kE2M1, 128>(a, maps, stream);
}

}  // namespace tree
}  // namespace dspark
