// tree_attend4.cu -- tree_attend.cuh over a cache of e2m1 codes.
#include "tree_attend.cuh"

namespace dspark {
namespace tree {
namespace {

template <bool F16, int DP>
cudaError_t launch_ready(const AttendArgs& a, uint32_t* ready, cudaStream_t stream) {
  if (!(*ready & kReadyMany)) {
    cudaError_t e = setup<F16, kE2M1, DP>();
    if (e == cudaSuccess) e = setup_join<F16, DP>();
    if (e != cudaSuccess) return e;
    *ready |= kReadyMany;
  }
  return launch<F16, kE2M1, DP>(a, TileMaps{}, stream);
}

}  // namespace

cudaError_t attend4_launch(const AttendArgs& a, bool f16, uint32_t* ready, cudaStream_t stream) {
  if (padded_dim(a.D) == 64)
    return f16 ? launch_ready<true, 64>(a, ready, stream) : launch_ready<false, 64>(a, ready, stream);
  return f16 ? launch_ready<true, 128>(a, ready, stream) : launch_ready<false, 128>(a, ready, stream);
}

}  // namespace tree
}  // namespace dspark
