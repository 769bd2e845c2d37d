// tree_attend_few4_128.cu -- tree_attend_few4.cuh for heads of more than 64 elements.
#include "tree_attend_few4.cuh"

namespace dspark {
namespace tree {

cudaError_t few4_setup128() {
  cudaError_t e = setup<128, 1, 16, false, false>();
  if (e == cudaSuccess) e = setup<128, 1, 16, false, true>();
  if (e == cudaSuccess) e = setup<128, 1, 16, true, false>();
  if (e == cudaSuccess) e = setup<128, 1, 16, true, true>();
  if (e == cudaSuccess) e = setup<128, 1, 4, true, false>();
  if (e == cudaSuccess) e = setup<128, 2, 12, false, false>();
  if (e == cudaSuccess) e = setup<128, 2, 12, false, true>();
  if (e == cudaSuccess) e = setup<128, 2, 12, true, false>();
  if (e == cudaSuccess) e = setup<128, 2, 12, true, true>();
  if (e == cudaSuccess) e = setup<128, 2, 4, true, false>();
  return e;
}

cudaError_t few4_launch128(const AttendArgs& a, bool two, bool alone, bool runs, cudaStream_t stream) {
  const bool cap = a.softcap > 0.f;
  if (!runs) {
    if (two) return cap ? launch<128, 2, 12, false, true>(a, stream) : launch<128, 2, 12, false, false>(a, stream);
    return cap ? launch<128, 1, 16, false, true>(a, stream) : launch<128, 1, 16, false, false>(a, stream);
  }
  if (two) {
    if (cap) return launch<128, 2, 12, true, true>(a, stream);
    return alone ? launch<128, 2, 12, true, false>(a, stream) : launch<128, 2, 4, true, false>(a, stream);
  }
  if (cap) return launch<128, 1, 16, true, true>(a, stream);
  return alone ? launch<128, 1, 16, true, false>(a, stream) : launch<128, 1, 4, true, false>(a, stream);
}

}  // namespace tree
}  // namespace dspark
