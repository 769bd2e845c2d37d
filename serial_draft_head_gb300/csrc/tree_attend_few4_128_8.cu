// tree_attend_few4_128_8.cu -- tree_attend_few4.cuh for heads of up to 128 elements and items of
// 8 rows.
#include "tree_attend_few4.cuh"

namespace dspark {
namespace tree {

template <>
cudaError_t few4_launch_of<128, 1>(const AttendArgs& a, bool alone, bool runs, uint32_t* ready, cudaStream_t stream) {
  return launch_all<128, 1, 16>(a, alone, runs, ready, stream);
}

}  // namespace tree
}  // namespace dspark
