// tree_attend_few4_128_32.cu -- tree_attend_few4.cuh for heads of up to 128 elements and items of
// 32 rows.
#include "tree_attend_few4.cuh"

namespace dspark {
namespace tree {

template <>
cudaError_t few4_launch_of<128, 4>(const AttendArgs& a, bool alone, bool runs, uint32_t* ready, cudaStream_t stream) {
  return launch_all<128, 4, 8>(a, alone, runs, ready, stream);
}

}  // namespace tree
}  // namespace dspark
