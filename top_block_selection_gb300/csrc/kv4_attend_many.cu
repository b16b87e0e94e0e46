// kv4_attend_many.cu - launch of the 4-bit cache's attention of many rows.
#include "kv_attend_many.cuh"

namespace qsa {

cudaError_t launch_attend4_many(const AttendArgs& a, int grid, bool split, int device, cudaStream_t stream) {
  return launch_many<true>(a, grid, split, device, stream);
}

}  // namespace qsa
