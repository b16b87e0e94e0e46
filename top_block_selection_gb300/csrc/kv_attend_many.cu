// kv_attend_many.cu - launch of the 8-bit cache's attention of many rows.
#include "kv_attend_many.cuh"

namespace qsa {

cudaError_t launch_attend_many(const AttendArgs& a, int grid, bool split, int device, cudaStream_t stream) {
  return launch_many<false>(a, grid, split, device, stream);
}

}  // namespace qsa
