// kv_attend_d64.cu - the cache attention for heads of 64 dimensions.
#include "kv_attend_kernel.cuh"

namespace qsa {
cudaError_t attend_rows_d64(int rt, const CUtensorMap& tk, const CUtensorMap& tv, const AttendArgs& a, int grid,
                            bool init, cudaStream_t stream) {
  return attend_rows<64>(rt, tk, tv, a, grid, init, stream);
}
}  // namespace qsa
