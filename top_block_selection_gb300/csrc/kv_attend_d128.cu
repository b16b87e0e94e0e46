// kv_attend_d128.cu - the cache attention for heads of 128 dimensions.
#include "kv_attend_kernel.cuh"

namespace qsa {
cudaError_t attend_rows_d128(int rt, const CUtensorMap& tk, const CUtensorMap& tv, const AttendArgs& a, int grid,
                            bool init, cudaStream_t stream) {
  return attend_rows<128>(rt, tk, tv, a, grid, init, stream);
}
}  // namespace qsa
