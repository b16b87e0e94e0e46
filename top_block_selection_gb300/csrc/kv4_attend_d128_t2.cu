// kv4_attend_d128_t2.cu - the 4-bit cache's attention for heads of 128 dimensions
// in 2 terms (bf16 calls).
#include "kv_attend_kernel.cuh"

namespace qsa {
cudaError_t attend4_d128_t2(int rt, const CUtensorMap& tk, const CUtensorMap& tv, const AttendArgs& a, int grid,
                          int device, cudaStream_t stream) {
  return attend_rows<128, 2, true>(rt, tk, tv, a, grid, device, stream);
}
}  // namespace qsa
