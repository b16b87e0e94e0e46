// kv4_attend_d64_t3.cu - the 4-bit cache's attention for heads of 64 dimensions
// in 3 terms (fp16 calls).
#include "kv_attend_kernel.cuh"

namespace qsa {
cudaError_t attend4_d64_t3(int rt, const CUtensorMap& tk, const CUtensorMap& tv, const AttendArgs& a, int grid,
                          int device, cudaStream_t stream) {
  return attend_rows<64, 3, true>(rt, tk, tv, a, grid, device, stream);
}
}  // namespace qsa
