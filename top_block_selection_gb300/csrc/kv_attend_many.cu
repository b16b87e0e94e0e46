// kv_attend_many.cu - launch of the cache attention of many rows.
#include "kv_attend_many.cuh"

namespace qsa {
namespace {

template <int D, bool BF16>
cudaError_t many_form(const AttendArgs& a, int grid, bool split, int device, cudaStream_t stream) {
  constexpr int smem = 1024 + 6 * kKvTile * D * 2 + static_cast<int>(sizeof(ManyShared<D>));
  static_assert(smem <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << device;
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(kv_attend_many_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  cudaError_t e = launch_pdl(kv_attend_many_kernel<D, BF16>, dim3(grid), dim3(kManyThreads), smem, stream, a);
  if (e != cudaSuccess) return e;
  plan_add("kv_attend_many_kernel");
  if (!split) return cudaSuccess;
  const int64_t items = static_cast<int64_t>(a.c.B) * a.n_qt * a.c.Hkv;
  // Few items have many parts each: more CTAs an item read them.
  constexpr int kRowGroups = 2 * kManyRows / 32;
  if (items * 4 < grid)
    e = launch_pdl(kv_combine_many_kernel<D, 2>, dim3(grid, D / (2 * kJoinWarps), kRowGroups), dim3(32 * kJoinWarps), 0,
                   stream, a);
  else
    e = launch_pdl(kv_combine_many_kernel<D, 8>, dim3(grid, D / (8 * kJoinWarps), kRowGroups), dim3(32 * kJoinWarps), 0,
                   stream, a);
  if (e == cudaSuccess) plan_add("kv_combine_many_kernel");
  return e;
}

}  // namespace

cudaError_t launch_attend_many(const AttendArgs& a, int grid, bool split, int device, cudaStream_t stream) {
  if (a.c.D == 64)
    return a.bf16 ? many_form<64, true>(a, grid, split, device, stream)
                  : many_form<64, false>(a, grid, split, device, stream);
  return a.bf16 ? many_form<128, true>(a, grid, split, device, stream)
                : many_form<128, false>(a, grid, split, device, stream);
}

}  // namespace qsa
