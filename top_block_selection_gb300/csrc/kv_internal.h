// kv_internal.h - declarations shared by the paged caches' kernels and
// the C-ABI layer, and the device helpers of its e4m3 codes and scales.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "qsa_internal.h"

namespace qsa {

// The cache as the kernels see it (fields as in qsa_kv_cache).
struct KvCacheArgs {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  const int32_t* page_table;
  const int32_t* lens;
  const int32_t* n_new;
  int64_t page_stride;
  int32_t n_pages, max_blocks, B, Hkv, block, D;
  // The 4-bit cache's scales, one a token (k_scale and v_scale are null then).
  uint16_t* k_scale4 = nullptr;
  uint16_t* v_scale4 = nullptr;
};

// Rows [B, n, heads, D] of 16-bit floats, strides in elements.
struct KvRows {
  const void* data;
  int64_t sb, sn, sh;
};

struct KvAppendProblem {
  KvCacheArgs cache;
  KvRows k, v, q;  // q.data null: no queries
  int32_t n, Hq, rot, max_pos;
  bool bf16, interleaved;
  const float* cos;
  const float* sin;
  void* q_out;
  uint16_t* kb;
  const int32_t* offset = nullptr;  // 4-bit cache only
};
// CTAs of the append, of which *units each own a (block, head, K or V).
int64_t kv_append_grid(const KvAppendProblem& p, int64_t* units, int32_t* blocks_per_seq);
cudaError_t launch_kv_append(const KvAppendProblem& p, const DeviceInfo& dev, cudaStream_t stream);
int64_t kv4_append_grid(const KvAppendProblem& p, int64_t* units, int32_t* blocks_per_seq);
cudaError_t launch_kv4_append(const KvAppendProblem& p, const DeviceInfo& dev, cudaStream_t stream);
int64_t kv4_read_grid(const KvCacheArgs& c, int32_t n);
cudaError_t launch_kv4_read(const KvCacheArgs& c, int32_t n, bool bf16, void* k, void* v, const DeviceInfo& dev,
                            cudaStream_t stream);

struct KvAttendProblem {
  KvCacheArgs cache;
  KvRows q;
  int32_t n, Hq;
  bool bf16;
  float scale;
  const int32_t* ids;  // null: every block
  int32_t n_lists, k;
  void* out;
  float* lse;
  void* workspace;
};
// 0 for sizes the attention does not take.
size_t kv_attend_workspace_bytes(int32_t B, int32_t n, int32_t Hq, int32_t Hkv, int32_t D);
cudaError_t launch_kv_attend(const KvAttendProblem& p, const DeviceInfo& dev, cudaStream_t stream);
size_t kv4_attend_workspace_bytes(int32_t B, int32_t n, int32_t Hq, int32_t Hkv, int32_t D);
cudaError_t launch_kv4_attend(const KvAttendProblem& p, const DeviceInfo& dev, cudaStream_t stream);

struct Kv4WeightsProblem {
  KvCacheArgs cache;
  KvRows q;
  int32_t n, Hq;
  bool bf16;
  float scale, decay;
  const float* lse;
  float* weights;
};
cudaError_t launch_kv4_weights(const Kv4WeightsProblem& p, const DeviceInfo& dev, cudaStream_t stream);

struct Kv4EvictProblem {
  KvCacheArgs cache;
  float* weights;
  int32_t budget, sink, recent;
  int32_t* lens_out;
  int32_t* offset;
  int32_t* list;  // [B, Hkv, budget]: where the tokens of an item's slots come from
};
size_t kv4_evict_workspace_bytes(int32_t B, int32_t Hkv, int32_t budget);
cudaError_t launch_kv4_evict(const Kv4EvictProblem& p, const DeviceInfo& dev, cudaStream_t stream);

constexpr int kKvMaxGroup = 32;             // query heads per KV head
constexpr uint32_t kKvIndexBit = 1u << 5;   // kErrCacheIndex (qsa_device.cuh) for host code

#ifdef __CUDACC__
// Loads of what an earlier kernel on the stream may have written. These kernels
// start before that one has ended (programmatic dependent launch) and wait for
// it, so the read-only path, which takes memory to be constant over a kernel's
// life, is not for them.
__device__ __forceinline__ int32_t load_global(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float load_global(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t load_global(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 load_global(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 load_global(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ float4 load_global(const float4* p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// The new tokens of sequence b: the first n_new of its n rows, at positions
// first .. len - 1 (first < 0: those before position 0 do not exist).
struct Span {
  int32_t len, n_new, first;
};
__device__ __forceinline__ Span span_of(const KvCacheArgs& c, int b, int n) {
  Span s;
  s.len = load_global(c.lens + b);
  s.n_new = c.n_new ? min(max(load_global(c.n_new + b), 0), n) : n;
  s.len = max(s.len, 0);
  s.first = s.len - s.n_new;
  return s;
}

// Two floats to two e4m3 codes (lo in bits 0-7), to nearest even, finite
// overflow and infinities to +-448, NaN to NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The smallest power of two s >= 2^-100 with amax <= 448 s, 448 = 1.75 * 2^8
// (an infinite amax counts as the largest finite one).
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t u = __float_as_uint(fminf(amax, 3.402823466e38f));
  int e = static_cast<int>(u >> 23) - 127 - 8;
  if ((u & 0x7FFFFFu) > 0x600000u) ++e;
  return __uint_as_float(static_cast<uint32_t>(max(e, -100) + 127) << 23);
}
#endif

}  // namespace qsa
