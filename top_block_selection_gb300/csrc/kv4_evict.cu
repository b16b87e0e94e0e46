// kv4_evict.cu - shortening sequences of the paged 4-bit cache by what
// attention weight their tokens gathered.
//
// For each (sequence, KV head) with more than `budget` tokens: of the tokens
// between the first `sink` and the last `recent` the K = budget - sink - recent
// of the largest weights stay, found exactly: the K-th largest key (the float's
// bits, ordered) by three histograms of 11, 11 and 10 bits, and of the keys equal
// to it the lowest slots. Kept tokens move together in their order.
//
// One cluster of 1 to 16 CTAs an item: a CTA holds its part of the keys in shared
// memory, so that the weights are read once; histograms are added over
// distributed shared memory. The move is in place: a token never moves up, so a
// chunk's stores touch no later chunk's sources; within a chunk all CTAs load
// before any stores. What bounds it: bytes for many items; for few, the chain of
// a chunk's dependent loads (list, page, codes) and its cluster barrier.
#include <algorithm>
#include <atomic>

#include "kv_internal.h"
#include "qsa_device.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 512;
constexpr int kBins = 2048;
constexpr int kMaxKeys = 40960;  // of a CTA's part, in shared memory; those past it are read again in each pass
constexpr int kBatch = 8;        // keys of a thread whose loads are in flight together
constexpr int kPieces = 4;       // of 32 bytes, a thread's share of a chunk of the move

struct EvictArgs {
  KvCacheArgs c;
  float* weights;
  int32_t budget, sink, recent;
  int32_t* lens_out;
  int32_t* offset;
  int32_t* list;
  uint32_t* status;
  int32_t ctas, cap, block_log2;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint4 load_remote4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 load_remote2(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}

// 32 bytes, loaded and stored by one instruction.
struct Piece {
  uint64_t v[4];
};
__device__ __forceinline__ Piece load_piece(const void* p) {
  Piece x;
  asm volatile("ld.global.v4.u64 {%0, %1, %2, %3}, [%4];"
               : "=l"(x.v[0]), "=l"(x.v[1]), "=l"(x.v[2]), "=l"(x.v[3])
               : "l"(p)
               : "memory");
  return x;
}
__device__ __forceinline__ void store_piece(void* p, const Piece& x) {
  asm volatile("st.global.v4.u64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(x.v[0]), "l"(x.v[1]), "l"(x.v[2]), "l"(x.v[3])
               : "memory");
}

struct EvictShared {
  alignas(16) uint32_t hist[3][kBins];
  uint32_t warp[kThreads / 32];
  alignas(8) uint2 counts[kThreads / 32];  // above, equal
  alignas(8) uint2 total;
  uint32_t bin, above;
};

// The bin that holds the `need`-th largest key, and how many keys lie above it.
__device__ __forceinline__ void find_bin(EvictShared& s, int pass, int ctas, uint32_t need, uint32_t& bin, uint32_t& above) {
  const int tid = threadIdx.x, lane = tid % 32;
  uint32_t n[4] = {0, 0, 0, 0};
  for (int r = 0; r < ctas; ++r) {
    const uint4 v = load_remote4(remote(&s.hist[pass][kBins - 4 - 4 * tid], r));
    n[0] += v.w, n[1] += v.z, n[2] += v.y, n[3] += v.x;  // from the highest bin down
  }
  const uint32_t sum = n[0] + n[1] + n[2] + n[3];
  uint32_t before = sum;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, before, d);
    if (lane >= d) before += v;
  }
  if (lane == 31) s.warp[tid / 32] = before;
  __syncthreads();
  before -= sum;
  for (int w = 0; w < tid / 32; ++w) before += s.warp[w];
  if (before < need && need <= before + sum) {
    int i = 0;
    while (need > before + n[i]) before += n[i++];
    s.bin = kBins - 1 - 4 * tid - i;
    s.above = before;
  }
  __syncthreads();
  bin = s.bin;
  above = s.above;
}

__global__ void __launch_bounds__(kThreads, 2) kv4_evict_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint8_t raw[];
  EvictShared& s = *reinterpret_cast<EvictShared*>(raw);
  uint32_t* const keys = reinterpret_cast<uint32_t*>(raw + sizeof(EvictShared));
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  for (int i = tid; i < 3 * kBins; i += kThreads) s.hist[0][i] = 0;
  pdl_wait();
  pdl_launch_dependents();
  const int item = blockIdx.x / a.ctas, rank = blockIdx.x % a.ctas;
  const int b = item / a.c.Hkv, h = item - b * a.c.Hkv;
  const int capacity = a.c.max_blocks << a.block_log2, mask = a.c.block - 1;
  int len = max(load_global(a.c.lens + b), 0);
  bool bad = len > capacity;
  len = min(len, capacity);
  if (h == 0 && rank == 0 && tid == 0) {
    const int now = min(len, a.budget);
    a.lens_out[b] = now;
    if (a.offset) a.offset[b] += len - now;
  }
  if (len <= a.budget) {
    if (bad && tid == 0) atomicOr(a.status, kErrCacheIndex);
    return;
  }
  const int32_t* const table = a.c.page_table + static_cast<int64_t>(b) * a.c.max_blocks;
  // The page of a slot, -1: no such page; and the slot's row in scales and weights.
  // (Without branches, so that the loads of several go out together.)
  auto page_of = [&](int slot) -> int {
    const int page = load_global(table + (slot >> a.block_log2));
    const bool there = page >= 0 && page < a.c.n_pages;
    bad = bad || !there;
    return there ? page : -1;
  };
  auto row_in = [&](int page, int slot) {
    return ((static_cast<int64_t>(page) * a.c.Hkv + h) << a.block_log2) + (slot & mask);
  };
  auto row_of = [&](int slot) -> int64_t {
    const int page = page_of(slot);
    return page < 0 ? -1 : row_in(page, slot);
  };

  const int keep = a.budget - a.sink - a.recent;
  const int middle = len - a.recent - a.sink;
  const int part = (middle + a.ctas - 1) / a.ctas;
  const int first = a.sink + min(rank * part, middle), count = a.sink + min((rank + 1) * part, middle) - first;
  auto key_of = [](float w) { return isnan(w) ? 0xFFFFFFFFu : score_key(w); };
  auto fresh_key = [&](int i) -> uint32_t {
    const int64_t row = row_of(first + i);
    return key_of(row >= 0 ? load_global(a.weights + row) : 0.0f);
  };
  auto key = [&](int i) -> uint32_t { return i < a.cap ? keys[i] : fresh_key(i); };

  int32_t* const list = a.list + static_cast<int64_t>(item) * a.budget;
  if (keep > 0) {
    __syncthreads();  // the histograms are clear
    for (int i0 = tid; i0 < count; i0 += kBatch * kThreads) {
      int64_t row[kBatch];
      float w[kBatch];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) row[x] = i0 + x * kThreads < count ? row_of(first + i0 + x * kThreads) : -1;
#pragma unroll
      for (int x = 0; x < kBatch; ++x) w[x] = row[x] >= 0 ? load_global(a.weights + row[x]) : 0.0f;
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const int i = i0 + x * kThreads;
        if (i >= count) break;
        const uint32_t k = key_of(w[x]);
        if (i < a.cap) keys[i] = k;
        atomicAdd(&s.hist[0][k >> 21], 1u);
      }
    }
    uint32_t need = keep, prefix = 0, bin, above;
    cluster_sync();
    find_bin(s, 0, a.ctas, need, bin, above);
    need -= above;
    prefix = bin;
    for (int i = tid; i < count; i += kThreads) {
      const uint32_t k = key(i);
      if (k >> 21 == prefix) atomicAdd(&s.hist[1][(k >> 10) & 2047], 1u);
    }
    cluster_sync();
    find_bin(s, 1, a.ctas, need, bin, above);
    need -= above;
    prefix = prefix << 11 | bin;
    for (int i = tid; i < count; i += kThreads) {
      const uint32_t k = key(i);
      if (k >> 10 == prefix) atomicAdd(&s.hist[2][k & 1023], 1u);
    }
    cluster_sync();
    find_bin(s, 2, a.ctas, need, bin, above);
    need -= above;  // of the keys equal to the least one kept, so many stay
    const uint32_t least = prefix << 10 | bin;

    // Their places: each warp counts a contiguous run, then numbers it.
    const int run = ((count + kThreads - 1) / kThreads) * 32;
    const int from = min(warp * run, count), to = min(from + run, count);
    uint2 n = make_uint2(0, 0);
    for (int i = from; i < to; i += 32) {
      const uint32_t k = i + lane < to ? key(i + lane) : 0;
      n.x += __popc(__ballot_sync(0xFFFFFFFFu, i + lane < to && k > least));
      n.y += __popc(__ballot_sync(0xFFFFFFFFu, i + lane < to && k == least));
    }
    if (lane == 0) s.counts[warp] = n;
    __syncthreads();
    if (tid == 0) {
      uint2 t = make_uint2(0, 0);
      for (int w = 0; w < kThreads / 32; ++w) {
        const uint2 v = s.counts[w];
        s.counts[w] = t;
        t.x += v.x;
        t.y += v.y;
      }
      s.total = t;
    }
    cluster_sync();
    n = s.counts[warp];
    for (int r = 0; r < rank; ++r) {
      const uint2 v = load_remote2(remote(&s.total, r));
      n.x += v.x;
      n.y += v.y;
    }
    const uint32_t below = (1u << lane) - 1;
    for (int i = from; i < to; i += 32) {
      const uint32_t k = i + lane < to ? key(i + lane) : 0;
      const uint32_t more = __ballot_sync(0xFFFFFFFFu, i + lane < to && k > least);
      const uint32_t same = __ballot_sync(0xFFFFFFFFu, i + lane < to && k == least);
      const uint32_t equal = n.y + __popc(same & below);
      const uint32_t place = n.x + __popc(more & below) + min(equal, need);
      if ((more >> lane & 1) || ((same >> lane & 1) && equal < need)) list[a.sink + place] = first + i + lane;
      n.x += __popc(more);
      n.y += __popc(same);
    }
    cluster_sync();
  }

  // The move. A token's codes are `lanes` pieces, one to a lane: its key's first.
  const int lanes = a.c.D / 32, piece = tid % lanes, tokens = kThreads * kPieces / lanes;
  const int newest = a.budget - a.recent, shift = len - a.budget;
  uint8_t* const codes = (piece < lanes / 2 ? a.c.k : a.c.v) + piece % (lanes / 2) * 32;
  auto codes_at = [&](int page, int slot) {
    return codes + page * a.c.page_stride + ((h << a.block_log2) + (slot & mask)) * static_cast<int64_t>(a.c.D / 2);
  };
  // Beside its codes a lane moves the key's scale (the first lane), the value's
  // (the second) and the weight (the last).
  uint16_t* const scales = piece == 0 ? a.c.k_scale4 : a.c.v_scale4;
  for (int base = a.sink; base < a.budget; base += a.ctas * tokens) {
    const int mine = base + rank * tokens + tid / lanes;
    int src[kPieces], from[kPieces], to[kPieces];
    Piece data[kPieces];
    uint16_t scale[kPieces];
    float weight[kPieces];
#pragma unroll
    for (int r = 0; r < kPieces; ++r) {
      const int slot = mine + r * (kThreads / lanes);
      src[r] = slot >= a.budget ? slot : slot >= newest ? slot + shift : __ldcg(list + slot);
    }
#pragma unroll
    for (int r = 0; r < kPieces; ++r) {
      const int slot = mine + r * (kThreads / lanes);
      from[r] = to[r] = -1;
      if (src[r] != slot) {
        from[r] = page_of(src[r]);
        to[r] = page_of(slot);
      }
    }
#pragma unroll
    for (int r = 0; r < kPieces; ++r)
      if (from[r] >= 0 && to[r] >= 0) {
        data[r] = load_piece(codes_at(from[r], src[r]));
        const int64_t row = row_in(from[r], src[r]);
        if (piece < 2) scale[r] = scales[row];
        if (piece == lanes - 1) weight[r] = load_global(a.weights + row);
      }
    cluster_sync();
#pragma unroll
    for (int r = 0; r < kPieces; ++r)
      if (from[r] >= 0 && to[r] >= 0) {
        const int slot = mine + r * (kThreads / lanes);
        store_piece(codes_at(to[r], slot), data[r]);
        const int64_t row = row_in(to[r], slot);
        if (piece < 2) scales[row] = scale[r];
        if (piece == lanes - 1) a.weights[row] = weight[r];
      }
  }
  if (bad) atomicOr(a.status, kErrCacheIndex);
  // An attention next on the stream may start early and reads codes by bulk copies.
  fence_proxy_async_global();
}

}  // namespace

size_t kv4_evict_workspace_bytes(int32_t B, int32_t Hkv, int32_t budget) {
  if (B < 0 || Hkv < 1 || budget < 1) return 0;
  return sizeof(int32_t) * static_cast<size_t>(B) * Hkv * budget;
}

cudaError_t launch_kv4_evict(const Kv4EvictProblem& p, const DeviceInfo& dev, cudaStream_t stream) {
  EvictArgs a{};
  a.c = p.cache;
  a.weights = p.weights;
  a.budget = p.budget;
  a.sink = p.sink;
  a.recent = p.recent;
  a.lens_out = p.lens_out;
  a.offset = p.offset;
  a.list = p.list;
  a.status = dev.status_word;
  while ((1 << a.block_log2) < p.cache.block) ++a.block_log2;
  // As many CTAs an item as the GPU holds at two an SM, each with 1,024 tokens or
  // more of the longest sequence there can be.
  const int64_t items = static_cast<int64_t>(p.cache.B) * p.cache.Hkv;
  const int64_t longest = static_cast<int64_t>(p.cache.max_blocks) * p.cache.block;
  a.ctas = 16;
  while (a.ctas > 1 && (items * a.ctas > 2 * dev.sm_count || longest < 1024 * a.ctas)) a.ctas /= 2;
  a.cap = static_cast<int32_t>(std::min<int64_t>((longest + a.ctas - 1) / a.ctas, kMaxKeys));
  const size_t smem = sizeof(EvictShared) + sizeof(uint32_t) * a.cap;
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << dev.id;
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kv4_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(sizeof(EvictShared) + sizeof(uint32_t) * kMaxKeys));
    if (e != cudaSuccess) return e;
    const cudaError_t e2 = cudaFuncSetAttribute(kv4_evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e2 != cudaSuccess) return e2;
    ready.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items * a.ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(a.ctas), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_evict_kernel, a);
  if (e == cudaSuccess) plan_add("kv4_evict_kernel");
  return e;
}

}  // namespace qsa
