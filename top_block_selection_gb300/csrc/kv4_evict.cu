// kv4_evict.cu - shortening sequences of the paged 4-bit cache by what
// attention weight their tokens gathered.
//
// For each (sequence, KV head) with more than `budget` tokens: of the tokens
// between the first `sink` and the last `recent` the K = budget - sink - recent
// of the largest weights stay, found exactly: the K-th largest key (the float's
// bits, ordered) by three histograms of 11, 11 and 10 bits, and of the keys equal
// to it the lowest slots. Kept tokens move together in their order.
//
// One cluster of 1 to 8 CTAs an item: a CTA holds its part of the keys in shared
// memory, so that the weights are read once; histograms are added over
// distributed shared memory. The move is in place: a token never moves up, so a
// chunk's stores touch no later chunk's sources; within a chunk all CTAs load
// before any stores, until the chunks come from beyond the budget altogether.
//
// What bounds it: bytes for many items (64 sequences of 4,160 tokens to 4,096, 8 heads,
// with weights that no eviction has seen: 118 us, 72% of a plain copy's rate); for few,
// the chain of a chunk's dependent loads (list, page, codes), its cluster barrier and the
// three histograms' (8 heads of 131,072 tokens to 32,768: 50 us, 1.5 TB/s). The same
// sequences shortened over and over take 86 and 38.8 us, the basis of the figures below:
// fewer tokens change their place then, and those lie side by side.
#include <algorithm>
#include <atomic>

#include "kv_internal.h"
#include "qsa_device.cuh"

namespace qsa {
namespace {

constexpr int kBins = 2048, kCoarse = 64, kFine = kBins / kCoarse;
// CTAs of an item at most. (16 are a cluster that few GPCs take beside another: 8
// heads of 131,072 tokens 84 us instead of 71.)
constexpr int kMaxCluster = 8;
constexpr int kMaxKeys = 40960;  // of a CTA's part, in shared memory; those past it are read again in each pass
constexpr int kBatch = 8;        // keys of a thread side by side
constexpr int kQuads = 4;        // loads of four weights of a thread in flight together

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

template <int CLUSTER>
__device__ __forceinline__ void cluster_sync() {
  if (CLUSTER == 1) __syncthreads();
  else asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t load_remote(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
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
  alignas(8) uint32_t coarse[3][kCoarse];  // sums of kBins / kCoarse bins
  alignas(8) uint2 counts[32];  // above, equal
  alignas(8) uint2 total;
  uint32_t bin, above;
};

// The sums of runs of bins, once a CTA's histogram is there; then the cluster's barrier.
template <int THREADS, int CLUSTER>
__device__ __forceinline__ void publish(EvictShared& s, int pass) {
  constexpr int kPer = kBins / THREADS;
  static_assert(kPer % 4 == 0 && kFine % kPer == 0, "bins of a thread");
  __syncthreads();
  uint32_t n = 0;
#pragma unroll
  for (int i = 0; i < kPer; i += 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(&s.hist[pass][kPer * threadIdx.x + i]);
    n += (v.x + v.y) + (v.z + v.w);
  }
#pragma unroll
  for (int d = 1; d < kFine / kPer; d *= 2) n += __shfl_xor_sync(0xFFFFFFFFu, n, d);
  if (threadIdx.x % (kFine / kPer) == 0) s.coarse[pass][threadIdx.x / (kFine / kPer)] = n;
  cluster_sync<CLUSTER>();
}

// Of counts n held by the lanes, the higher lanes' first: the lane where the
// `need`-th is, and how many come before it.
__device__ __forceinline__ int lane_of_rank(uint32_t n, uint32_t need, uint32_t& before) {
  const int lane = threadIdx.x % 32;
  uint32_t sum = n;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t v = __shfl_down_sync(0xFFFFFFFFu, sum, d);
    if (lane + d < 32) sum += v;
  }
  const uint32_t at = __ballot_sync(0xFFFFFFFFu, sum >= need);  // the lanes up to the one sought
  const int found = 31 - __clz(at);
  before = __shfl_sync(0xFFFFFFFFu, sum - n, found);
  return found;
}

// The bin that holds the `need`-th largest key, and how many keys lie above it:
// a warp adds up the CTAs' sums of runs, then the bins of one run. (All bins of 16
// CTAs were 128 KB to read for each of them, 8,000 cycles.)
template <int CLUSTER>
__device__ __forceinline__ void find_bin(EvictShared& s, int pass, int ctas, uint32_t need, uint32_t& bin, uint32_t& above) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    uint2 v[CLUSTER];
    uint32_t u[CLUSTER];
#pragma unroll
    for (int r = 0; r < CLUSTER; ++r)
      v[r] = r < ctas ? load_remote2(remote(&s.coarse[pass][2 * lane], r)) : make_uint2(0, 0);
    uint2 n = make_uint2(0, 0);
#pragma unroll
    for (int r = 0; r < CLUSTER; ++r) {
      n.x += v[r].x;
      n.y += v[r].y;
    }
    uint32_t before;
    const int at = lane_of_rank(n.x + n.y, need, before);
    const uint32_t high = __shfl_sync(0xFFFFFFFFu, n.y, at);
    const bool low = need > before + high;
    if (low) before += high;
    const int run = 2 * at + (low ? 0 : 1);
#pragma unroll
    for (int r = 0; r < CLUSTER; ++r)
      u[r] = r < ctas ? load_remote(remote(&s.hist[pass][run * kFine + lane], r)) : 0;
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < CLUSTER; ++r) m += u[r];
    uint32_t more;
    const int in_run = lane_of_rank(m, need - before, more);
    if (lane == 0) {
      s.bin = run * kFine + in_run;
      s.above = before + more;
    }
  }
  __syncthreads();
  bin = s.bin;
  above = s.above;
}

// PIECES of 32 bytes are a thread's share of a chunk of the move.
template <int THREADS, int PIECES, int CTAS_PER_SM, int CLUSTER>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM) kv4_evict_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint8_t raw[];
  EvictShared& s = *reinterpret_cast<EvictShared*>(raw);
  uint32_t* const keys = reinterpret_cast<uint32_t*>(raw + sizeof(EvictShared));
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  for (int i = tid; i < 3 * kBins; i += THREADS) s.hist[0][i] = 0;
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
  const bool resident = count <= a.cap;
  // Keys i, i + step, .. of n (0 past the CTA's), from shared memory or, of a part
  // too long for it, from global memory again.
  auto keys_at = [&](int i, int step, auto& k) {
    constexpr int n = sizeof(k) / sizeof(k[0]);
    if (resident) {
#pragma unroll
      for (int x = 0; x < n; ++x) k[x] = i + x * step < count ? keys[i + x * step] : 0;
    } else {
#pragma unroll 1
      for (int x = 0; x < n; ++x) {
        const int j = i + x * step;
        const uint32_t v = j >= count ? 0 : j < a.cap ? keys[j] : fresh_key(j);
#pragma unroll
        for (int y = 0; y < n; ++y)
          if (y == x) k[y] = v;
      }
    }
  };
  // Counts the keys whose bits above `shift + bits` are `prefix` by the next `bits`.
  auto count_bins = [&](uint32_t* hist, int shift, int bits, uint32_t prefix) {
    for (int i = tid; i < count; i += kBatch * THREADS) {
      uint32_t k[kBatch];
      keys_at(i, THREADS, k);
#pragma unroll
      for (int x = 0; x < kBatch; ++x)
        if (i + x * THREADS < count && k[x] >> (shift + bits) == prefix)
          atomicAdd(&hist[(k[x] >> shift) & ((1u << bits) - 1)], 1u);
    }
  };

  int32_t* const list = a.list + static_cast<int64_t>(item) * a.budget;  // (there is one: the budget is below some length)
  if (keep > 0) {
    __syncthreads();  // the histograms are clear
    // Four slots a load, the first aligned; four such loads of a thread together.
    const int lead = first & 3;
    for (int j0 = tid; 4 * j0 < count + lead; j0 += kQuads * THREADS) {
      int page[kQuads];
      float4 w[kQuads];
#pragma unroll
      for (int x = 0; x < kQuads; ++x) {
        const int i = 4 * (j0 + x * THREADS) - lead;
        page[x] = i < count ? page_of(first + i) : -1;
      }
#pragma unroll
      for (int x = 0; x < kQuads; ++x) {
        w[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (page[x] >= 0)
          w[x] = load_global(reinterpret_cast<const float4*>(
              a.weights + row_in(page[x], first + 4 * (j0 + x * THREADS) - lead)));
      }
#pragma unroll
      for (int x = 0; x < kQuads; ++x) {
        const float each[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 4 * (j0 + x * THREADS) - lead + e;
          if (i < 0 || i >= count) continue;
          const uint32_t k = key_of(each[e]);
          if (i < a.cap) keys[i] = k;
          atomicAdd(&s.hist[0][k >> 21], 1u);
        }
      }
    }
    uint32_t need = keep, prefix, bin, above;
    publish<THREADS, CLUSTER>(s, 0);
    find_bin<CLUSTER>(s, 0, a.ctas, need, bin, above);
    need -= above;
    prefix = bin;
    count_bins(s.hist[1], 10, 11, prefix);
    publish<THREADS, CLUSTER>(s, 1);
    find_bin<CLUSTER>(s, 1, a.ctas, need, bin, above);
    need -= above;
    prefix = prefix << 11 | bin;
    count_bins(s.hist[2], 0, 10, prefix);
    publish<THREADS, CLUSTER>(s, 2);
    find_bin<CLUSTER>(s, 2, a.ctas, need, bin, above);
    need -= above;  // of the keys equal to the least one kept, so many stay
    const uint32_t least = prefix << 10 | bin;

    // Their places: each warp counts a contiguous run, then numbers it.
    constexpr int kSteps = 4;  // of 32 keys, side by side
    const int run = ((count + THREADS * kSteps - 1) / (THREADS * kSteps)) * 32 * kSteps;
    const int from = min(warp * run, count), to = min(from + run, count);
    uint2 n = make_uint2(0, 0);
    for (int i = from; i < to; i += 32 * kSteps) {
      uint32_t k[kSteps];
      keys_at(i + lane, 32, k);
#pragma unroll
      for (int x = 0; x < kSteps; ++x) {
        const bool in = i + 32 * x + lane < to;
        n.x += __popc(__ballot_sync(0xFFFFFFFFu, in && k[x] > least));
        n.y += __popc(__ballot_sync(0xFFFFFFFFu, in && k[x] == least));
      }
    }
    if (lane == 0) s.counts[warp] = n;
    __syncthreads();
    if (tid == 0) {
      uint2 t = make_uint2(0, 0);
      for (int w = 0; w < THREADS / 32; ++w) {
        const uint2 v = s.counts[w];
        s.counts[w] = t;
        t.x += v.x;
        t.y += v.y;
      }
      s.total = t;
    }
    cluster_sync<CLUSTER>();
    // What the CTAs before this one have: a lane each.
    n = lane < rank ? load_remote2(remote(&s.total, lane)) : make_uint2(0, 0);
    n.x = __reduce_add_sync(0xFFFFFFFFu, n.x) + s.counts[warp].x;
    n.y = __reduce_add_sync(0xFFFFFFFFu, n.y) + s.counts[warp].y;
    const uint32_t below = (1u << lane) - 1;
    for (int i = from; i < to; i += 32 * kSteps) {
      uint32_t k[kSteps];
      keys_at(i + lane, 32, k);
#pragma unroll
      for (int x = 0; x < kSteps; ++x) {
        const int at = i + 32 * x + lane;
        const uint32_t more = __ballot_sync(0xFFFFFFFFu, at < to && k[x] > least);
        const uint32_t same = __ballot_sync(0xFFFFFFFFu, at < to && k[x] == least);
        const uint32_t equal = n.y + __popc(same & below);
        const uint32_t place = n.x + __popc(more & below) + min(equal, need);
        if ((more >> lane & 1) || ((same >> lane & 1) && equal < need)) list[a.sink + place] = first + at;
        n.x += __popc(more);
        n.y += __popc(same);
      }
    }
    cluster_sync<CLUSTER>();
  }

  // The move. A token's codes are `lanes` pieces, one to a lane: its key's first.
  const int lanes = a.c.D / 32, piece = tid % lanes, tokens = THREADS * PIECES / lanes;
  const int newest = a.budget - a.recent, shift = len - a.budget;
  uint8_t* const codes = (piece < lanes / 2 ? a.c.k : a.c.v) + piece % (lanes / 2) * 32;
  auto codes_at = [&](int page, int slot) {
    return codes + page * a.c.page_stride + ((h << a.block_log2) + (slot & mask)) * static_cast<int64_t>(a.c.D / 2);
  };
  // Beside its codes a lane moves the key's scale (the first lane), the value's
  // (the second) and the weight (the last).
  uint16_t* const scales = piece == 0 ? a.c.k_scale4 : a.c.v_scale4;
  int src[PIECES], from[PIECES];
  auto look_up = [&](int mine) {  // where the pieces of a chunk come from
#pragma unroll
    for (int r = 0; r < PIECES; ++r) {
      const int slot = mine + r * (THREADS / lanes);
      src[r] = slot >= a.budget ? slot : slot >= newest ? slot + shift : __ldcg(list + slot);
    }
#pragma unroll
    for (int r = 0; r < PIECES; ++r) from[r] = src[r] != mine + r * (THREADS / lanes) ? page_of(src[r]) : -1;
  };
  int mine = a.sink + rank * tokens + tid / lanes;
  look_up(mine);
  for (int base = a.sink; base < a.budget; base += a.ctas * tokens) {
    Piece data[PIECES];
    uint16_t scale[PIECES];
    float weight[PIECES];
    uint32_t moves = 0;
#pragma unroll
    for (int r = 0; r < PIECES; ++r) {
      if (from[r] < 0) continue;
      moves |= 1u << r;
      data[r] = load_piece(codes_at(from[r], src[r]));
      const int64_t row = row_in(from[r], src[r]);
      if (piece < 2) scale[r] = scales[row];
      if (piece == lanes - 1) weight[r] = load_global(a.weights + row);
    }
    const int now = mine;
    mine += a.ctas * tokens;
    // Tokens from beyond the budget lie where nothing is stored. Once a chunk begins
    // with one (all later ones come from further up), what it overwrites has been
    // loaded: the chunks before it waited for that.
    const int begins_at = base >= newest ? base + shift : __ldcg(list + base);
    if (base + a.ctas * tokens < a.budget) look_up(mine);
    if (begins_at < a.budget) cluster_sync<CLUSTER>();
#pragma unroll
    for (int r = 0; r < PIECES; ++r) {
      if (!(moves >> r & 1)) continue;
      const int slot = now + r * (THREADS / lanes), to = page_of(slot);
      if (to < 0) continue;
      store_piece(codes_at(to, slot), data[r]);
      const int64_t row = row_in(to, slot);
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

namespace {

template <int THREADS, int PIECES, int CTAS_PER_SM, int CLUSTER>
cudaError_t evict_form(const EvictArgs& a, int64_t items, int device, cudaStream_t stream) {
  const auto kernel = kv4_evict_kernel<THREADS, PIECES, CTAS_PER_SM, CLUSTER>;
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << device;
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(sizeof(EvictShared) + sizeof(uint32_t) * kMaxKeys));
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items * a.ctas));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = sizeof(EvictShared) + sizeof(uint32_t) * a.cap;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(a.ctas), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e == cudaSuccess) plan_add("kv4_evict_kernel");
  return e;
}

}  // namespace

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
  a.ctas = kMaxCluster;
  while (a.ctas > 1 && (items * a.ctas > 2 * dev.sm_count || longest < 1024 * a.ctas)) a.ctas /= 2;
  // (Keys by the table's room: past some 22,500 tokens a CTA of the first form has no
  // other beside it on its SM. The 64 sequences of 4,160 tokens take 118 us with tables
  // of that length, 129 with room for 16,384 tokens, 175 for 32,832, 185 for 131,072.)
  a.cap = static_cast<int32_t>(std::min<int64_t>((longest + a.ctas - 1) / a.ctas, kMaxKeys));
  // Many items: small CTAs, two an SM, whose phases overlap (64 x 8 items of 4,160
  // tokens 120 us; four an SM with half the pieces 159, one of 512 threads 138). Few:
  // clusters, of large CTAs where half of the SMs stay idle all the same (8 items of
  // 131,072 tokens 54 us, 72 with small ones; 16 items 107 and 97, 64 of 32,768 103
  // and 87). (A second kernel on all SMs for the tokens from beyond the budget, about
  // 5 us of work there, cost more than it saved: 46 us instead of 42 for 8 items in a
  // stream of calls, 69 instead of 61 for 64.)
  if (a.ctas == 1) return evict_form<256, 8, 2, 1>(a, items, dev.id, stream);
  if (items * a.ctas <= dev.sm_count / 2) return evict_form<512, 8, 1, kMaxCluster>(a, items, dev.id, stream);
  return evict_form<256, 8, 2, kMaxCluster>(a, items, dev.id, stream);
}

}  // namespace qsa
