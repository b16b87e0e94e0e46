// kv_attend.cu - launcher of the cache attention, and the kernel that joins
// the partial results of items that were split over several CTAs.
#include "kv_attend_many.cuh"

#include <algorithm>

namespace qsa {
namespace {

constexpr int kCombineRows = 4;  // rows of a CTA, 128 threads each
// What an item costs beside its tiles, in tiles: a batch of 32 requests of 100
// tokens and 32 of 16,384 takes 168 us instead of 484 at 0, 256 requests of 64 to
// 829 tokens 50 us instead of 114, 64 requests of 1,000 to 16,384 tokens 175 at
// both (at 3 the first two take 165 and 57, at 8 169 and 50; taken when
// references only rose, the second is 54 us since).
constexpr int kItemCost = 5;

// Joins the parts of the item that CTA blockIdx.x of the attention began and
// others ended: that CTA's second slot and the first slots of the CTAs after
// it, added in order. A CTA a row would be up to 4,900 CTAs, nearly all with
// nothing to do, and their launch longer than the work: one token over 1,000
// tokens took 10.8 us instead of 9.7. The sums are fp32 and the parts added in
// the order of the tokens, so a call repeats its bits. It is bound by its
// launch and two dependent loads: about 2 us.
__global__ void __launch_bounds__(128 * kCombineRows) kv_combine_kernel(const __grid_constant__ AttendArgs a) {
  __shared__ float s_f[kCombineRows][kKvMaxCtas];
  __shared__ float s_max[kCombineRows][4], s_sum[kCombineRows][4];
  pdl_wait();
  pdl_launch_dependents();  // after the wait: at most one kernel ahead of the one that runs
  const int group = threadIdx.x / 128, tid = threadIdx.x % 128, rows = a.qt * a.R, D = a.c.D;
  const int c0 = blockIdx.x, r = blockIdx.y * kCombineRows + group;
  const int4 job = *reinterpret_cast<const int4*>(a.jobs + 4 * c0);
  if (job.x < 0) return;
  const int e = job.x, h = job.y, parts = job.z - c0 + 1;
  const int b = e / a.n_qt, j = (e - b * a.n_qt) * a.qt + r / a.R;
  const bool there = r < rows && j < a.n;
  auto part = [&](int i) { return part_row(a, i == 0 ? 2 * c0 + 1 : 2 * (c0 + i), rows, r); };
  float m = -INFINITY, l = 0.0f;
  if (there)
    for (int i = tid; i < parts; i += 128) m = fmaxf(m, part(i)[D]);
  m = warp_max(m);
  if (tid % 32 == 0) s_max[group][tid / 32] = m;
  __syncthreads();
  m = fmaxf(fmaxf(s_max[group][0], s_max[group][1]), fmaxf(s_max[group][2], s_max[group][3]));
  if (there)
    for (int i = tid; i < parts; i += 128) {
      const float f = exp2_approx(part(i)[D] - m);
      s_f[group][i] = f;
      l += part(i)[D + 1] * f;
    }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
  if (tid % 32 == 0) s_sum[group][tid / 32] = l;
  __syncthreads();
  if (!there) return;
  l = (s_sum[group][0] + s_sum[group][1]) + (s_sum[group][2] + s_sum[group][3]);
  const int64_t at = (static_cast<int64_t>(b) * a.n + j) * a.Hq + h * a.R + r % a.R;
  if (tid < D) {
    float v = 0.0f;
#pragma unroll 8
    for (int i = 0; i < parts; ++i) v += part(i)[tid] * s_f[group][i];
    v = l == 0.0f ? 0.0f : v / l;
    if (a.bf16) static_cast<__nv_bfloat16*>(a.out)[at * D + tid] = __float2bfloat16_rn(v);
    else static_cast<__half*>(a.out)[at * D + tid] = __float2half_rn(v);
  }
  if (a.lse && tid == 0)
    a.lse[at] = l == 0.0f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

// Whether kv_attend_many_kernel takes a call over the whole cache: where a tile
// of its rows is full, and there are so many rows in all that joining parts of
// 256 rows does not outweigh its faster tiles. Both forms, 4 to 32 heads of 128
// dimensions, us (many | kv_attend_kernel): 8 KV heads x 128 rows over 8,192
// tokens 33.5 | 29.3, 8 x 256 35.0 | 40.2, 8 x 512 44.1 | 65.4; 64 x 128 rows
// over 4,096 50.9 | 67.9; 1 x 256 over 32,768 42.5 | 28.3, 1 x 512 41 | 39. The
// rows alone decide, although longer contexts favour the first form (2 x 1,024
// rows over 100,000 tokens 132 | 268): calls of fewer rows over such contexts were
// not measured.
bool takes_many(int32_t B, int32_t n, int32_t Hq, int32_t Hkv) {
  return static_cast<int64_t>(n) * (Hq / Hkv) >= kManyRows && static_cast<int64_t>(B) * n * Hq >= 2048;
}

// Rows of the instantiation for `rows` of them.
int rows_form(int rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

bool encode_cache_map(CUtensorMap* tm, const uint8_t* base, const KvCacheArgs& c) {
  const EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.Hkv) * c.block,
                              static_cast<cuuint64_t>(c.n_pages)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.page_stride)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(c.D), static_cast<cuuint32_t>(c.block), 1};
  const cuuint32_t elem[3] = {1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(base), dims, strides, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t kv_attend_workspace_bytes(int32_t B, int32_t n, int32_t Hq, int32_t Hkv, int32_t D) {
  if (B < 0 || n < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > kKvMaxGroup || (D != 64 && D != 128))
    return 0;
  const size_t rows = takes_many(B, n, Hq, Hkv) ? 2 * kManyRows : kKvMaxGroup;
  return sizeof(float) * 2 * kKvMaxCtas * rows * (static_cast<size_t>(D) + 2) + 4 * sizeof(int32_t) * kKvMaxCtas;
}

cudaError_t launch_kv_attend(const KvAttendProblem& p, const DeviceInfo& dev, cudaStream_t stream) {
  AttendArgs a{};
  a.c = p.cache;
  a.q = p.q;
  a.out = p.out;
  a.lse = p.lse;
  a.ids = p.ids;
  a.status = dev.status_word;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.n = p.n;
  a.Hq = p.Hq;
  a.R = p.Hq / p.cache.Hkv;
  a.n_lists = p.n_lists;
  a.k = p.k;
  a.spt = kKvTile / p.cache.block;
  a.bf16 = p.bf16;
  // Chosen blocks are each query's own; over the whole cache, consecutive
  // queries of a sequence share a tile, of up to 16 rows (the form of 32 rows
  // holds too much state for its threads and takes more than twice as long a
  // tile) or two of up to 128.
  const bool many = !p.ids && takes_many(p.cache.B, p.n, p.Hq, p.cache.Hkv);
  a.qt = p.ids ? 1 : many ? 2 * (kManyRows / a.R) : std::max(1, std::min(p.n, 16 / a.R));
  a.n_qt = (p.n + a.qt - 1) / a.qt;
  a.fixed = p.ids ? (p.k + a.spt - 1) / a.spt : 0;
  const int rt = rows_form(a.qt * a.R);
  // One CTA an SM, or one a tile where the lists or tables allow fewer tiles.
  const int64_t item_tiles = a.fixed > 0 ? a.fixed : (p.cache.max_blocks - 1) / a.spt + 1;
  const int64_t most = static_cast<int64_t>(p.cache.B) * a.n_qt * p.cache.Hkv * item_tiles;
  const int grid = static_cast<int>(std::min<int64_t>(std::min(dev.sm_count, kKvMaxCtas), most));
  // (No item costs more than another where a CTA has a tile or two.)
  a.item_cost = many ? kManyItemCost : p.ids || most <= 2 * grid ? 0 : kItemCost;
  a.jobs = static_cast<int32_t*>(p.workspace);
  a.parts = reinterpret_cast<float*>(a.jobs + 4 * kKvMaxCtas);

  if (many) return launch_attend_many(a, grid, item_tiles > 1, dev.id, stream);

  CUtensorMap tk, tv;
  if (!encode_cache_map(&tk, p.cache.k, p.cache) || !encode_cache_map(&tv, p.cache.v, p.cache))
    return cudaErrorInvalidValue;
  const AttendLaunch form = p.cache.D == 64 ? (p.bf16 ? attend_d64_t2 : attend_d64_t3)
                                            : (p.bf16 ? attend_d128_t2 : attend_d128_t3);
  cudaError_t e = form(rt, tk, tv, a, grid, dev.id, stream);
  if (e != cudaSuccess) return e;
  plan_add("kv_attend_kernel");
  // Items of one tile are never split.
  if (item_tiles == 1) return cudaSuccess;
  e = launch_pdl(kv_combine_kernel, dim3(grid, (a.qt * a.R + kCombineRows - 1) / kCombineRows),
                 dim3(128 * kCombineRows), 0, stream, a);
  if (e == cudaSuccess) plan_add("kv_combine_kernel");
  return e;
}

}  // namespace qsa
