// kv_attend.cu - launcher of the cache attention, and the kernel that joins
// the partial results of items that were split over several CTAs.
#include "kv_attend_many.cuh"

#include <algorithm>

namespace qsa {
namespace {

constexpr int kCombineRows = 4;   // rows of a CTA, a warp each
constexpr int kCombineAhead = 4;  // parts whose values are asked for before their number is known
constexpr int kCombineLoads = 12;  // parts after these, asked for together (4: 2 x 131,073 tokens of 8 bits 53.4 us, not 52.5)
// What an item costs beside its tiles, in tiles: a batch of 32 requests of 100
// tokens and 32 of 16,384 takes 168 us instead of 484 at 0, 256 requests of 64 to
// 829 tokens 50 us instead of 114, 64 requests of 1,000 to 16,384 tokens 175 at
// both (at 3 the first two take 165 and 57, at 8 169 and 50; taken when
// references only rose, the second is 54 us since).
constexpr int kItemCost = 5;

// Joins the parts of the item that CTA blockIdx.x of the attention began and
// others ended: that CTA's second slot and the first slots of the CTAs after
// it, added in order. The sums are fp32 and the parts added in the order of the
// tokens, so a call repeats its bits.
//
// It is bound by its launch and its loads' latency, which every call over a whole
// context waits for: a warp has a row, so that nothing waits for a barrier; the first
// parts are read (from the workspace, whatever stands there) together with the note
// that says how many there are; and a CTA is small enough to lie beside one of the
// attention's, waiting for its end. One token over 1,000 tokens took 8.6 us with CTAs
// of 512 threads and three loads one after the other.
__global__ void __launch_bounds__(32 * kCombineRows) kv_combine_kernel(const __grid_constant__ AttendArgs a) {
  pdl_wait();
  pdl_launch_dependents();  // after the wait: at most one kernel ahead of the one that runs
  const int lane = threadIdx.x % 32, rows = a.qt * a.R, D = a.c.D, per = D / 64;
  const int c0 = blockIdx.x, r = blockIdx.y * kCombineRows + threadIdx.x / 32;
  if (r >= rows) return;
  auto part = [&](int i) { return part_row(a, i == 0 ? 2 * c0 + 1 : 2 * (c0 + i), rows, r); };
  const int there = static_cast<int>(gridDim.x) - c0;  // parts that there can be
  const uint4 job = load_global(reinterpret_cast<const uint4*>(a.jobs + 4 * c0));
  float2 ml = make_float2(-INFINITY, 0.0f);  // reference and sum of part `lane`
  if (lane < there) ml = *reinterpret_cast<const float2*>(part(lane) + D);
  float2 v[kCombineAhead][2];
#pragma unroll
  for (int i = 0; i < kCombineAhead; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (i < there && k < per) v[i][k] = *reinterpret_cast<const float2*>(part(i) + 64 * k + 2 * lane);
  if (static_cast<int>(job.x) < 0) return;
  const int e = job.x, h = job.y, parts = static_cast<int>(job.z) - c0 + 1;
  const int b = e / a.n_qt, j = (e - b * a.n_qt) * a.qt + r / a.R;
  if (j >= a.n) return;
  float m = lane < parts ? ml.x : -INFINITY;
  for (int i = lane + 32; i < parts; i += 32) m = fmaxf(m, part(i)[D]);
  m = warp_max(m);
  // The weights' sum in four trees, of parts 32 q .. 32 q + 31 (and 128 more) each.
  float f = lane < parts ? exp2_approx(ml.x - m) : 0.0f, sums[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (32 * q >= parts) break;
    float l = 0.0f;
    for (int i = 32 * q + lane; i < parts; i += 128)
      l += i == lane ? ml.y * f : part(i)[D + 1] * exp2_approx(part(i)[D] - m);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
    sums[q] = l;
  }
  const float l = (sums[0] + sums[1]) + (sums[2] + sums[3]);
  float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](const float2 (&x)[2], float w) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (k < per) {
        o[2 * k] += x[k].x * w;
        o[2 * k + 1] += x[k].y * w;
      }
  };
#pragma unroll
  for (int i = 0; i < kCombineAhead; ++i)
    if (i < parts) add(v[i], __shfl_sync(0xFFFFFFFFu, f, i));
  for (int i0 = kCombineAhead; i0 < parts; i0 += kCombineLoads) {
    float2 u[kCombineLoads][2];
#pragma unroll
    for (int i = 0; i < kCombineLoads; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (i0 + i < parts && k < per) u[i][k] = *reinterpret_cast<const float2*>(part(i0 + i) + 64 * k + 2 * lane);
#pragma unroll
    for (int i = 0; i < kCombineLoads; ++i) {
      if (i0 + i >= parts) break;
      if ((i0 + i) % 32 == 0) f = i0 + i + lane < parts ? exp2_approx(part(i0 + i + lane)[D] - m) : 0.0f;
      add(u[i], __shfl_sync(0xFFFFFFFFu, f, (i0 + i) % 32));
    }
  }
  const int64_t at = (static_cast<int64_t>(b) * a.n + j) * a.Hq + h * a.R + r % a.R;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k < per) {
      const float x = l == 0.0f ? 0.0f : o[2 * k] / l, y = l == 0.0f ? 0.0f : o[2 * k + 1] / l;
      static_cast<uint32_t*>(a.out)[(at * D + 64 * k) / 2 + lane] = a.bf16 ? bf162_of(x, y) : half2_of(x, y);
    }
  if (a.lse && lane == 0) a.lse[at] = l == 0.0f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

// 4-bit cache: the join is a launch of its own, about 4 us of a call in a stream, as
// long as so many tiles of a CTA. Where a CTA for each item is no more than that
// behind equal shares, nothing is split (one token over 1,000 tokens 7.2 us instead
// of 8.3, replayed by a graph, 32 requests with 64 chosen blocks 20.4 instead of 25.1;
// 4 and 16 tiles were no better). Of whole contexts the table's room decides, as lengths
// are on the device: the same token with a table for 131,072 takes the 8.3 us.
constexpr int kJoinTiles = 8;
// 4-bit cache: tiles of a CTA up to which the heads of an item are split in two where
// one item's columns would need the form of 32, which takes 1.8 to 2 times as long a
// tile as that of 16 but has half of the tiles. us (split | whole), 32 heads on each
// of 2 KV heads, 128 dimensions, fp16: 64 requests of 2,000 tokens (13 tiles a CTA)
// 34.0 | 39.2, 2 of 131,073 (27) 45.2 | 47.5, 32 of 8,000 (27) 45.3 | 45.8, 64 of 8,000
// (53) 83.9 | 77.7, 16 of 40,000 (66) 97.9 | 83.7; bf16 31.8 | 33.0, 38.3 | 39.9,
// 40.1 | 38.6, 70.2 | 65.6, 78.2 | 70.8. (16 heads of 64 dimensions: 64 of 8,000
// 43.7 | 46.0, 128 of 8,000 75.8 | 79.7, bf16 72.8 | 69.7.)
constexpr int kSplitTiles = 32;

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

// The same for the 4-bit cache, where it takes `tokens` into account, those that a
// table has room for. us (many | kv_attend_kernel), fp16, 128 dimensions: 1 x 512 rows
// over 32,768 tokens 40.0 | 41.8, over 131,072 68.5 | 126; 1 x 1,024 over 8,192 30.5 | 29.4,
// over 32,768 44.3 | 71.0; 8 x 128 over 8,192 32.4 | 28.0, over 32,768 60.1 | 70.8;
// 2 x 1,024 over 1,024 21.5 | 11.4, over 4,096 29.1 | 31.0, over 8,192 35.1 | 45.0; 8 x 512
// over 1,024 26.1 | 27.8. 64 dimensions: 1 x 512 over 8,192 24.8 | 19.4, over 32,768
// 31.8 | 39.2; 1 x 1,024 over 4,096 21.3 | 20.8, over 8,192 22.6 | 27.4; 2 x 1,024 over
// 1,024 16.7 | 18.7, over 4,096 21.8 | 30.7. The first form costs 6 to 10 us more for
// any call and, of rows times tokens, a third of the time. (Under 512 rows, where
// only contexts past 32,768 tokens would gain, calls keep the small workspace.)
bool may_take_many4(int32_t B, int32_t n, int32_t Hq, int32_t Hkv) {
  return static_cast<int64_t>(n) * (Hq / Hkv) >= kManyRows && static_cast<int64_t>(B) * n * Hq >= 512;
}
bool takes_many4(int32_t B, int32_t n, int32_t Hq, int32_t Hkv, int32_t D, int64_t tokens) {
  return may_take_many4(B, n, Hq, Hkv) &&
         static_cast<double>(B) * n * Hq * tokens >= (D == 128 ? 10.0 : 4.0) * (1 << 20);
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

size_t workspace_bytes(int32_t B, int32_t n, int32_t Hq, int32_t Hkv, int32_t D, bool four) {
  if (B < 0 || n < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > kKvMaxGroup || (D != 64 && D != 128)) return 0;
  const size_t rows = (four ? may_take_many4 : takes_many)(B, n, Hq, Hkv) ? 2 * kManyRows : kKvMaxGroup;
  return sizeof(float) * 2 * kKvMaxCtas * rows * (static_cast<size_t>(D) + 2) + 4 * sizeof(int32_t) * kKvMaxCtas;
}

// Either cache's attention.
cudaError_t launch(const KvAttendProblem& p, const DeviceInfo& dev, cudaStream_t stream, bool four) {
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
  a.split = 1;
  a.n_lists = p.n_lists;
  a.k = p.k;
  a.bf16 = p.bf16;
  // Chosen blocks are each query's own; over the whole cache, consecutive
  // queries of a sequence share a tile, of up to 16 rows (the form of 32 rows
  // holds too much state for its threads and takes more than twice as long a
  // tile) or two of up to 128. A row of the 4-bit cache's 64 dimensions has a
  // column for each of the two tokens in an operand row.
  const KvCacheArgs& c = p.cache;
  const bool many = !p.ids && (four ? takes_many4(c.B, p.n, p.Hq, c.Hkv, c.D, static_cast<int64_t>(c.max_blocks) * c.block)
                                    : takes_many(c.B, p.n, p.Hq, c.Hkv));
  const int columns = four && !many ? 128 / c.D : 1;
  a.tile_log2 = columns == 2 ? 8 : 7;
  a.spt = (1 << a.tile_log2) / c.block;
  a.fixed = p.ids ? (p.k + a.spt - 1) / a.spt : 0;
  const int64_t item_tiles = a.fixed > 0 ? a.fixed : (c.max_blocks - 1) / a.spt + 1;
  const int ctas = std::min(dev.sm_count, kKvMaxCtas);
  // Whether a CTA has an item each. (Lists are known here; of whole contexts only
  // that none has more than item_tiles.)
  auto an_item_each = [&](int64_t items) {
    return four && !many && items <= ctas &&
           (p.ids ? item_tiles * (ctas - items) <= kJoinTiles * ctas : item_tiles <= kJoinTiles);
  };
  if (four && !many && a.R * columns > 16) {
    // Split (where two equal parts of 16 columns or fewer make an item of up to 32)
    // items read the same tiles, at about the same time while there are few of them.
    const int fine = head_split(a.R, columns, 16), least = head_split(a.R, columns, 32);
    const int64_t items = static_cast<int64_t>(c.B) * p.n * c.Hkv;  // of one query each
    const bool pays = an_item_each(items * fine) ||
                      (!an_item_each(items * least) && items * least * item_tiles <= kSplitTiles * ctas);
    a.split = fine <= 2 * least && pays ? fine : least;
    a.R /= a.split;
  }
  a.heads = c.Hkv * a.split;
  a.qt = p.ids ? 1 : many ? 2 * (kManyRows / a.R) : std::max(1, std::min(p.n, 16 / (a.R * columns)));
  a.n_qt = (p.n + a.qt - 1) / a.qt;
  const int rt = rows_form(a.qt * a.R * columns);
  // One CTA an SM, or one a tile where the lists or tables allow fewer tiles.
  const int64_t items = static_cast<int64_t>(c.B) * a.n_qt * a.heads, most = items * item_tiles;
  a.per_item = an_item_each(items);
  const int grid = static_cast<int>(a.per_item ? items : std::min<int64_t>(ctas, most));
  // (No item costs more than another where a CTA has a tile or two.)
  a.item_cost = many ? kManyItemCost : p.ids || a.per_item || most <= 2 * grid ? 0 : kItemCost;
  a.jobs = static_cast<int32_t*>(p.workspace);
  a.parts = reinterpret_cast<float*>(a.jobs + 4 * kKvMaxCtas);

  if (many) return (four ? launch_attend4_many : launch_attend_many)(a, grid, item_tiles > 1, dev.id, stream);

  CUtensorMap tk, tv;
  const auto encode = four ? encode_cache_map4 : encode_cache_map;
  if (!encode(&tk, p.cache.k, p.cache) || !encode(&tv, p.cache.v, p.cache)) return cudaErrorInvalidValue;
  const AttendLaunch forms[2][2][2] = {{{attend_d64_t3, attend_d64_t2}, {attend_d128_t3, attend_d128_t2}},
                                       {{attend4_d64_t3, attend4_d64_t2}, {attend4_d128_t3, attend4_d128_t2}}};
  cudaError_t e = forms[four][p.cache.D == 128][p.bf16](rt, tk, tv, a, grid, dev.id, stream);
  if (e != cudaSuccess) return e;
  plan_add(four ? "kv4_attend_kernel" : "kv_attend_kernel");
  // Items of one tile are never split.
  if (item_tiles == 1 || a.per_item) return cudaSuccess;
  e = launch_pdl(kv_combine_kernel, dim3(grid, (a.qt * a.R + kCombineRows - 1) / kCombineRows),
                 dim3(32 * kCombineRows), 0, stream, a);
  if (e == cudaSuccess) plan_add("kv_combine_kernel");
  return e;
}

}  // namespace

// Of the 4-bit cache: operand rows of 128 codes, one token of 128 dimensions or
// two of 64, which the copy spreads to 128 bytes.
bool encode_cache_map4(CUtensorMap* tm, const uint8_t* base, const KvCacheArgs& c) {
  const EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const int rows = c.block * c.D / 128;
  const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(c.Hkv) * rows, static_cast<cuuint64_t>(c.n_pages)};
  const cuuint64_t strides[2] = {64, static_cast<cuuint64_t>(c.page_stride)};
  const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(rows), 1};
  const cuuint32_t elem[3] = {1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 3, const_cast<uint8_t*>(base), dims, strides, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int head_split(int R, int per_row, int columns) {
  int s = 1;
  while (R % s != 0 || R / s * per_row > columns) ++s;
  return s;
}

size_t kv_attend_workspace_bytes(int32_t B, int32_t n, int32_t Hq, int32_t Hkv, int32_t D) {
  return workspace_bytes(B, n, Hq, Hkv, D, false);
}
size_t kv4_attend_workspace_bytes(int32_t B, int32_t n, int32_t Hq, int32_t Hkv, int32_t D) {
  return workspace_bytes(B, n, Hq, Hkv, D, true);
}

cudaError_t launch_kv_attend(const KvAttendProblem& p, const DeviceInfo& dev, cudaStream_t stream) {
  return launch(p, dev, stream, false);
}
cudaError_t launch_kv4_attend(const KvAttendProblem& p, const DeviceInfo& dev, cudaStream_t stream) {
  return launch(p, dev, stream, true);
}

}  // namespace qsa
