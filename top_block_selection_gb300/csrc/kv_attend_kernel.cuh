// kv_attend_kernel.cuh - attention over the paged 8-bit cache, whole or over
// chosen blocks. One instantiation per head size and row count.
//
// For the R query heads of one KV head (and, over the whole cache, a few
// consecutive queries), rows r and cached tokens t:
//     x[r,t] = scale * q_r . (sk_b code_k[t]),  t visible to r;  m_r = max_t x
//     out_r  = sum_t 2^(x - m) (sv_b code_v[t]) / sum_t 2^(x - m)   (x in log2 units)
// with sk_b, sv_b the scales of the token's block.
//
// The codes go to the tensor cores as they are. Both products are
// tcgen05.mma kind::f8f6f4 with the cache as the M = 128 operand (128 tokens
// for the scores, the D dimensions for the output, read MN-major), loaded by
// TMA and never touched by a thread. The other operand is made e4m3 without
// losing its bits, as a sum of T terms of 4 significant bits, T = 3 for fp16
// and 2 for bf16 calls:
//   queries        y1 = e4m3(y), y2 = e4m3(16 (y - y1)), y3 = ...: exact for every
//                  fp16 (T = 3) or bf16 (T = 2) element above 2^-13 of its
//                  row's largest, the rest to 2^-25 (T = 2: 2^-21) of that;
//   probabilities  T = 3: cut, cut and rounded, to 2^-12 of each; T = 2:
//                  rounded twice, to 2^-9: a fraction of the rounding of the
//                  result (2^-11 and 2^-8 at most). The later terms are scaled
//                  up (T = 3 by 8 and 128, T = 2 by 16) and take what the one
//                  before leaves, its smallest step included. A probability is
//                  then lost only below 2^-22 of the largest (T = 2: 2^-19).
// The terms are groups of columns of one product, added in fp32 after it.
// With few rows a tile's product is bound by reading the M operand from
// shared memory, so the extra columns cost little.
//
// The softmax reference m_r is not each tile's maximum but one that lags: it
// is set above the largest weight, score plus logarithm of the value scale (by
// two in log2), and a tile keeps it as long as its codes still fit below 448.
// Most tiles thus need one vote of the warpgroup instead of a maximum over its
// tokens for each row, and the output stays in TMEM, accumulated by the product
// itself, until a reference moves or the item ends. Every 8th tile (T = 2: 4th)
// of a warpgroup since is looked at for each row, and a reference more than
// five above its largest weight goes down: codes have steps, and behind one
// token far above all others (the first of a context often is) every later
// one would be lost below them, however much they are together. The value
// scales ride on the probabilities, relative to the largest at the last move.
//
// What bounds it: decoding reads every code once from HBM (about 23 bytes a
// cycle and SM); over chosen blocks of many queries the codes come from L2.
// Each CTA (one per SM) runs a ring of 128-token stages, two or three
// warpgroups that take the tiles in turn, each with its own running reference,
// sum and output (so that loads, products and the softmax of different tiles
// overlap without a hand-over between them) and its own producer warp (one
// warp for all took 1,200 to 1,450 cycles a tile: as long as everything else),
// and one warp that prepares the next query rows. All tiles of a call are
// dealt to the CTAs in equal contiguous shares, whatever the lengths; a (query
// tile, head) item that ends up in several CTAs leaves partial results in the
// workspace, which kv_combine_kernel joins.
//
// Measured (with the join): a decode step of 64 requests over 1,000 to 16,384
// tokens, 8 KV heads, bf16: 175 us, 6.5 TB/s (97% of a plain copy's rate). One
// token over 2 x 131,073 tokens, 16 heads on each of 4 KV heads, fp16: 53 us,
// 5.0 TB/s. 4,096 queries with 64 chosen blocks each, 16 heads on one KV head:
// 491 us, 280 TFLOP/s; there the shared-memory pipe was 75% to 85% busy at 460 us
// (terms without the steps' remainders, references that only rose).
#pragma once

#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_internal.h"
#include "qsa_device.cuh"

namespace qsa {

constexpr int kKvTile = 128;       // tokens of a tile
constexpr int kKvMaxSlots = 8;     // blocks of a tile (block >= 16)
constexpr int kKvMaxCtas = 192;    // bound of the grid, sizes the workspace
constexpr int kKvNoToken = 0x3FFFFFFF;

struct AttendArgs {
  KvCacheArgs c;
  KvRows q;
  void* out;
  float* lse;
  const int32_t* ids;
  float* parts;      // [2 * grid][rows][D + 2]: of each row its output, reference and sum
  int32_t* jobs;     // [grid][4]: entry, head, last CTA of an item that this CTA begins and others end; or -1
  uint32_t* status;
  float scale_log2;
  int32_t n, Hq, R;
  int32_t qt, n_qt;  // queries of a tile, query tiles of a sequence
  int32_t n_lists, k;
  int32_t spt;       // blocks of a tile
  int32_t fixed;     // tiles of every item over chosen blocks, else 0
  int32_t item_cost; // what an item costs beside its tiles, in tiles: counts where they are dealt out
  bool bf16;
};

// Row r of partial `slot`: D outputs, then all rows' maxima and sums.
__device__ __forceinline__ float* part_row(const AttendArgs& a, int slot, int rows, int r) {
  return a.parts + (static_cast<int64_t>(slot) * rows + r) * (a.c.D + 2);
}

// a / b for a >= 0, b > 0, in 32 bits where they suffice.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (((static_cast<uint64_t>(a) | static_cast<uint64_t>(b)) >> 32) == 0)
    return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// What the query tile `e` sees: its rows' queries j0 .. j0 + nq - 1 (those that
// exist), the position of the first and the last, and its tiles.
struct Entry {
  int32_t b, j0, nq, first_pos, last_pos, tiles;
};
__device__ __forceinline__ Entry entry_of(const AttendArgs& a, int e) {
  Entry t;
  t.b = a.n_qt > 1 ? e / a.n_qt : e;
  t.j0 = (e - t.b * a.n_qt) * a.qt;
  const Span s = span_of(a.c, t.b, a.n);
  t.nq = min(t.j0 + a.qt, s.n_new) - t.j0;
  t.last_pos = t.nq > 0 ? s.first + t.j0 + t.nq - 1 : -1;
  t.first_pos = s.first + t.j0;  // may be negative: those rows see nothing
  if (a.fixed > 0) {
    t.tiles = a.fixed;
  } else {
    const int keys = min(t.last_pos + 1, a.c.max_blocks * a.c.block);
    t.tiles = keys > 0 ? (keys - 1) / kKvTile + 1 : 1;
  }
  return t;
}

// A CTA's walk over its share of the tiles: the part [t, t + n) of item (e, h).
struct Walk {
  int32_t e, h, t;
  int64_t left;
};
struct Start {
  Walk walk;
  Entry entry;  // of walk.e
};

// A CTA's share of all tiles, [lo, hi) of total dealt to `grid` CTAs.
struct Share {
  Start start;
  int64_t lo, hi, total;
  int32_t grid;
};

// ------------------------------------------------------------ tcgen05 pieces
// D[tmem] (+)= A[smem] * B[smem]^T on e4m3 codes, issued by one thread.
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor: fp32 D (bits 4-5 = 1), e4m3 A and B (formats 0), A
// and B MN-major when asked (bits 15, 16), N >> 3 at bits 17-22, M >> 4 at
// bits 24-28.
__host__ __device__ constexpr uint32_t idesc_f8(int N, bool mn_major) {
  return (1u << 4) | (mn_major ? 3u << 15 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}

// Shared-memory descriptor of rows of ROW bytes (128 or 64) swizzled over
// their own width, 8-row groups 8 * ROW bytes apart. K-major, the group stride
// steps over rows; MN-major (rows run along K), it steps over 8 K. The leading
// offset only matters for an MN-major tile wider than a row: rows of 64 bytes
// then repeat at the next group (the output lanes 64-127 they give are not read).
template <int ROW>
__device__ __forceinline__ uint64_t smem_desc_rows(uint32_t saddr) {
  constexpr uint64_t swizzle = ROW == 128 ? 2 : 4;
  constexpr uint64_t group = (8 * ROW) >> 4;
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (group << 16) | (group << 32) | (1ull << 46) |
         (swizzle << 61);
}

// The probabilities: MN-major without swizzle, 16 columns of a token in 16
// bytes, 8 tokens in 128, then the next 8 tokens (leading offset), the next 16
// columns behind all 128 tokens (stride offset). A thread writes its token's
// terms by 16-byte stores, 32 threads of a warp 512 consecutive bytes.
__device__ __forceinline__ uint64_t smem_desc_tokens(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 16) |
         (static_cast<uint64_t>(16 * kKvTile >> 4) << 32) | (1ull << 46);
}

template <int ROW>
__device__ __forceinline__ uint32_t swizzled(uint32_t off) {
  return ROW == 128 ? off ^ ((off >> 3) & 0x70u) : off ^ ((off >> 3) & 0x30u);
}

// Each thread reads NC consecutive columns of its TMEM lane.
template <int NC>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&r)[NC]);
template <>
__device__ __forceinline__ void tmem_ld_cols<4>(uint32_t taddr, float (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3])
               : "r"(taddr)
               : "memory");
}
template <>
__device__ __forceinline__ void tmem_ld_cols<8>(uint32_t taddr, float (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
               : "r"(taddr)
               : "memory");
}
template <>
__device__ __forceinline__ void tmem_ld_cols<16>(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
      : "memory");
}
template <>
__device__ __forceinline__ void tmem_ld_cols<32>(uint32_t taddr, float (&r)[32]) {
  uint32_t u[32];
  tmem_ld_32cols(taddr, u);
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __uint_as_float(u[i]);
}

// ------------------------------------------------------------- small pieces
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Whether a phase has completed, without waiting for it at all (try_wait may
// hold the thread for a while).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// bar_sync that also tells every thread whether any of them passed true.
__device__ __forceinline__ bool bar_any(int id, int threads, bool p) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(p))
      : "memory");
  return r != 0;
}
// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// A value that all lanes hold, known to the compiler as such: descriptors and
// addresses of single-thread instructions then stay in uniform registers.
template <class V>
__device__ __forceinline__ V uniform(V x) {
  return __shfl_sync(0xFFFFFFFFu, x, 0);
}
__device__ __forceinline__ float log2_approx(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float warp_max(float x) {  // NaN counts as nothing
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two fp32 operations in one instruction.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void f2_get(F2 a, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v));
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Waits for a phase of `bar`, but at most kWaitTimeoutNs; the first wait of a
// CTA that runs out sets its stop flag (and the device's status word), and
// from then on every wait of the CTA returns at once. Loop counts never hang
// on what a failed wait would have guarded, so all warps still reach the end.
__device__ __forceinline__ bool wait_or_stop(uint64_t* bar, uint32_t parity, volatile uint32_t* stop,
                                             uint32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*stop) return false;
    if (global_timer_ns() - t0 > kWaitTimeoutNs) {
      *stop = 1;
      atomicOr(status, kErrKvWaitTimeout);
      return false;
    }
  }
}

// ------------------------------------------------------------ configuration
template <int D_, int RT_, int T_>
struct AttendCfg {
  static constexpr int D = D_;
  static constexpr int RT = RT_;                            // rows
  static constexpr int T = T_;                              // e4m3 terms of a value
  static constexpr int N = (T * RT + 15) / 16 * 16;         // columns: the terms of each row
  static constexpr int W = RT >= 32 ? 2 : 3;                // warpgroups
  static constexpr int kThreads = W * 128 + W * 32 + 32;    // they, a producer warp for each, the query warp
  static constexpr int kStageBytes = 2 * kKvTile * D;       // K then V
  // A stage serves one warpgroup only: a parity wait may not run two phases
  // ahead, and only a stage's own last user knows that its phase has passed.
  static constexpr int kStages = (RT >= 32 ? 4 : 6) * (128 / D);
  static_assert(kStages % W == 0, "a stage serves one warpgroup");
  static constexpr int kQBytes = N * D;                     // one of two buffers
  static constexpr int kPBytes = N * kKvTile;               // one of W
  static constexpr int kJoinRows = RT <= 8 ? RT : RT / 2;   // rows joined at a time, over the P buffers
  static constexpr int kJoinBytes = W * kJoinRows * D * 4;
  static constexpr int kPRegion = W * kPBytes > kJoinBytes ? W * kPBytes : kJoinBytes;
  static constexpr int kTmemCols = 2 * N * W <= 128 ? 128 : (2 * N * W <= 256 ? 256 : 512);
  static_assert(2 * N * W <= 512, "TMEM");
  // Tiles of a warpgroup after which it looks whether its references stand too
  // high for the tokens that come now.
  static constexpr int kRun = T == 3 ? 8 : 4;
};

struct StageMeta {
  int32_t base[kKvMaxSlots];  // position of the slot's first token, kKvNoToken if none
  float ks[kKvMaxSlots];      // key scale
  float vs[kKvMaxSlots];      // value scale (0: no block)
  float vmax;                 // the largest of them
};

template <int RT>
struct ItemInfo {
  alignas(16) int32_t row_pos[RT];  // last position the row sees; -1: nothing
  alignas(16) float row_mul[RT];    // query scale * softmax scale * log2(e)
  int64_t row_at[RT];               // index of the row in out (rows of D) and lse; -1: none
  int32_t tiles;                    // of this CTA's part; 0 ends the walk
  int32_t lo_pos, hi_pos;           // smallest and largest row_pos of rows that see anything
  int32_t rows;
  int32_t slot;                     // partial result to write, -1: the whole item
};

template <class C>
struct AttendShared {
  ItemInfo<C::RT> item[2];
  StageMeta meta[C::kStages];
  alignas(16) float red[C::W][C::RT][4];     // per-warp maxima, then sums
  alignas(16) float spread[C::W][4];         // per-warp: the largest value scale over its tokens' smallest (log2)
  // References and factors of what was summed, where they move (all warps write the
  // same); at an item's end, references or the largest scores, if these are above.
  alignas(16) float moved[C::W][C::RT], alpha[C::W][C::RT];
  alignas(16) float ml[2][C::W][C::RT];  // the warpgroups' references (then weights) and sums
  float mx[C::RT], sum[C::RT], inv[C::RT];  // joined, 1 / sum
  alignas(16) int32_t poison[128];  // first position whose value code is NaN, per dimension
  uint64_t full[C::kStages], empty[C::kStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_bar[C::W];
  int64_t scan[C::W + 1];
  Share share;
  uint32_t tmem;
  uint32_t stop;
};

// Past what is left of an item's cost, which lies in front of its tiles (t < 0).
__device__ __forceinline__ void skip_cost(Walk& w) {
  if (w.t >= 0) return;
  const int n = static_cast<int>(min(static_cast<int64_t>(-w.t), w.left));
  w.t += n;
  w.left -= n;
}
// Advances the walk past `part` tiles of an item of `tiles`.
__device__ __forceinline__ void step(Walk& w, int part, int tiles, int heads, int cost) {
  w.left -= part;
  w.t += part;
  if (w.t >= tiles) {
    w.t = -cost;
    if (++w.h == heads) {
      w.h = 0;
      ++w.e;
    }
    skip_cost(w);
  }
}

// ------------------------------------------------------------------ producer
// The tiles of warpgroup p: block lists, pages and scales for up to 32 blocks
// at a time, one per lane, then two TMA loads a block.
template <class C>
__device__ void attend_produce(const AttendArgs& a, const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                               AttendShared<C>& s, uint8_t* ring, const Start& start, int p) {
  constexpr int W = C::W;
  const int lane = threadIdx.x % 32;
  const int spt = a.spt, per_batch = 32 / spt;
  const int my_k = lane / spt, my_slot = lane % spt;
  uint32_t g0 = 0;         // tiles of the CTA before this item
  uint32_t last = 0;       // tiles of this warp so far
  uint32_t last_g[C::kStages / W];
  bool ok = true;
  Walk w = start.walk;
  Entry en = start.entry;
  int en_of = w.e;
  while (w.left > 0 && ok) {
    if (en_of != w.e) {
      en = entry_of(a, w.e);
      en_of = w.e;
    }
    const int part = static_cast<int>(min(static_cast<int64_t>(en.tiles - w.t), w.left));
    const int first = (W - g0 % W + p) % W;  // this warpgroup's tiles: first, first + W, ...
    const int own = part > first ? (part - first + W - 1) / W : 0;
    const int cap = a.c.max_blocks * a.c.block;
    bool bad = en.last_pos >= cap;  // longer than its page table
    const int keys = min(en.last_pos + 1, cap);
    const int32_t* list = nullptr;
    if (a.ids)
      list = a.ids + ((static_cast<int64_t>(en.b) * a.n_lists + (a.n_lists > 1 ? w.h : 0)) * a.n + en.j0) * a.k;
    const int32_t* table = a.c.page_table + static_cast<int64_t>(en.b) * a.c.max_blocks;
    for (int k0 = 0; k0 < own && ok; k0 += per_batch) {
      const int slot = (w.t + first + (k0 + my_k) * W) * spt + my_slot;
      const bool in_part = k0 + my_k < own;
      int blk = in_part ? slot : -1;
      if (list) blk = in_part && slot < a.k ? load_global(list + slot) : -1;
      if (list && blk >= a.c.max_blocks) {
        bad = true;
        blk = -1;
      }
      if (blk >= 0 && static_cast<int64_t>(blk) * a.c.block >= keys) blk = -1;
      int page = blk >= 0 ? load_global(table + blk) : -1;
      if (blk >= 0 && (page < 0 || page >= a.c.n_pages)) {
        bad = true;
        blk = page = -1;
      }
      float ks = 0.0f, vs = 0.0f;
      if (page >= 0) {
        ks = load_global(a.c.k_scale + static_cast<int64_t>(page) * a.c.Hkv + w.h);
        vs = load_global(a.c.v_scale + static_cast<int64_t>(page) * a.c.Hkv + w.h);
      }
      const int z = page >= 0 ? page : a.c.n_pages;  // no block: reads past the last page give zeros
      const int base = page >= 0 ? blk * a.c.block : kKvNoToken;
      const int tiles = min(per_batch, own - k0);
      const int y = uniform(w.h * a.c.block), slab = a.c.block * C::D;
      for (int i = 0; i < tiles; ++i) {
        const uint32_t g = uniform(g0 + first + (k0 + i) * W);
        const uint32_t st = g % C::kStages;
        if (g >= C::kStages)
          ok = wait_or_stop(&s.empty[st], ((g / C::kStages) & 1) ^ 1, &s.stop, a.status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        uint8_t* const k_at = ring + st * C::kStageBytes;
        if (elect_one()) mbar_arrive_expect_tx(&s.full[st], C::kStageBytes);
        for (int j = 0; j < spt; ++j) {
          const int zj = __shfl_sync(0xFFFFFFFFu, z, i * spt + j);
          if (elect_one()) {
            tma_load_3d(k_at + j * slab, tm_k, 0, y, zj, &s.full[st]);
            tma_load_3d(k_at + kKvTile * C::D + j * slab, tm_v, 0, y, zj, &s.full[st]);
          }
          __syncwarp();
        }
        float vmax = vs;
        for (int d = 1; d < spt; d *= 2) vmax = fmaxf(vmax, __shfl_xor_sync(0xFFFFFFFFu, vmax, d));
        if (my_k == i) {
          if (my_slot == 0) s.meta[st].vmax = vmax;
          s.meta[st].base[my_slot] = base;
          s.meta[st].ks[my_slot] = ks;
          s.meta[st].vs[my_slot] = vs;
        }
        last_g[last % (C::kStages / W)] = g;
        ++last;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.full[st]);
      }
    }
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(a.status, kErrCacheIndex);
    g0 += part;
    step(w, part, en.tiles, a.c.Hkv, a.item_cost);
  }
  if (!ok) {  // let the copies in flight land before the CTA gives its memory back
    const uint32_t n = min(last, static_cast<uint32_t>(C::kStages / W));
    for (uint32_t i = last - n; i < last; ++i) {
      const uint32_t g = last_g[i % (C::kStages / W)];
      mbar_wait_bounded(&s.full[g % C::kStages], (g / C::kStages) & 1, 100000000ull);
    }
  }
}

// --------------------------------------------------------- the query's terms
// Rows r0, r0 + step, ... (K of them, below RT) of the query tile `en` for KV
// head h, by one warp: all loaded, then each scaled by a power of two to the
// range of e4m3 and split in terms. Rows that are not there are zero. `dst`
// holds rows of D bytes, term after term.
template <class C, int K>
__device__ __forceinline__ void query_rows(const AttendArgs& a, ItemInfo<C::RT>& info, uint8_t* dst, const Entry& en,
                                           int h, int r0, int step) {
  constexpr int kPer = C::D / 32;  // elements of a lane
  const int lane = threadIdx.x % 32, rows = a.qt * a.R;
  uint32_t u[K][kPer / 2];
  int row_pos[K];
  int64_t row_at[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int r = r0 + k * step, j = a.qt > 1 ? r / a.R : 0, head = h * a.R + (r - j * a.R);
    const bool there = r < rows && j < en.nq && en.first_pos + j >= 0;
    row_pos[k] = r >= rows ? kKvNoToken : (there ? en.first_pos + j : -1);
    row_at[k] = r < rows && en.j0 + j < a.n ? (static_cast<int64_t>(en.b) * a.n + en.j0 + j) * a.Hq + head : -1;
#pragma unroll
    for (int e = 0; e < kPer / 2; ++e) u[k][e] = 0;
    if (there) {
      const uint16_t* const src = static_cast<const uint16_t*>(a.q.data) + en.b * a.q.sb +
                                  static_cast<int64_t>(en.j0 + j) * a.q.sn + static_cast<int64_t>(head) * a.q.sh +
                                  lane * kPer;
      if (kPer == 4) {
        const uint2 v = load_global(reinterpret_cast<const uint2*>(src));
        u[k][0] = v.x;
        u[k][kPer / 2 - 1] = v.y;
      } else {
        u[k][0] = load_global(reinterpret_cast<const uint32_t*>(src));
      }
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int r = r0 + k * step;
    if (r >= C::RT) break;
    float x[kPer], m = 0.0f;
#pragma unroll
    for (int e = 0; e < kPer / 2; ++e) {
      if (a.bf16) {
        x[2 * e] = __uint_as_float(u[k][e] << 16);
        x[2 * e + 1] = __uint_as_float(u[k][e] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[k][e]));
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
      }
      m = fmaxf(m, fmaxf(fabsf(x[2 * e]), fabsf(x[2 * e + 1])));
    }
    const float t = pow2_scale(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m))));
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(t));
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      x[e] *= inv;
      if (isinf(x[e])) x[e] = __int_as_float(0x7FC00000);
    }
#pragma unroll
    for (int term = 0; term < C::T; ++term) {
      uint32_t code[kPer / 2];
#pragma unroll
      for (int e = 0; e < kPer / 2; ++e) {
        code[e] = e4m3x2(x[2 * e], x[2 * e + 1]);
        const float2 back = e4m3x2_to_float2(code[e]);
        x[2 * e] = 16.0f * (x[2 * e] - back.x);  // at most half a step of the code: no more than 16
        x[2 * e + 1] = 16.0f * (x[2 * e + 1] - back.y);
      }
      uint8_t* const to = dst + swizzled<C::D>((term * C::RT + r) * C::D + lane * kPer);
      if (kPer == 4) *reinterpret_cast<uint32_t*>(to) = code[0] | (code[kPer / 2 - 1] << 16);
      else *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(code[0]);
    }
    if (lane == 0) {
      info.row_pos[r] = row_pos[k];
      info.row_mul[r] = t * a.scale_log2;
      info.row_at[r] = row_at[k];
    }
  }
}

// The rest of an item's description, and the note for kv_combine_kernel where
// this CTA begins an item that others end (one thread). `at`: the place of the
// item's first tile among all tiles.
template <class C>
__device__ __forceinline__ void describe_item(const AttendArgs& a, ItemInfo<C::RT>& info, const Entry& en, const Walk& w,
                                              int part, int64_t at, int64_t total, int grid) {
  info.tiles = part;
  info.lo_pos = en.last_pos < 0 ? -1 : max(en.first_pos, 0);
  info.hi_pos = en.last_pos;
  info.rows = a.qt * a.R;
  const bool begins = w.t == 0, ends = w.t + part == en.tiles;
  info.slot = begins && ends ? -1 : 2 * static_cast<int>(blockIdx.x) + (begins ? 1 : 0);
  if (begins && !ends) {
    int32_t* const job = a.jobs + 4 * blockIdx.x;
    job[0] = w.e;
    job[1] = w.h;
    // Tile g belongs to the last CTA c with total * c / grid <= g.
    job[2] = static_cast<int32_t>(divide((at + en.tiles) * grid - 1, total));
  }
}

// The query warp: every item of the CTA's walk but the first (which the
// warpgroups prepare themselves), one ahead of its use.
template <class C>
__device__ void attend_queries(const AttendArgs& a, AttendShared<C>& s, uint8_t* q_smem, const Start& start,
                               int64_t at, int64_t total, int grid) {
  const int lane = threadIdx.x % 32;
  bool ok = true;
  Walk w = start.walk;
  Entry en = start.entry;
  int en_of = w.e;
  for (uint32_t it = 0;; ++it) {
    const int buf = it & 1;
    if (it >= 2) ok = wait_or_stop(&s.q_empty[buf], ((it >> 1) & 1) ^ 1, &s.stop, a.status);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (!ok) break;
    ItemInfo<C::RT>& info = s.item[buf];
    if (w.left <= 0) {
      if (lane == 0) {
        info.tiles = 0;
        mbar_arrive(&s.q_full[buf]);
      }
      break;
    }
    if (en_of != w.e) {
      en = entry_of(a, w.e);
      en_of = w.e;
    }
    const int part = static_cast<int>(min(static_cast<int64_t>(en.tiles - w.t), w.left));
    if (it > 0) {
#pragma unroll 1
      for (int r = 0; r < C::RT; r += 4) query_rows<C, 4>(a, info, q_smem + buf * C::kQBytes, en, w.h, r, 1);
      if (lane == 0) describe_item<C>(a, info, en, w, part, at, total, grid);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.q_full[buf]);
    }
    at += w.t + part + a.item_cost;
    step(w, part, en.tiles, a.c.Hkv, a.item_cost);
  }
}

// ---------------------------------------------------------- the warpgroups
// A value row whose token no row of the tile sees is zeroed, so that 0 * code
// stays 0 whatever stands there. One that some rows see has its NaN codes
// zeroed and remembered: the rows that see them get NaN at the end.
template <int D>
__device__ __noinline__ void clean_value_row(uint8_t* v_row_base, int t, int pos, bool unseen, int32_t* poison) {
  uint4* const row = reinterpret_cast<uint4*>(v_row_base + t * D);
  for (int i = 0; i < D / 16; ++i) {
    if (unseen) {
      row[i] = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint4 u = row[i];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t hit = 0;
    for (int k = 0; k < 4; ++k) hit |= ((w[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    if (!hit) continue;
    uint8_t* const bytes = reinterpret_cast<uint8_t*>(row + i);
    const uint32_t chunk = swizzled<D>(t * D + i * 16) - t * D;  // the swizzle is its own inverse
    for (int k = 0; k < 16; ++k)
      if ((bytes[k] & 0x7F) == 0x7F) {
        bytes[k] = 0;
        atomicMin(&poison[chunk + k], pos);
      }
  }
}

// The columns of RT rows at `taddr`, their T terms added, each 1/16 of the one
// before it (of three terms of a probability, the second 1/8), a few rows at a
// time (the terms of all would not fit in registers beside the softmax state).
template <class C, bool kProbs>
__device__ __forceinline__ void tmem_rows(uint32_t taddr, float (&x)[C::RT]) {
  constexpr int kPart = C::RT <= 8 ? C::RT : C::RT / 2;
#pragma unroll
  for (int r0 = 0; r0 < C::RT; r0 += kPart) {
    float t0[kPart], t1[kPart], t2[kPart];
    tmem_ld_cols<kPart>(taddr + r0, t0);
    tmem_ld_cols<kPart>(taddr + C::RT + r0, t1);
    if (C::T == 3) tmem_ld_cols<kPart>(taddr + 2 * C::RT + r0, t2);
    tmem_ld_wait();
#pragma unroll
    for (int r = 0; r < kPart; r += 2) {
      constexpr float down = kProbs && C::T == 3 ? 0.125f : 0.0625f;
      F2 sum = f2(t1[r], t1[r + 1]);
      if (C::T == 3) sum = fma2(f2(t2[r], t2[r + 1]), f2(0.0625f, 0.0625f), sum);
      sum = fma2(sum, f2(down, down), f2(t0[r], t0[r + 1]));
      f2_get(sum, x[r0 + r], x[r0 + r + 1]);
    }
  }
}

constexpr float kUnset = -3e38f;     // a reference that no score has set yet
// A reference is set so far (log2) above the largest weight: 3 would move it less
// often (4,096 queries with chosen blocks 454 us instead of 461, when references
// only rose) but makes the smallest terms coarser.
constexpr float kMargin = 2.0f;
constexpr float kProbScale = 128.0f; // code of a probability 1 at the largest value scale
constexpr float kMaxCode = 8.8f;     // log2 of the largest code, 448
// How far (log2) below the largest value scale a token's counts where references
// are set, and a reference may go below the largest score: sums of 2^30 tokens
// then stay in fp32's range.
constexpr float kRange = 40.0f;
constexpr float kSlack = 3.0f;        // log2 that a reference may stand too high

template <class C>
__device__ void attend_consume(const AttendArgs& a, AttendShared<C>& s, uint8_t* ring, uint8_t* q_smem,
                               uint8_t* p_smem) {
  constexpr int RT = C::RT, N = C::N, W = C::W, D = C::D;
  constexpr int kAll = W * 128;
  const int wg = uniform(static_cast<int>(threadIdx.x / 128)), warp = uniform(static_cast<int>(threadIdx.x / 32 % 4));
  const int t = threadIdx.x % 128, lane = t % 32;
  const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
  uint8_t* const p_buf = p_smem + wg * C::kPBytes;
  const uint32_t ring_addr = smem_u32(ring), q_addr = smem_u32(q_smem), p_addr = smem_u32(p_buf);
  const int my_slot = t / a.c.block, my_off = t - my_slot * a.c.block;
  uint32_t g0 = 0;      // tiles of the CTA before this item
  uint32_t phase = 0;   // of this warpgroup's score barrier
  uint32_t last_st = 0, last_turn = 0;  // stage of the last tile, and its phase
  const bool leader = elect_one();
  bool bad = false;     // a wait ran out: what follows is not used
  const float kNegInf = -INFINITY;
  uint32_t tm_s = 0, tm_o = 0;

  // Scores of a tile, issued by one thread of the warpgroup's last warp.
  auto issue_scores = [&](uint32_t st, int buf) {
    tc_fence_after_sync();
    const uint64_t ka = smem_desc_rows<D>(ring_addr + st * C::kStageBytes);
    const uint64_t qa = smem_desc_rows<D>(q_addr + buf * C::kQBytes);
    if (leader) {
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks) mma_f8_ss(tm_s, ka + ks * 2, qa + ks * 2, idesc_f8(N, false), ks > 0);
      mma_commit(&s.s_bar[wg]);
    }
    __syncwarp();
  };

  // The service warps have found the share by now, or will.
  bar_sync(9, C::kThreads);
  tc_fence_after_sync();
  pdl_wait();
  pdl_launch_dependents();
  const int64_t total = s.share.total;
  const int grid = s.share.grid;
  if (s.share.hi <= s.share.lo) return;
  tm_s = uniform(s.tmem) + wg * 2 * N;
  tm_o = tm_s + N;
  {
    const Walk walk = s.share.start.walk;
    const Entry en = s.share.start.entry;
    const int64_t at0 = s.share.lo - walk.t;
    if (wg * 4 + warp < RT)
      query_rows<C, (RT + W * 4 - 1) / (W * 4)>(a, s.item[0], q_smem, en, walk.h, wg * 4 + warp, W * 4);
    if (threadIdx.x == W * 128 - 1)
      describe_item<C>(a, s.item[0], en, walk,
                       static_cast<int>(min(static_cast<int64_t>(en.tiles - walk.t), walk.left)), at0, total, grid);
    fence_proxy_async_smem();
  }

  for (uint32_t it = 0;; ++it) {
    const int buf = it & 1;
    if (it > 0 && !wait_or_stop(&s.q_full[buf], ((it - 1) >> 1) & 1, &s.stop, a.status)) bad = true;
    if (threadIdx.x < 128) s.poison[threadIdx.x] = kKvNoToken;
    if (bar_any(8, kAll, bad)) break;
    const ItemInfo<RT>& info = s.item[buf];
    const int tiles = uniform(info.tiles);
    if (tiles == 0) break;
    const int lo_pos = info.lo_pos, hi_pos = info.hi_pos;

    float o[RT], l[RT], m[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      o[r] = 0.0f;
      l[r] = 0.0f;
      m[r] = kUnset;
    }
    float vref = 0.0f, inv_vref = 0.0f;  // largest value scale when references were last set, kProbScale / it
    float mine = kUnset;                 // reference of row `lane`
    float peak = kNegInf;                // of row `lane`: no score was higher where references were set
    int rest = C::kRun;                  // tiles until the references are looked at
    bool pending = false;                // a product runs that was not waited for
    bool held = false;                   // TMEM holds output not yet in o[]
    bool issued = false;                 // this tile's scores are under way
    // Waits for the last tile's output: its stage is given back then.
    auto settle = [&]() {
      if (pending && !wait_or_stop(&s.empty[last_st], last_turn, &s.stop, a.status)) bad = true;
      pending = false;
    };
    // Moves what TMEM holds to o[].
    auto flush = [&]() {
      if (!held) return;
      held = false;
      __syncwarp();
      tc_fence_after_sync();
      float x[RT];
      tmem_rows<C, true>(tm_o + lane_addr, x);
#pragma unroll
      for (int r = 0; r < RT; ++r) o[r] += x[r];
    };

    for (int i = (W - g0 % W + wg) % W; i < tiles; i += W) {
      const uint32_t g = g0 + i;
      const uint32_t st = g % C::kStages;
      const uint32_t turn = (g / C::kStages) & 1;
      if (!issued && warp == 3) {
        if (!wait_or_stop(&s.full[st], turn, &s.stop, a.status)) bad = true;
        __syncwarp();
        issue_scores(st, buf);
      }
      // The load (for its description) and the scores, asked for together.
      const bool there = mbar_test(&s.full[st], turn), scored = mbar_test(&s.s_bar[wg], phase);
      if (!there && !wait_or_stop(&s.full[st], turn, &s.stop, a.status)) bad = true;
      const StageMeta& meta = s.meta[st];
      const int pos = meta.base[my_slot] + my_off;
      const float k_mul = meta.ks[my_slot], v_scale = meta.vs[my_slot];
      const bool masks = pos > lo_pos;
      if (masks)
        clean_value_row<D>(ring + st * C::kStageBytes + kKvTile * D, t, pos, pos > hi_pos, s.poison);
      if (!scored && !wait_or_stop(&s.s_bar[wg], phase, &s.stop, a.status)) bad = true;
      phase ^= 1;
      __syncwarp();
      tc_fence_after_sync();
      float e[RT];
      // e = x - m, or x itself.
      auto scores = [&](bool relative) {
        tmem_rows<C, false>(tm_s + lane_addr, e);
#pragma unroll
        for (int r = 0; r < RT; r += 2) {
          const F2 f = f2(info.row_mul[r], info.row_mul[r + 1]) * f2(k_mul, k_mul);
          const F2 base = relative ? f2(-m[r], -m[r + 1]) : f2(0.0f, 0.0f);
          f2_get(fma2(f2(e[r], e[r + 1]), f, base), e[r], e[r + 1]);
        }
        if (masks) {
#pragma unroll
          for (int r = 0; r < RT; ++r)
            if (pos > info.row_pos[r]) e[r] = kNegInf;
        }
      };
      scores(true);
      tc_fence_before_sync();
      float top = kNegInf;
#pragma unroll
      for (int r = 0; r < RT; ++r) top = fmaxf(top, e[r]);
      float v_mul = v_scale * inv_vref;
      const bool due = --rest == 0;
      if (bar_any(1 + wg, 128, due || top + fmaxf(log2_approx(v_mul), 7.0f - kRange) > kMaxCode ||
                                   (vref == 0.0f && v_scale > 0.0f))) {
        // Each row's largest weight in this tile: a score plus its value scale's
        // logarithm. (Scores alone where they may pass 2^24, products of two
        // codes being below 2^17.7: they have no steps below 1 then.)
        scores(false);
        const float vnow = fmaxf(vref, meta.vmax);
        const float mul = warp_max(lane < RT ? fabsf(info.row_mul[lane]) : 0.0f) * k_mul;
        const float lv = mul < 0.5f ? fmaxf(log2_approx(v_scale) - log2_approx(vnow), -kRange) : 0.0f;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const float v = warp_max(e[r] + lv);
          if (lane == r) top = v;
        }
        const float spread = warp_max(v_scale > 0.0f ? -lv : 0.0f);
        if (lane < RT) s.red[wg][lane][warp] = top;
        if (lane == 0) s.spread[wg][warp] = spread;
        tc_fence_before_sync();
        bar_sync(1 + wg, 128);
        // Lane r of every warp finds row r's reference.
        float to = mine;
        if (lane < RT) {
          const float4 v = *reinterpret_cast<const float4*>(s.red[wg][lane]);
          const float4 k = *reinterpret_cast<const float4*>(s.spread[wg]);
          const float here = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
          peak = fmaxf(peak, here + fmaxf(fmaxf(k.x, k.y), fmaxf(k.z, k.w)));
          const float want = fmaxf(here + kMargin, peak - kRange);
          if (here != kNegInf && (want > mine || want < mine - kSlack)) to = want;
        }
        if (__any_sync(0xFFFFFFFFu, to != mine) || vnow != vref) {
          settle();
          flush();
          const float less = vref > 0.0f ? __fdividef(vref, vnow) : 1.0f;
          if (lane < RT) {
            s.moved[wg][lane] = to;
            s.alpha[wg][lane] = exp2_approx(mine - to);
          }
          mine = to;
          __syncwarp();
#pragma unroll
          for (int r = 0; r < RT; r += 4) {
            const float4 mn = *reinterpret_cast<const float4*>(&s.moved[wg][r]);
            const float4 f = *reinterpret_cast<const float4*>(&s.alpha[wg][r]);
            m[r] = mn.x, m[r + 1] = mn.y, m[r + 2] = mn.z, m[r + 3] = mn.w;
            l[r] *= f.x, l[r + 1] *= f.y, l[r + 2] *= f.z, l[r + 3] *= f.w;
            o[r] *= f.x * less, o[r + 1] *= f.y * less, o[r + 2] *= f.z * less, o[r + 3] *= f.w * less;
          }
          vref = vnow;
          inv_vref = vref > 0.0f ? __fdividef(kProbScale, vref) : 0.0f;
          v_mul = v_scale * inv_vref;
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) e[r] -= m[r];
        rest = C::kRun;
      }
      // The scores have been read: the next tile's may overwrite them.
      issued = false;
      if (warp == 3 && i + W < tiles) {
        const uint32_t g2 = g + W, st2 = g2 % C::kStages;
        issued = __all_sync(0xFFFFFFFFu, mbar_test(&s.full[st2], (g2 / C::kStages) & 1));
        if (issued) issue_scores(st2, buf);
      }
      if (pending && mbar_test(&s.empty[last_st], last_turn)) pending = false;  // asked early: by now it is done
      uint32_t codes[N / 4];
#pragma unroll
      for (int r = 0; r < RT; r += 2) {
        float p0 = exp2_approx(e[r]), p1 = exp2_approx(e[r + 1]);
        F2 p = f2(p0, p1);
        f2_get(f2(l[r], l[r + 1]) + p, l[r], l[r + 1]);
        F2 y = p * f2(v_mul, v_mul);
#pragma unroll
        for (int term = 0; term < C::T; ++term) {
          f2_get(y, p0, p1);
          uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
          if (term < C::T - 1) {
            // 4 significant bits: cut (T = 3) or rounded half up (T = 2), and to
            // e4m3's smallest step (24576 has steps of 2^-9), so that what the
            // code leaves goes to the next term, whole.
            b0 = (b0 + (C::T == 2 ? 0x80000u : 0u)) & 0xFFF00000u;
            b1 = (b1 + (C::T == 2 ? 0x80000u : 0u)) & 0xFFF00000u;
            const F2 cut = f2(__uint_as_float(b0), __uint_as_float(b1)) + f2(24576.0f, 24576.0f) + f2(-24576.0f, -24576.0f);
            f2_get(cut, p0, p1);
            b0 = __float_as_uint(p0);
            b1 = __float_as_uint(p1);
            const float up = C::T == 3 && term == 0 ? 8.0f : 16.0f;
            y = fma2(cut, f2(-up, -up), y * f2(up, up));
          }
          const uint32_t pair = e4m3x2(__uint_as_float(b0), __uint_as_float(b1));
          const int col = term * RT + r;
          if (col % 4 == 0) codes[col / 4] = pair;
          else codes[col / 4] |= pair << 16;
        }
      }
      // The product before this one has to be done with the probabilities' buffer.
      settle();
#pragma unroll
      for (int c = 0; c < C::T * RT; c += 16) {
        uint8_t* const to = p_buf + c * kKvTile + t * 16;
        if (C::T * RT - c >= 16)
          *reinterpret_cast<uint4*>(to) = make_uint4(codes[c / 4], codes[c / 4 + 1], codes[c / 4 + 2], codes[c / 4 + 3]);
        else
          for (int k = 0; k < (C::T * RT - c) / 4; ++k) reinterpret_cast<uint32_t*>(to)[k] = codes[c / 4 + k];
      }
      tc_fence_before_sync();
      fence_proxy_async_smem();
      bar_sync(1 + wg, 128);
      if (warp == 0) {
        tc_fence_after_sync();
        const uint64_t va = smem_desc_rows<D>(ring_addr + st * C::kStageBytes + kKvTile * D);
        const uint64_t pa = smem_desc_tokens(p_addr);
        const uint32_t add = uniform(static_cast<uint32_t>(held));
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < kKvTile / 32; ++ks)
            mma_f8_ss(tm_o, va + ks * (32 * D / 16), pa + ks * (512 / 16), idesc_f8(N, true), ks > 0 ? 1u : add);
          mma_commit(&s.empty[st]);
        }
        __syncwarp();
      }
      pending = held = true;
      last_st = st;
      last_turn = turn;
    }
    settle();
    flush();
    g0 += tiles;

    // Join the warpgroups. The sums over the tokens first: in each step half
    // of a lane's rows go to its partner, until a lane has one row.
    {
#pragma unroll
      for (int d = 16; d > 0; d /= 2) {
        const bool up = lane & d;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          if (r < RT * d / 32) {
            const int o2 = r + RT * d / 32;
            const float give = up ? l[r] : l[o2];
            l[r] = (up ? l[o2] : l[r]) + __shfl_xor_sync(0xFFFFFFFFu, give, d);
          }
        }
        if (RT * d < 32) l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], d);
      }
      if (lane % (32 / RT) == 0) s.red[wg][lane / (32 / RT)][warp] = l[0];
      if (t < RT) {
        s.ml[0][wg][t] = mine;
        s.moved[wg][t] = fmaxf(mine, peak);
      }
    }
    bar_sync(8, kAll);
    // Then the common reference, and each warpgroup's weight against it. (At least
    // the largest score: sums are large where a reference went below it.)
    if (t < RT) {
      float mx = s.moved[0][t];
#pragma unroll
      for (int w = 1; w < W; ++w) mx = fmaxf(mx, s.moved[w][t]);
      s.ml[1][wg][t] = exp2_approx(s.ml[0][wg][t] - mx);
      if (wg == 0) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float4 v = *reinterpret_cast<const float4*>(s.red[w][t]);
          sum += ((v.x + v.y) + (v.z + v.w)) * exp2_approx(s.ml[0][w][t] - mx);
        }
        s.mx[t] = mx;
        s.sum[t] = sum;
        s.inv[t] = __fdividef(1.0f, sum);
      }
    }
    bar_sync(1 + wg, 128);
    float* const join = reinterpret_cast<float*>(p_smem);
    const int rows = info.rows, part = info.slot;
#pragma unroll
    for (int r0 = 0; r0 < RT; r0 += C::kJoinRows) {
      if (r0 > 0) bar_sync(8, kAll);
      if (t < D) {
#pragma unroll
        for (int r = 0; r < C::kJoinRows; ++r)
          join[(wg * C::kJoinRows + r) * D + t] = o[r0 + r] * s.ml[1][wg][r0 + r] * (vref * (1.0f / kProbScale));
      }
      bar_sync(8, kAll);
      // Four dimensions of a row a thread.
      for (int c = threadIdx.x; c < C::kJoinRows * (D / 4); c += kAll) {
        const int row = c / (D / 4), r = r0 + row, d = c % (D / 4) * 4;
        if (r >= rows) break;
        float4 v = *reinterpret_cast<const float4*>(&join[row * D + d]);
#pragma unroll
        for (int w = 1; w < W; ++w) {
          const float4 u = *reinterpret_cast<const float4*>(&join[(w * C::kJoinRows + row) * D + d]);
          v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        const int4 bad_from = *reinterpret_cast<const int4*>(&s.poison[d]);
        const int row_pos = info.row_pos[r];
        const int64_t at = info.row_at[r];
        const float sum = s.sum[r], inv = s.inv[r], mx = s.mx[r], nan = __int_as_float(0x7FC00000);
        if (row_pos >= bad_from.x) v.x = nan;
        if (row_pos >= bad_from.y) v.y = nan;
        if (row_pos >= bad_from.z) v.z = nan;
        if (row_pos >= bad_from.w) v.w = nan;
        if (part >= 0) {
          float* const to = part_row(a, part, rows, r);
          *reinterpret_cast<float2*>(to + d) = make_float2(v.x, v.y);
          *reinterpret_cast<float2*>(to + d + 2) = make_float2(v.z, v.w);
          if (d == 0) *reinterpret_cast<float2*>(to + D) = row_pos < 0 ? make_float2(kUnset, 0.0f) : make_float2(mx, sum);
        } else if (at >= 0) {
          const bool none = row_pos < 0 || sum == 0.0f;
          v = none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
          uint2 packed;
          if (a.bf16) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
            packed = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
          } else {
            const __half2 x = __floats2half2_rn(v.x, v.y), y = __floats2half2_rn(v.z, v.w);
            packed = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
          }
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * D + d) = packed;
          if (a.lse && d == 0) a.lse[at] = none ? kNegInf : mx * 0.6931471805599453f + logf(sum);
        }
      }
    }
    bar_sync(8, kAll);
    if (threadIdx.x == 0) mbar_arrive(&s.q_empty[buf]);
  }
}

// This CTA's share of all tiles, [total c / grid, total (c + 1) / grid), and
// the item that its first tile belongs to. An item counts item_cost tiles more
// than it has, in front of them; lo is given as the first tile's place. Every item of a list has the same
// tiles; up to 32 query tiles are one to a lane of every warp; more are dealt
// to the calling threads: kThreads of them, whole warps from kFirst on (by way
// of scan and shared, in shared memory, and barrier kBarrier).
template <int kThreads, int kFirst, int kBarrier>
__device__ __forceinline__ void find_share(const AttendArgs& a, int64_t* scan, Start& shared, Start& start,
                                           int64_t& total, int64_t& lo, int64_t& hi, int& grid) {
  const int tid = threadIdx.x - kFirst, warp = tid / 32, lane = tid % 32;
  const int entries = a.c.B * a.n_qt, heads = a.c.Hkv;
  auto share = [&](int64_t tiles) {
    total = tiles * heads;
    grid = static_cast<int>(min(static_cast<int64_t>(gridDim.x), total));
    const int cta = blockIdx.x;
    lo = hi = 0;
    if (cta < grid) {
      lo = divide(total * cta, grid);
      hi = divide(total * (cta + 1), grid);
    }
    start.walk.left = hi - lo;
  };
  // The walk starts in the item of entry e, whose tiles begin at `at`.
  auto begin = [&](int e, const Entry& en, int64_t at) {
    const int each = en.tiles + a.item_cost;
    const int64_t h = divide(lo - at, each);
    start.walk.e = e;
    start.walk.h = static_cast<int32_t>(h);
    start.walk.t = static_cast<int32_t>(lo - at - h * each) - a.item_cost;
    start.entry = en;
  };
  if (a.fixed > 0) {
    const int64_t each = static_cast<int64_t>(a.fixed) * heads;
    share(static_cast<int64_t>(entries) * a.fixed);
    const int64_t e = divide(lo, each);
    begin(static_cast<int>(e), entry_of(a, static_cast<int>(e)), e * each);
  } else if (entries <= 32) {
    Entry mine{};
    if (lane < entries) mine = entry_of(a, lane);
    const int units = lane < entries ? mine.tiles + a.item_cost : 0;
    int64_t before = units;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, before, d);
      if (lane >= d) before += v;
    }
    share(__shfl_sync(0xFFFFFFFFu, before, 31));
    before = (before - units) * heads;
    const int e = __popc(__ballot_sync(0xFFFFFFFFu, lane < entries && before <= lo)) - 1;
    Entry en;
    en.b = __shfl_sync(0xFFFFFFFFu, mine.b, e);
    en.j0 = __shfl_sync(0xFFFFFFFFu, mine.j0, e);
    en.nq = __shfl_sync(0xFFFFFFFFu, mine.nq, e);
    en.first_pos = __shfl_sync(0xFFFFFFFFu, mine.first_pos, e);
    en.last_pos = __shfl_sync(0xFFFFFFFFu, mine.last_pos, e);
    en.tiles = __shfl_sync(0xFFFFFFFFu, mine.tiles, e);
    begin(e, en, __shfl_sync(0xFFFFFFFFu, before, e));
  } else {
    const int64_t per = (entries + kThreads - 1) / kThreads;
    const int64_t e0 = min(per * tid, static_cast<int64_t>(entries)), e1 = min(e0 + per, static_cast<int64_t>(entries));
    int64_t sum = 0;
    Entry mine{};
    for (int64_t e = e0; e < e1; ++e) {
      mine = entry_of(a, static_cast<int>(e));
      sum += mine.tiles + a.item_cost;
    }
    int64_t before = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, before, d);
      if (lane >= d) before += v;
    }
    if (lane == 31) scan[warp] = before;
    bar_sync(kBarrier, kThreads);
    int64_t all = 0;
    before -= sum;
#pragma unroll 1
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += scan[w];
      all += scan[w];
    }
    share(all);
    int64_t at = before * heads;
    if (at <= lo && lo < at + sum * heads) {
      int64_t e = e0;
      if (per > 1)
        for (;; ++e) {
          mine = entry_of(a, static_cast<int>(e));
          const int64_t units = static_cast<int64_t>(mine.tiles + a.item_cost) * heads;
          if (lo < at + units) break;
          at += units;
        }
      begin(static_cast<int>(e), mine, at);
      shared = start;
    }
    bar_sync(kBarrier, kThreads);
    start = shared;
    start.walk.left = hi - lo;
  }
  skip_cost(start.walk);
  lo = hi - start.walk.left;
}

// -------------------------------------------------------------- the kernel
template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    kv_attend_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ AttendArgs a) {
  extern __shared__ uint8_t raw[];
  uint8_t* const ring = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* const q_smem = ring + C::kStages * C::kStageBytes;
  uint8_t* const p_smem = q_smem + 2 * C::kQBytes;
  AttendShared<C>& s = *reinterpret_cast<AttendShared<C>*>(p_smem + C::kPRegion);
  const int tid = threadIdx.x, warp = tid / 32;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&s.full[i], 2);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.q_full[i], 1);
      mbar_init(&s.q_empty[i], 1);
    }
    for (int i = 0; i < C::W; ++i) {
      mbar_init(&s.s_bar[i], 1);
    }
    s.stop = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // The service warps find the CTA's share while the warpgroups enter their code:
  // its first instructions come from a far cache (1 us of a call's start).
  constexpr int kService = C::W * 128;
  if (warp < C::W * 4) {
    attend_consume<C>(a, s, ring, q_smem, p_smem);
  } else {
    // What is above overlaps the end of the work before this launch.
    pdl_wait();
    fence_proxy_async_global();  // its plain stores, before this kernel's bulk loads
    // The accumulators' memory is asked for only now, and later kernels of the
    // stream may start only once every CTA has it: a kernel that waits for this
    // one, or that this one waits for, then never holds what the other needs.
    if (warp == C::W * 4) {
      tmem_alloc(&s.tmem, C::kTmemCols);
      tmem_relinquish();
    }
    if (tid == kService) a.jobs[4 * blockIdx.x] = -1;
    Start start{};
    int64_t total, lo, hi;
    int grid;
    find_share<C::kThreads - kService, kService, 10>(a, s.scan, s.share.start, start, total, lo, hi, grid);
    if (tid == kService) {
      s.share.start = start;
      s.share.lo = lo;
      s.share.hi = hi;
      s.share.total = total;
      s.share.grid = grid;
    }
    tc_fence_before_sync();
    bar_sync(9, C::kThreads);
    tc_fence_after_sync();
    pdl_launch_dependents();
    if (hi > lo) {
      if (warp < C::W * 5) attend_produce<C>(a, &tm_k, &tm_v, s, ring, start, warp - C::W * 4);
      else attend_queries<C>(a, s, q_smem, start, lo - start.walk.t, total, grid);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == C::W * 4) tmem_dealloc(s.tmem, C::kTmemCols);
}

// Launch with the given tensor maps on the current device; grid CTAs.
template <int D, int RT, int T>
cudaError_t attend_form(const CUtensorMap& tk, const CUtensorMap& tv, const AttendArgs& a, int grid, int device,
                        cudaStream_t stream) {
  using C = AttendCfg<D, RT, T>;
  constexpr int smem = 1024 + C::kStages * C::kStageBytes + 2 * C::kQBytes + C::kPRegion +
                       static_cast<int>(sizeof(AttendShared<C>));
  static_assert(smem <= 227 * 1024, "shared memory");
  // Set when a form is first used on a device: loading all of them with the
  // library would slow down the first call of programs that use none.
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << device;
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kv_attend_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  return launch_pdl(kv_attend_kernel<C>, dim3(grid), dim3(C::kThreads), smem, stream, tk, tv, a);
}

// All row counts of one head size and term count (kv_attend_d*_t*.cu).
template <int D, int T>
cudaError_t attend_rows(int rt, const CUtensorMap& tk, const CUtensorMap& tv, const AttendArgs& a, int grid,
                        int device, cudaStream_t stream) {
  switch (rt) {
    case 4: return attend_form<D, 4, T>(tk, tv, a, grid, device, stream);
    case 8: return attend_form<D, 8, T>(tk, tv, a, grid, device, stream);
    case 16: return attend_form<D, 16, T>(tk, tv, a, grid, device, stream);
    default: return attend_form<D, 32, T>(tk, tv, a, grid, device, stream);
  }
}
using AttendLaunch = cudaError_t (*)(int rt, const CUtensorMap& tk, const CUtensorMap& tv, const AttendArgs& a,
                                     int grid, int device, cudaStream_t stream);
cudaError_t attend_d64_t2(int, const CUtensorMap&, const CUtensorMap&, const AttendArgs&, int, int, cudaStream_t);
cudaError_t attend_d64_t3(int, const CUtensorMap&, const CUtensorMap&, const AttendArgs&, int, int, cudaStream_t);
cudaError_t attend_d128_t2(int, const CUtensorMap&, const CUtensorMap&, const AttendArgs&, int, int, cudaStream_t);
cudaError_t attend_d128_t3(int, const CUtensorMap&, const CUtensorMap&, const AttendArgs&, int, int, cudaStream_t);

}  // namespace qsa
