// kv_attend_many.cuh - attention of many query rows over the whole paged 8-bit
// cache: a chunk of a prompt. The formulas are kv_attend_kernel.cuh's.
//
// With hundreds of rows on the same tokens the products are no longer bound by
// reading the cache, so here the rows are the M = 128 operand, and the cache
// is converted to 16 bits once for all rows of a CTA, exactly (every e4m3
// value is an fp16 and a bf16 value; the block's scales stay outside):
//   scores         queries (as they are) times key codes, kind::f16, in the
//                  type of the call;
//   output         probabilities times value codes, in fp16. Of fp16 calls the
//                  probabilities go in as two terms, the first 11 bits and
//                  what they leave (off by 2^-22 of each): one alone would add
//                  an error as large as the result's rounding. Of bf16 calls
//                  one term (2^-11) is a quarter of it.
// A thread owns a row: maximum, sum and rescaling need no other thread. Its
// reference follows the largest score (where value scales lie far apart, the
// largest score plus logarithm of the value scale), but only once it is 2^8 too
// low: the probabilities of fp16 have the range for that, and the output in
// tensor memory is then seldom touched before the end of the item.
//
// One CTA an SM takes two tiles of 128 rows (consecutive queries of a
// sequence, the R heads of a KV head each) through the same key tiles of 128
// tokens. Two warpgroups have a row tile each; one converts keys and values
// into two buffers each; a warp issues the products, those of one row tile
// under the exponentials of the other; and a warp looks pages and scales up
// ahead. The probabilities take the place of the
// scores in tensor memory (M operand of the second product), 32 tokens at a
// time. Codes are loaded by plain 16-byte loads, a tile ahead of their use:
// they pass through registers for the conversion in any case.
//
// The tiles of a call are dealt to CTAs as in kv_attend_kernel.cuh; parts of
// an item lie in the workspace with a row's values 256 floats apart, so that
// a warp's rows make whole lines.
//
// What bounds it: the products take 3,700 of the 5,100 cycles of a pair of row
// tiles and 128 tokens at D = 128 (fp16), the rest is waiting for
// probabilities; at D = 64 the latency of tensor memory reads and barriers (no
// pipe above 42%, an instruction in 54% of the cycles). Measured with the join,
// 32 heads on 8 KV heads, 4,096 queries over 32,768 tokens: fp16 2,157 us,
// 956 TFLOP/s, bf16 1,882 us, 1,096 TFLOP/s; over their own 4,096 tokens 197 and
// 184 us. 2,048 queries of 64 dimensions over 32,768 tokens: fp16 911 us,
// 585 TFLOP/s, bf16 749 us.
#pragma once

#include "kv_attend_kernel.cuh"

namespace qsa {

constexpr int kManyRows = 128;     // of a row tile, two a CTA
constexpr int kManyRing = 4;       // tiles that are looked up ahead
constexpr int kManyThreads = 448;  // 2 x 4 warps of rows, 4 converting, 1 issuing products, 1 looking up
constexpr int kManyItemCost = 3;   // an item's queries and results, and its tiles' start, in tiles
constexpr float kManyLag = 8.0f;   // log2 that a reference may fall behind
constexpr float kManyNear = 6.0f;  // log2 between value scales that costs probabilities nothing
constexpr float kFine = 16777216.0f;  // scores beyond this have no steps below 1
constexpr float kManyScale = 64.0f;  // of a probability 1 at the largest value scale: 2^14 at most

// Places for scores in tensor memory: 128 columns each beside the two outputs.
// With three of them the scores of a row tile's next key tile are there when
// its warpgroup has done with the last one's.
__host__ __device__ constexpr int many_buffers(int D) { return (512 - 2 * D) / 128; }

struct ManyMeta {
  alignas(16) float ks[8], vs[8];  // key and value scales of 16 tokens each
  alignas(16) float lv[8];         // log2 of the value scales against vmax, -kRange at least
  alignas(16) int32_t page[8];     // -1: no block
  float vmax, shift;               // the largest value scale of the item so far; log2 of its growth here
  uint32_t holes;                  // bit i: tokens 16 i .. 16 i + 15 have no block; bit 8: a value
                                   // scale is below 2^-kManyNear of vmax
};

template <int D>
struct ManyShared {
  ManyMeta meta[kManyRing];
  alignas(16) int32_t poison[kManyRing][D];  // of item i in i % kManyRing: first position with a NaN value code
  int32_t poisoned[kManyRing];
  float row_mul[2][kManyRows];
  uint64_t meta_full[kManyRing], meta_empty[kManyRing];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t q_full[2], s_full[many_buffers(D)], p_full[many_buffers(D)], o_full[2];
  int64_t scan[4];
  Share share;
  uint32_t tmem, stop;
};

// Value `col` of row r (of 256) of a partial result: D outputs, reference, sum.
template <int D>
__device__ __forceinline__ float* many_part(const AttendArgs& a, int slot, int col, int r) {
  return a.parts + (static_cast<int64_t>(slot) * (D + 2) + col) * (2 * kManyRows) + r;
}

// Instruction descriptor of kind::f16: fp32 D, bf16 or fp16 operands, M = 128,
// B MN-major when asked.
__host__ __device__ constexpr uint32_t idesc_many(int N, bool bf16, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}

// D[tmem] (+)= A[tmem] * B[smem], issued by one thread.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t bf162_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// An item of a CTA's walk: `tiles` tiles of (entry, head) from t on. at: the
// place of its first tile among all tiles and item costs.
struct ManyItem {
  int32_t e, h, t, tiles;
  int64_t at;
};
// f(entry, item) for each of the CTA's items, in the same order in every warp.
template <class F>
__device__ __forceinline__ void many_items(const AttendArgs& a, const Start& start, int64_t lo, F&& f) {
  Walk w = start.walk;
  Entry en = start.entry;
  int en_of = w.e;
  int64_t at = lo - w.t;
  while (w.left > 0) {
    if (en_of != w.e) {
      en = entry_of(a, w.e);
      en_of = w.e;
    }
    const int tiles = static_cast<int>(min(static_cast<int64_t>(en.tiles - w.t), w.left));
    f(en, ManyItem{w.e, w.h, w.t, tiles, at});
    at += en.tiles + a.item_cost;
    step(w, tiles, en.tiles, a.c.Hkv, a.item_cost);
  }
}
// Until the CTA's share is known and the accumulators' memory is there.
template <class S>
__device__ __forceinline__ void many_begin(S& s) {
  tc_fence_before_sync();
  bar_sync(9, kManyThreads);
  tc_fence_after_sync();
  pdl_wait();
  pdl_launch_dependents();
}

// Whether row tile w has rows to work on. With three places for scores both row
// tiles always work (on zeros, if need be): a place's barrier is then waited for
// by the two in turn, each after the other's unit, and none runs ahead of it. (The
// outputs' barriers are each row tile's own; see the wait at an item's last tile.)
template <int D>
__device__ __forceinline__ bool many_active(const AttendArgs& a, const Entry& en, int w) {
  return many_buffers(D) > 2 || en.nq > w * (a.qt / 2);
}

// ------------------------------------------------------------ pages, scales
// One warp; lane i (of 8) looks up tokens 16 i .. of a tile.
template <int D>
__device__ void many_lookup(const AttendArgs& a, ManyShared<D>& s, const Start& start) {
  const int lane = threadIdx.x % 32, i = lane % 8;
  uint32_t g = 0;
  bool bad = false;
  many_items(a, start, 0, [&](const Entry& en, const ManyItem& w) {
    const int part = w.tiles;
    float vmax = 0.0f, room = kRange;  // what shifts may add up to: sums stay in fp32's range
    const int32_t* const table = a.c.page_table + static_cast<int64_t>(en.b) * a.c.max_blocks;
    if (en.last_pos >= a.c.max_blocks * a.c.block) bad = true;  // longer than its page table
    for (int t = 0; t < part; ++t, ++g) {
      const int blk = (w.t + t) * a.spt + i * 16 / a.c.block;
      int page = -1;
      if (blk < a.c.max_blocks && static_cast<int64_t>(blk) * a.c.block <= en.last_pos) {
        page = load_global(table + blk);
        if (page < 0 || page >= a.c.n_pages) {
          bad = true;
          page = -1;
        }
      }
      float ks = 0.0f, vs = 0.0f;
      if (page >= 0) {
        ks = load_global(a.c.k_scale + static_cast<int64_t>(page) * a.c.Hkv + w.h);
        vs = load_global(a.c.v_scale + static_cast<int64_t>(page) * a.c.Hkv + w.h);
      }
      const float vnow = fmaxf(vmax, warp_max(vs)), lnow = log2_approx(vnow);
      const float lv = fmaxf(log2_approx(vs) - lnow, -kRange);
      const float shift = vmax > 0.0f ? fminf(lnow - log2_approx(vmax), room) : 0.0f;
      room -= shift;
      vmax = vnow;
      const bool far = __any_sync(0xFFFFFFFFu, page >= 0 && lv < -kManyNear);
      const uint32_t holes = __ballot_sync(0xFFFFFFFFu, page < 0) & 0xFFu;
      const uint32_t at = g % kManyRing;
      if (g >= kManyRing) wait_or_stop(&s.meta_empty[at], (g / kManyRing + 1) & 1, &s.stop, a.status);
      __syncwarp();
      ManyMeta& m = s.meta[at];
      if (lane < 8) {
        m.ks[i] = ks;
        m.vs[i] = vs;
        m.lv[i] = lv;
        m.page[i] = page;
        if (lane == 0) {
          m.vmax = vmax;
          m.shift = shift;
          m.holes = holes | (far ? 0x100u : 0u);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.meta_full[at]);
    }
  });
  if (bad) atomicOr(a.status, kErrCacheIndex);
}

// -------------------------------------------------------------- conversion
// 16 codes to 16 halves (or bf16), two 16-byte pieces of a row of 128 bytes.
template <bool BF16>
__device__ __forceinline__ void convert16(uint8_t* tile, uint32_t off, const uint4& codes) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2 * i]) : "h"(static_cast<uint16_t>(w[i])));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2 * i + 1]) : "h"(static_cast<uint16_t>(w[i] >> 16)));
  }
  if (BF16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      h[i] = bf162_of(f.x, f.y);
    }
  }
  *reinterpret_cast<uint4*>(tile + swizzled<128>(off)) = make_uint4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<uint4*>(tile + swizzled<128>(off + 16)) = make_uint4(h[4], h[5], h[6], h[7]);
}

// Bits 7, 15, .. where a code is NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// Four warps. A thread takes the same 16 dimensions of kPasses tokens: loads of
// a tile's values go out before its keys are converted, and of the next tile's
// keys before its values are.
template <int D, bool BF16>
__device__ void many_convert(const AttendArgs& a, ManyShared<D>& s, uint8_t* k16, uint8_t* v16, const Start& start) {
  constexpr int kPer = D / 16;                 // threads of a token
  constexpr int kPasses = kKvTile * kPer / 128;
  constexpr int kBytes = kKvTile * D * 2;
  const int t = threadIdx.x % 128, lane = t % 32, warp = t / 32;
  // Eight neighbouring lanes write to eight different 16-byte columns.
  const int c = D == 128 ? (lane & 3) | ((lane >> 4) << 2) : lane & 3;
  const int row0 = D == 128 ? warp * 4 + ((lane >> 2) & 3) : warp * 8 + (lane >> 2);
  const uint32_t off0 = (c / 4) * (kKvTile * 128) + row0 * 128 + (c % 4) * 32;
  uint32_t g = 0, it = 0;
  uint4 key[kPasses], val[kPasses];
  // Unconditional, so that all of a tile's loads are in flight together: where
  // there is no block, page 0 (its scores are masked, its values made zero).
  auto load = [&](const uint8_t* base, const ManyMeta& m, int h, uint4 (&to)[kPasses]) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int row = row0 + p * (kKvTile / kPasses);
      to[p] = load_global(reinterpret_cast<const uint4*>(
          base + max(m.page[row / 16], 0) * a.c.page_stride +
          (static_cast<int64_t>(h) * a.c.block + (row & (a.c.block - 1))) * D + c * 16));
    }
  };
  auto published = [&](uint64_t* bar) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  many_items(a, start, 0, [&](const Entry& en, const ManyItem& w) {
    const int part = w.tiles;
    const int lo_pos = max(en.first_pos, 0), hi_pos = en.last_pos;
    int32_t* const poison = s.poison[it % kManyRing];
    for (int i = 0; i < part; ++i, ++g) {
      const uint32_t at = g % kManyRing, buf = g & 1;
      const ManyMeta& m = s.meta[at];
      if (i == 0) {  // the keys of an item's first tile were not asked for ahead
        wait_or_stop(&s.meta_full[at], (g / kManyRing) & 1, &s.stop, a.status);
        // The lookup of this tile waited for the item that had this poison before.
        if (t < D) poison[t] = kKvNoToken;
        if (t == 0) s.poisoned[it % kManyRing] = 0;
        bar_sync(1, 128);
        load(a.c.k, m, w.h, key);
      }
      load(a.c.v, m, w.h, val);
      if (g >= 2) wait_or_stop(&s.k_empty[buf], ((g >> 1) + 1) & 1, &s.stop, a.status);
#pragma unroll
      for (int p = 0; p < kPasses; ++p)
        convert16<BF16>(k16 + buf * kBytes, off0 + p * (kKvTile / kPasses) * 128, key[p]);
      published(&s.k_full[buf]);
      if (i + 1 < part) {
        const uint32_t next = (g + 1) % kManyRing;
        wait_or_stop(&s.meta_full[next], ((g + 1) / kManyRing) & 1, &s.stop, a.status);
        load(a.c.k, s.meta[next], w.h, key);
      }
      // Values that no row sees are zeros, so that 0 times them is 0; NaN codes
      // that some rows see are zeros too, and noted for the rows that do.
      const int pos0 = (w.t + i) * kKvTile;
      if (pos0 + kKvTile - 1 > lo_pos || m.holes != 0) {
        uint32_t hits = 0;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
          const int pos = pos0 + row0 + p * (kKvTile / kPasses);
          uint4& u = val[p];
          if (pos > hi_pos || m.page[(pos - pos0) / 16] < 0) u = make_uint4(0, 0, 0, 0);
          if (pos > lo_pos && (nan_codes(u.x) | nan_codes(u.y) | nan_codes(u.z) | nan_codes(u.w))) hits |= 1u << p;
        }
        if (hits) s.poisoned[it % kManyRing] = 1;
#pragma unroll 1
        for (; hits != 0; hits &= hits - 1) {
          const int p = __ffs(hits) - 1;
          uint32_t u[4] = {val[0].x, val[0].y, val[0].z, val[0].w};
#pragma unroll
          for (int e = 1; e < kPasses; ++e)
            if (e == p) u[0] = val[e].x, u[1] = val[e].y, u[2] = val[e].z, u[3] = val[e].w;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if ((nan_codes(u[e / 4]) >> (8 * (e % 4))) & 0x80u) {
              u[e / 4] &= ~(0xFFu << (8 * (e % 4)));
              atomicMin(&poison[c * 16 + e], pos0 + row0 + p * (kKvTile / kPasses));
            }
#pragma unroll
          for (int e = 0; e < kPasses; ++e)
            if (e == p) val[e] = make_uint4(u[0], u[1], u[2], u[3]);
        }
      }
      if (g >= 2) wait_or_stop(&s.v_empty[buf], ((g >> 1) + 1) & 1, &s.stop, a.status);
#pragma unroll
      for (int p = 0; p < kPasses; ++p)
        convert16<false>(v16 + buf * kBytes, off0 + p * (kKvTile / kPasses) * 128, val[p]);
      published(&s.v_full[buf]);
      if (lane == 0) mbar_arrive(&s.meta_empty[at]);
    }
    ++it;
  });
}

// ---------------------------------------------------------------- products
// One warp, in a fixed order: units of a row tile and a key tile, the row tiles
// in turn; a unit's output, then the scores of the unit that gets its place.
// Whatever the two warpgroups begin with, one then has its products while the
// other has the exponentials. (With a warp for each row tile both
// fell into step: 8,600 cycles a tile instead of 7,700, at that time.)
template <int D, bool BF16>
__device__ void many_products(const AttendArgs& a, ManyShared<D>& s, uint32_t q_addr, uint32_t k_addr, uint32_t v_addr,
                              const Start& start) {
  constexpr uint32_t kBytes = kKvTile * D * 2, kPanel = kKvTile * 128, kBuffers = many_buffers(D);
  const uint32_t tmem = uniform(s.tmem), tm_out = tmem + kBuffers * 128;
  // Values run along N: the next 64 dimensions a panel further (leading
  // offset), the next 8 tokens 1024 bytes (stride offset).
  const uint64_t v_mn = (smem_desc_rows<128>(0) & ~(0x3FFFull << 16)) | (static_cast<uint64_t>(kPanel >> 4) << 16);
  const bool leader = elect_one();
  uint32_t g0 = 0, it[2] = {0, 0}, n[2] = {0, 0};  // tiles; items and tiles of each row tile so far
  many_items(a, start, 0, [&](const Entry& en, const ManyItem& wk) {
    const bool active[2] = {many_active<D>(a, en, 0), many_active<D>(a, en, 1)};
    const uint32_t end = 2 * (g0 + wk.tiles);
    // Unit u: row tile u % 2 on tile u / 2.
    auto scores = [&](uint32_t u) {
      const uint32_t buf = u / 2 & 1, at = u % kBuffers;
      wait_or_stop(&s.k_full[buf], (u >> 2) & 1, &s.stop, a.status);
      __syncwarp();
      tc_fence_after_sync();
      if (leader) {
        if (u & 1 ? active[1] : active[0]) {
          const uint64_t q_desc = smem_desc_rows<128>(q_addr + (u & 1) * kBytes);
          const uint64_t k_desc = smem_desc_rows<128>(k_addr + buf * kBytes);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t step = ((ks / 4) * kPanel + (ks % 4) * 32) >> 4;
            mma_f16_ss(tmem + at * 128, q_desc + step, k_desc + step, idesc_many(kKvTile, BF16, false), ks > 0);
          }
          mma_commit(&s.s_full[at]);
          mma_commit(&s.k_empty[buf]);
        } else {
          mma_commit(&s.s_full[at]);
          mbar_arrive(&s.k_empty[buf]);
        }
      }
      __syncwarp();
    };
#pragma unroll
    for (int w = 0; w < 2; ++w)
      if (active[w]) wait_or_stop(&s.q_full[w], it[w]++ & 1, &s.stop, a.status);
#pragma unroll 1
    for (uint32_t u = 2 * g0; u < min(end, 2 * g0 + kBuffers); ++u) scores(u);
#pragma unroll 1
    for (uint32_t u = 2 * g0; u < end; ++u) {
      const uint32_t w = u & 1, buf = u / 2 & 1, at = u % kBuffers;
      wait_or_stop(&s.p_full[at], (u / kBuffers) & 1, &s.stop, a.status);
      wait_or_stop(&s.v_full[buf], (u >> 2) & 1, &s.stop, a.status);
      __syncwarp();
      tc_fence_after_sync();
      const bool work = w ? active[1] : active[0];
      if (leader) {
        if (work) {
          const uint64_t v_desc = v_mn | ((v_addr + buf * kBytes) >> 4);
          const uint32_t tm_o = tm_out + w * D;
#pragma unroll
          for (int ks = 0; ks < kKvTile / 16; ++ks) {
            const uint32_t p_at = tmem + at * 128 + (ks / 2) * 32 + (ks % 2) * 8;
            mma_f16_ts(tm_o, p_at, v_desc + ks * (2048 >> 4), idesc_many(D, false, true), u / 2 > g0 || ks > 0);
            if (!BF16) mma_f16_ts(tm_o, p_at + 16, v_desc + ks * (2048 >> 4), idesc_many(D, false, true), 1u);
          }
          mma_commit(&s.o_full[w]);
          mma_commit(&s.v_empty[buf]);
        } else {
          mbar_arrive(&s.v_empty[buf]);
        }
      }
      __syncwarp();
      // Scores take the place of these probabilities.
      if (work) wait_or_stop(&s.o_full[w], (w ? n[1]++ : n[0]++) & 1, &s.stop, a.status);
      if (u + kBuffers < end) scores(u + kBuffers);
    }
    g0 += wk.tiles;
  });
}

// ------------------------------------------------------------------- rows
// The 32 rows of a warp to shared memory, as they are but for a negative
// softmax scale (its sign goes to the queries), infinities (NaN: such a row is
// NaN whatever it sees), and, of bf16 calls, a power of two for each row that
// keeps fp32 scores in range.
//
// Short code counts here and at an item's end: it runs once an item, and its
// instructions come from a far cache, about 15 cycles each.
template <int D, bool BF16>
__device__ __forceinline__ void many_queries(const AttendArgs& a, ManyShared<D>& s, uint8_t* q_smem, const Entry& en,
                                             int h, int w, int j, int head) {
  constexpr int kLanes = D / 8, kEach = 32 / kLanes, kBatch = 8;  // lanes of a row, rows at a time, loads in flight
  const int lane = threadIdx.x % 32, c = lane % kLanes;
  const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
  // A lane finds its own row; rows that are not there load the tile's first
  // query, so that all loads go out together, and are then made zero.
  const bool mine = j < en.nq && en.first_pos + j >= 0 && head >= 0;
  const uint32_t all = __ballot_sync(0xFFFFFFFFu, mine);
  const int64_t mine_at = mine ? static_cast<int64_t>(j) * a.q.sn + static_cast<int64_t>(head) * a.q.sh : 0;
  const uint16_t* const base = static_cast<const uint16_t*>(a.q.data) + static_cast<int64_t>(en.b) * a.q.sb +
                               static_cast<int64_t>(en.j0) * a.q.sn + static_cast<int64_t>(h) * a.R * a.q.sh + c * 8;
  const int row0 = threadIdx.x / 32 % 4 * 32;
#pragma unroll 1
  for (int r0 = lane / kLanes; r0 < 32; r0 += kBatch * kEach) {
    uint4 u[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      u[i] = load_global(reinterpret_cast<const uint4*>(base + __shfl_sync(0xFFFFFFFFu, mine_at, r0 + i * kEach)));
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * kEach;
      const uint32_t keep = all >> r & 1 ? 0xFFFFFFFFu : 0u;
      uint32_t x[4] = {(u[i].x ^ flip) & keep, (u[i].y ^ flip) & keep, (u[i].z ^ flip) & keep, (u[i].w ^ flip) & keep};
      if (BF16) {
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          m = fmaxf(m, fmaxf(fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xFFFF0000u))));
#pragma unroll
        for (int d = 1; d < kLanes; d *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        const float t = pow2_scale(m);
        const float inv = __uint_as_float((254u << 23) - __float_as_uint(t));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo = __uint_as_float(x[e] << 16) * inv, hi = __uint_as_float(x[e] & 0xFFFF0000u) * inv;
          lo = fmaf(lo, 0.0f, lo);
          hi = fmaf(hi, 0.0f, hi);
          x[e] = bf162_of(lo, hi);
        }
        if (c == 0) s.row_mul[w][row0 + r] = t;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          __half2 v = *reinterpret_cast<__half2*>(&x[e]);
          v = __hfma2(v, __half2(__half(0.0f), __half(0.0f)), v);
          x[e] = *reinterpret_cast<uint32_t*>(&v);
        }
      }
      *reinterpret_cast<uint4*>(q_smem + swizzled<128>((c / 8) * (kKvTile * 128) + (row0 + r) * 128 + (c % 8) * 16)) =
          make_uint4(x[0], x[1], x[2], x[3]);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(&s.q_full[w]);
}

__device__ __forceinline__ float max3(float x, float y, float z) {  // NaN counts as nothing
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// A row's scores of 32 tokens against its reference -> their probabilities'
// sum and, times the value scales, fp16 terms in the place of the scores. MASK:
// of the first and second 16 tokens those up to limit0 and limit1 count, and the
// scores are rounded before the reference is taken off, as they were for the
// reference: where they are so large that this matters, a row's largest is 1.
// (zero is 0, unknown to the compiler, which would join product and difference.)
template <bool BF16, bool MASK>
__device__ __forceinline__ void many_probabilities(uint32_t taddr, float f0, float f1, float v0, float v1, float m,
                                                   int limit0, int limit1, float zero, F2& l) {
  float x[32];
  tmem_ld_cols<32>(taddr, x);
  tmem_ld_wait();
  uint32_t first[16], rest[16];
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float f = e < 16 ? f0 : f1, v = e < 16 ? v0 : v1;
    const F2 y = MASK ? fma2(f2(x[e], x[e + 1]), f2(f, f), f2(zero, zero)) + f2(-m, -m)
                      : fma2(f2(x[e], x[e + 1]), f2(f, f), f2(-m, -m));
    float p0, p1;
    f2_get(y, p0, p1);
    p0 = exp2_approx(p0);
    p1 = exp2_approx(p1);
    if (MASK) {
      const int limit = e < 16 ? limit0 : limit1;
      if (e > limit) p0 = 0.0f;
      if (e + 1 > limit) p1 = 0.0f;
    }
    F2 p = f2(p0, p1);
    l = l + p;
    p = p * f2(v, v);
    f2_get(p, p0, p1);
    if (BF16) {
      first[e / 2] = half2_of(p0, p1);
    } else {
      const float c0 = __uint_as_float(__float_as_uint(p0) & 0xFFFFE000u);
      const float c1 = __uint_as_float(__float_as_uint(p1) & 0xFFFFE000u);
      first[e / 2] = half2_of(c0, c1);
      p = fma2(f2(c0, c1), f2(-1.0f, -1.0f), p);
      f2_get(p, p0, p1);
      rest[e / 2] = half2_of(p0, p1);
    }
  }
  tmem_st16(taddr, first);
  if (!BF16) tmem_st16(taddr + 16, rest);
}

template <int D, bool BF16>
__device__ void many_rows(const AttendArgs& a, ManyShared<D>& s, uint8_t* q_smem, int w) {
  const int warp = uniform(static_cast<int>(threadIdx.x / 32 % 4)), t = threadIdx.x % 128, lane = t % 32;
  const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
  constexpr uint32_t kBuffers = many_buffers(D);
  const int qt = a.qt / 2, jt = t / a.R, j = w * qt + jt;
  uint32_t g = 0, it = 0, n = 0;  // tiles, items, tiles of this row tile so far
  many_begin(s);
  if (s.share.hi <= s.share.lo) return;
  const uint32_t tm_o = uniform(s.tmem) + kBuffers * 128 + w * D + lane_addr;
  const Start start = s.share.start;
  const int64_t lo = s.share.lo, total = s.share.total;
  const int grid = s.share.grid;
  many_items(a, start, lo, [&](const Entry& en, const ManyItem& wk) {
    const int part = wk.tiles;
    const bool active = many_active<D>(a, en, w);
    const bool begins = wk.t == 0, ends = wk.t + part == en.tiles;
    const int slot = begins && ends ? -1 : 2 * static_cast<int>(blockIdx.x) + (begins ? 1 : 0);
    if (begins && !ends && w == 0 && t == 0) {
      int32_t* const job = a.jobs + 4 * blockIdx.x;
      job[0] = wk.e;
      job[1] = wk.h;
      // Tile g belongs to the last CTA c with total * c / grid <= g.
      job[2] = static_cast<int32_t>(divide((wk.at + en.tiles) * grid - 1, total));
    }
    const bool there = t < qt * a.R && j < en.nq && en.first_pos + j >= 0;
    const int row_pos = there ? en.first_pos + j : -1;
    // Smallest position that a row of this tile sees: earlier tiles need no mask.
    const int lo_pos = max(en.first_pos + w * qt, 0);
    float m = kUnset, vref = 0.0f;
    F2 l = f2(0.0f, 0.0f);
    float mul = 0.0f, zero = 0.0f;
    asm volatile("" : "+f"(zero));
    __syncwarp();
    if (active) {
      many_queries<D, BF16>(a, s, q_smem + w * (kKvTile * D * 2), en, wk.h, w, j, t < qt * a.R ? t - jt * a.R : -1);
      mul = fabsf(a.scale_log2) * (BF16 ? s.row_mul[w][t] : 1.0f);
    }
    for (int i = 0; i < part; ++i, ++g) {
      const uint32_t at = g % kManyRing;
      const uint32_t unit = 2 * g + w, buf = unit % kBuffers;  // as in many_products
      wait_or_stop(&s.meta_full[at], (g / kManyRing) & 1, &s.stop, a.status);
      if (!active) {  // keeps its turn, with nothing to do
        wait_or_stop(&s.s_full[buf], (unit / kBuffers) & 1, &s.stop, a.status);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[buf]);
      } else {
        const ManyMeta& meta = s.meta[at];
        const int pos0 = (wk.t + i) * kKvTile;
        const uint32_t holes = meta.holes;
        const bool masked = holes != 0 || pos0 + kKvTile - 1 > lo_pos;
        const float vmax = meta.vmax;
        const uint32_t tm_s = uniform(s.tmem) + buf * 128 + lane_addr;
        wait_or_stop(&s.s_full[buf], (unit / kBuffers) & 1, &s.stop, a.status);
        __syncwarp();
        tc_fence_after_sync();
        // The loops over 32 columns stay loops: unrolled, the code of a tile does
        // not fit the instruction caches (a quarter of all stalls).
        float top = -INFINITY;
        float2 ks = *reinterpret_cast<const float2*>(&meta.ks[0]);  // a step ahead
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float x[32];
          tmem_ld_cols<32>(tm_s + c * 32, x);
          tmem_ld_wait();
          if (masked) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int limit = (holes >> (2 * c + hf)) & 1 ? -1 : row_pos - pos0 - c * 32 - hf * 16;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (e > limit) x[hf * 16 + e] = -INFINITY;
            }
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float mx = max3(x[hf * 16], x[hf * 16 + 1], x[hf * 16 + 2]);
#pragma unroll
            for (int e = 3; e < 15; e += 2) mx = max3(mx, x[hf * 16 + e], x[hf * 16 + e + 1]);
            mx = fmaxf(mx, x[hf * 16 + 15]);
            top = fmaxf(top, mx * (mul * (hf == 0 ? ks.x : ks.y)));
          }
          ks = *reinterpret_cast<const float2*>(&meta.ks[(2 * c + 2) & 7]);
        }
        // Where value scales lie far apart, the row's largest weight: a score plus
        // its value scale's logarithm (scores beyond 2^24, which have no steps
        // below 1, count alone).
        if (holes & 0x100u) {
          float weight = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            float x[16];
            tmem_ld_cols<16>(tm_s + c * 16, x);
            tmem_ld_wait();
            const int limit = (holes >> c) & 1 ? -1 : row_pos - pos0 - c * 16;
            float mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e <= limit) mx = fmaxf(mx, x[e]);
            weight = fmaxf(weight, fmaf(mx, mul * meta.ks[c], meta.lv[c]));
          }
          if (fabsf(top) < kFine) top = weight;
        }
        const bool grow = vmax > vref;
        if (__any_sync(0xFFFFFFFFu, top > m + kManyLag) || grow) {
          // Weights are relative to the largest value scale: a reference moves with it.
          const float base = grow && fabsf(m) < kFine ? m - meta.shift : m;
          const float mn = top > base + kManyLag ? top : base;
          float f = exp2_approx(m - mn);
          l = l * f2(f, f);
          m = mn;
          if (grow) {
            f *= vref > 0.0f ? __fdividef(vref, vmax) : 0.0f;
            vref = vmax;
          }
          if (i > 0) {
            wait_or_stop(&s.o_full[w], (n - 1) & 1, &s.stop, a.status);
            __syncwarp();
            tc_fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              tmem_ld_cols<16>(tm_o + c, o);
              tmem_ld_wait();
              uint32_t u[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * f);
              tmem_st16(tm_o + c, u);
            }
          }
        }
        const bool huge = __any_sync(0xFFFFFFFFu, m > 1048576.0f || (m < -1048576.0f && m != kUnset));
        const float inv = vref > 0.0f ? __fdividef(kManyScale, vref) : 0.0f;
        float2 vs = *reinterpret_cast<const float2*>(&meta.vs[0]);
        // A tile's sum apart: added one by one to a sum that one token above all
        // others made large, the small ones would lose bits each.
        F2 lt = f2(0.0f, 0.0f);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const float f0 = mul * ks.x, f1 = mul * ks.y, v0 = vs.x * inv, v1 = vs.y * inv;
          ks = *reinterpret_cast<const float2*>(&meta.ks[(2 * c + 2) & 7]);
          vs = *reinterpret_cast<const float2*>(&meta.vs[(2 * c + 2) & 7]);
          if (masked || huge) {
            const int limit = row_pos - pos0 - c * 32;
            many_probabilities<BF16, true>(tm_s + c * 32, f0, f1, v0, v1, m, (holes >> (2 * c)) & 1 ? -1 : limit,
                                           (holes >> (2 * c + 1)) & 1 ? -1 : limit, zero, lt);
          } else {
            many_probabilities<BF16, false>(tm_s + c * 32, f0, f1, v0, v1, m, 0, 0, zero, lt);
          }
        }
        l = l + lt;
        // With three places for scores, a warp that has its last tile's scores only
        // knows that the output two tiles back is done: these came after another
        // row tile's. The last tile's output may only be asked for by its parity
        // when the one before it is done, so that one is waited for here: ahead
        // of this warp's arrival, without which the last one cannot be done yet.
        if (kBuffers > 2 && i > 0 && i + 1 == part) wait_or_stop(&s.o_full[w], (n - 1) & 1, &s.stop, a.status);
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[buf]);
        ++n;
      }
      if (i + 1 < part) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.meta_empty[at]);
      }
    }
    if (active) {
      wait_or_stop(&s.o_full[w], (n - 1) & 1, &s.stop, a.status);
      __syncwarp();
      tc_fence_after_sync();
      float l0, l1;
      f2_get(l, l0, l1);
      float sum = l0 + l1, all = 1.0f;
      if (sum > kFine) {  // scores above the weights' reference: into the reference
        const float mn = m + floorf(log2_approx(sum));
        all = exp2_approx(m - mn);
        sum *= all;
        m = mn;
      }
      const bool none = row_pos < 0 || sum == 0.0f;
      const float f = vref * (1.0f / kManyScale) * (slot >= 0 ? all : __fdividef(all, sum));
      const int64_t at = (static_cast<int64_t>(en.b) * a.n + en.j0 + j) * a.Hq + wk.h * a.R + (t - jt * a.R);
      const bool mine = t < qt * a.R && en.j0 + j < a.n;
      float* const part_at = many_part<D>(a, slot, 0, w * kManyRows + t);
      uint16_t* const out_at = static_cast<uint16_t*>(a.out) + at * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        float o[16];
        tmem_ld_cols<16>(tm_o + c, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = none ? 0.0f : o[e] * f;
        if (slot >= 0) {
#pragma unroll
          for (int e = 0; e < 16; ++e) part_at[(c + e) * (2 * kManyRows)] = o[e];
        } else if (mine) {
          uint32_t u[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = BF16 ? bf162_of(o[2 * e], o[2 * e + 1]) : half2_of(o[2 * e], o[2 * e + 1]);
          uint4* const to = reinterpret_cast<uint4*>(out_at + c);
          to[0] = make_uint4(u[0], u[1], u[2], u[3]);
          to[1] = make_uint4(u[4], u[5], u[6], u[7]);
        }
        __syncwarp();
      }
      if (s.poisoned[it % kManyRing] != 0) {
#pragma unroll 1
        for (int c = 0; c < D; ++c)
          if (row_pos >= s.poison[it % kManyRing][c]) {
            if (slot >= 0) part_at[c * (2 * kManyRows)] = __int_as_float(0x7FC00000);
            else if (mine) out_at[c] = BF16 ? 0x7FC0 : 0x7E00;
          }
      }
      if (slot >= 0) {
        *many_part<D>(a, slot, D, w * kManyRows + t) = none ? kUnset : m;
        *many_part<D>(a, slot, D + 1, w * kManyRows + t) = none ? 0.0f : sum;
      } else if (mine && a.lse) {
        a.lse[at] = none ? -INFINITY : m * 0.6931471805599453f + logf(sum);
      }
      tc_fence_before_sync();
    } else if (slot < 0 && t < qt * a.R && en.j0 + j < a.n) {
      // Rows past a sequence's new ones: zeros.
      const int64_t at = (static_cast<int64_t>(en.b) * a.n + en.j0 + j) * a.Hq + wk.h * a.R + (t - jt * a.R);
      for (int c = 0; c < D / 8; ++c)
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at * D)[c] = make_uint4(0, 0, 0, 0);
      if (a.lse) a.lse[at] = -INFINITY;
    } else if (slot >= 0) {
      for (int c = 0; c < D + 2; ++c) *many_part<D>(a, slot, c, w * kManyRows + t) = c == D ? kUnset : 0.0f;
    }
    ++it;
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.meta_empty[(g - 1) % kManyRing]);
  });
}

// -------------------------------------------------------------- the kernel
template <int D, bool BF16>
__global__ void __launch_bounds__(kManyThreads, 1) kv_attend_many_kernel(const __grid_constant__ AttendArgs a) {
  extern __shared__ uint8_t raw[];
  constexpr int kBytes = kKvTile * D * 2;  // a tile of 16-bit rows
  uint8_t* const q_smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* const v16 = q_smem + 2 * kBytes;
  uint8_t* const k16 = v16 + 2 * kBytes;
  ManyShared<D>& s = *reinterpret_cast<ManyShared<D>*>(k16 + 2 * kBytes);
  const int warp = threadIdx.x / 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kManyRing; ++i) {
      mbar_init(&s.meta_full[i], 1);
      mbar_init(&s.meta_empty[i], 12);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.k_full[i], 4);
      mbar_init(&s.k_empty[i], 2);
      mbar_init(&s.v_full[i], 4);
      mbar_init(&s.v_empty[i], 2);
      mbar_init(&s.q_full[i], 4);
      mbar_init(&s.o_full[i], 1);
    }
    for (int i = 0; i < many_buffers(D); ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], 4);
    }
    s.stop = 0;
    fence_mbarrier_init();
  }
  // The converting warps find the CTA's share, the products' warp asks for
  // tensor memory (after the wait, and before later kernels may start: see
  // kv_attend_kernel), and the others enter their code.
  if (warp < 8) {
    many_rows<D, BF16>(a, s, q_smem, warp / 4);
  } else {
    if (warp < 12) {
      pdl_wait();
      if (threadIdx.x == 256) a.jobs[4 * blockIdx.x] = -1;
      Share found{};
      int grid;
      find_share<128, 256, 1>(a, s.scan, s.share.start, found.start, found.total, found.lo, found.hi, grid);
      if (threadIdx.x == 256) {
        found.grid = grid;
        s.share = found;
      }
    } else if (warp == 12) {
      pdl_wait();
      tmem_alloc(&s.tmem, 512);
      tmem_relinquish();
    }
    many_begin(s);
    const Start start = s.share.start;
    if (s.share.hi > s.share.lo) {
      if (warp < 12) many_convert<D, BF16>(a, s, k16, v16, start);
      else if (warp == 12) many_products<D, BF16>(a, s, smem_u32(q_smem), smem_u32(k16), smem_u32(v16), start);
      else many_lookup<D>(a, s, start);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 12) tmem_dealloc(s.tmem, 512);
}

// Joins the parts of an item as kv_combine_kernel does: a lane a row, 32 rows a
// CTA, DIMS dimensions a warp. The warps first find the parts' weights, a part a
// warp in turn; then each adds its dimensions over all parts, in their order.
constexpr int kJoinWarps = 8;
template <int D, int DIMS>
__global__ void __launch_bounds__(32 * kJoinWarps) kv_combine_many_kernel(const __grid_constant__ AttendArgs a) {
  __shared__ float s_f[kKvMaxCtas][32];
  __shared__ float s_max[kJoinWarps][32], s_sum[kJoinWarps][32];
  pdl_wait();
  pdl_launch_dependents();  // after the wait: at most one kernel ahead of the one that runs
  const int c0 = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int t = blockIdx.z * 32 + lane, d0 = (blockIdx.y * kJoinWarps + warp) * DIMS;
  const int4 job = *reinterpret_cast<const int4*>(a.jobs + 4 * c0);
  if (job.x < 0) return;
  const int e = job.x, h = job.y, parts = job.z - c0 + 1, qt = a.qt / 2;
  auto at = [&](int i, int col) { return many_part<D>(a, i == 0 ? 2 * c0 + 1 : 2 * (c0 + i), col, t); };
  float m = -INFINITY;
#pragma unroll 4
  for (int i = warp; i < parts; i += kJoinWarps) {
    const float x = *at(i, D);
    s_f[i][lane] = x;
    m = fmaxf(m, x);
  }
  s_max[warp][lane] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) m = fmaxf(m, s_max[i][lane]);
  float l = 0.0f;
#pragma unroll 4
  for (int i = warp; i < parts; i += kJoinWarps) {
    const float f = exp2_approx(s_f[i][lane] - m);
    s_f[i][lane] = f;
    l += *at(i, D + 1) * f;
  }
  s_sum[warp][lane] = l;
  __syncthreads();
  l = 0.0f;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) l += s_sum[i][lane];
  float o[DIMS];
#pragma unroll
  for (int d = 0; d < DIMS; ++d) o[d] = *at(0, d0 + d) * s_f[0][lane];
  const float* part = at(1, d0);
#pragma unroll 4
  for (int i = 1; i < parts; ++i, part += 2 * (D + 2) * 2 * kManyRows) {
    const float f = s_f[i][lane];
#pragma unroll
    for (int d = 0; d < DIMS; ++d) o[d] += part[d * 2 * kManyRows] * f;
  }
  const int r = t % kManyRows, jt = r / a.R;
  const int b = e / a.n_qt, j = (e - b * a.n_qt) * a.qt + t / kManyRows * qt + jt;
  if (r >= qt * a.R || j >= a.n) return;
  const int64_t row = (static_cast<int64_t>(b) * a.n + j) * a.Hq + h * a.R + (r - jt * a.R);
  uint32_t* const to = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + row * D + d0);
#pragma unroll
  for (int k = 0; k < DIMS / 2; ++k) {
    const float x0 = l == 0.0f ? 0.0f : o[k * 2] / l, x1 = l == 0.0f ? 0.0f : o[k * 2 + 1] / l;
    to[k] = a.bf16 ? bf162_of(x0, x1) : half2_of(x0, x1);
  }
  if (a.lse && d0 == 0) a.lse[row] = l == 0.0f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

// kv_attend_many.cu; one CTA an SM, then the join where items may be split.
cudaError_t launch_attend_many(const AttendArgs& a, int grid, bool split, int device, cudaStream_t stream);

}  // namespace qsa
