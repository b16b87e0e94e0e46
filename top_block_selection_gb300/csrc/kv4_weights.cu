// kv4_weights.cu - the attention weight that each cached token of the 4-bit
// cache gathers:
//     w[h, t] = decay w[h, t] + sum_{j, i} exp(scale q[j, i] . k_t - lse[j, i])
// over the call's rows j that see t and the query heads i of KV head h.
//
// The tokens are the M = 128 operand of the score product, as in
// kv_attend_kernel.cuh, so that a thread owns a token (of 64 dimensions, two) and
// adds its weights up alone: no exchange, no atomics, and results that do not
// depend on timing. The exponent is y c - lse log2(e), with y the scaled product
// and c = scale log2(e): a weight's relative error is the exponent's absolute one,
// 2^-24 of its parts each (2.1e-7 and 3.2e-7 for the measured cases; c in two floats,
// a tenth more time, made no difference that shows beside the others).
//
// One CTA an SM. The tiles of all (sequence, KV head) items are dealt to the
// CTAs in equal contiguous shares. A warp loads keys, scales and weights ahead by
// asynchronous copies, eight make the e4m3 terms of up to kGroups x RT rows, and two
// warpgroups take the tiles in turn, each with a warp that issues its products and
// two places for scores in tensor memory. (One warp for all products took 360
// cycles a tile beside its waits.) More rows than that go over the share's tiles of the item again
// (from L2), adding to what the pass before left.
//
// What bounds it: for a decode step the keys and weights from HBM (64 requests over
// 1,000 to 16,384 tokens, 8 KV heads: 60.7 us, 5.4 TB/s, 81% of a plain copy's rate; the
// rest is the start, the first tiles' chain of lengths, pages and loads). For many
// rows no unit is near its rate (64 rows over 32,805 tokens, 32 heads on 8 KV heads:
// 32.7 us, 524 TFLOP/s; exponentials and products 20% of the cycles each): a
// warpgroup's chain of tensor memory read, exponentials and sums is what a tile
// takes, and the queries' terms are made before the first.
#include "kv_attend_kernel.cuh"

#include <algorithm>

namespace qsa {
namespace {

constexpr int kQueryWarps = 8;
constexpr int kFirstProducer = 10;  // warps: 8 of weights, 2 of products, producers, queries
constexpr int kPlace = 128;      // columns of a place for scores

template <int D_, int RT_, int T_>
struct WeightsCfg : AttendCfg<D_, RT_, T_, true> {
  static constexpr int kProducers = RT_ < 32 ? 4 : 2;  // warps that load, a tile each in turn
  // A stage serves one warpgroup and one producer.
  static constexpr int kStages = RT_ < 32 ? 8 : 6;
  static constexpr int kFirstQuery = kFirstProducer + kProducers;
  static constexpr int kThreads = 32 * (kFirstQuery + kQueryWarps);
  static_assert(kStages % 2 == 0 && kStages % kProducers == 0, "stages");
  static constexpr int kGroups = RT_ < 32 ? 1 : 4;   // of rows, in one pass (fewer rows than 32 are one group)
};

struct WeightsArgs {
  AttendArgs a;      // out, lse, ids, parts, jobs unused; scale_log2 = 1
  const float* lse;
  float* weights;
  float c;           // scale * log2(e)
  float decay;
};

// 16 bytes to shared memory, behind the thread's back.
__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
// Arrives on `bar` when the thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

struct Sequence {
  int32_t len, first, n_new, tiles;  // tokens, slot of the first new one, new ones
};
__device__ __forceinline__ Sequence sequence_of(const AttendArgs& a, int b) {
  const Span s = span_of(a.c, b, a.n);
  Sequence q;
  q.len = min(s.len, a.c.max_blocks * a.c.block);
  q.first = s.first;
  q.n_new = s.n_new;
  q.tiles = (q.len + (1 << a.tile_log2) - 1) >> a.tile_log2;
  return q;
}

template <class C>
struct GroupRows {
  ItemInfo<C::RR> info;
  alignas(16) float c[C::RR], nl[C::RR];  // scale log2(e) times the unit of the row's terms; -lse log2(e)
  alignas(8) uint8_t silent[8];           // of a query warp: a row of it (with lse -inf, or not there) gives no token any weight
};

template <class C>
struct WeightsShared {
  GroupRows<C> rows[2][C::kGroups];
  alignas(16) uint16_t ks[C::kStages][C::kTokens];
  alignas(16) float old[C::kStages][C::kTokens];    // weights before the call
  alignas(16) int64_t row0[C::kStages][C::kSlots];  // of a slot's first token among the weights; -1: no block
  uint64_t k_full[C::kStages], k_empty[C::kStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2][2], s_empty[2][2];
  int64_t scan[C::kThreads / 32];
  int64_t lo, hi, total;
  int32_t b, h, t;  // where the share begins
  uint32_t tmem, stop;
};

// f(sequence number, sequence, head, first tile, tiles) for the items of the CTA's share.
template <class C, class F>
__device__ __forceinline__ void each_item(const AttendArgs& a, const WeightsShared<C>& s, F&& f) {
  int64_t left = s.hi - s.lo;
  int b = s.b, h = s.h, t = s.t;
  while (left > 0 && b < a.c.B) {
    const Sequence q = sequence_of(a, b);
    for (; h < a.c.Hkv && left > 0 && q.tiles > 0; ++h, t = 0) {
      const int part = static_cast<int>(min(static_cast<int64_t>(q.tiles - t), left));
      f(b, q, h, t, part);
      left -= part;
      if (t + part < q.tiles) return;
    }
    ++b;
    h = t = 0;
  }
}

// K columns of scores: their terms added, each 1/16 of the one before, RR columns on.
template <class C, int K>
__device__ __forceinline__ void score_part(uint32_t taddr, float (&x)[K]) {
  float t1[K], t2[K];
  tmem_ld_cols<K>(taddr, x);
  tmem_ld_cols<K>(taddr + C::RR, t1);
  if (C::T == 3) tmem_ld_cols<K>(taddr + 2 * C::RR, t2);
  tmem_ld_wait();
#pragma unroll
  for (int r = 0; r < K; r += 2) {
    F2 sum = f2(t1[r], t1[r + 1]);
    if (C::T == 3) sum = fma2(f2(t2[r], t2[r + 1]), f2(0.0625f, 0.0625f), sum);
    f2_get(fma2(sum, f2(0.0625f, 0.0625f), f2(x[r], x[r + 1])), x[r], x[r + 1]);
  }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    kv4_weights_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ WeightsArgs w) {
  constexpr int PAR = C::PAR, RT = C::RT, kStages = C::kStages, kGroups = C::kGroups;
  constexpr int kThreads = C::kThreads, kProducers = C::kProducers;
  constexpr int kTile = kKvTile * 128;  // bytes of a key tile
  extern __shared__ uint8_t raw[];
  uint8_t* const ring = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* const q_smem = ring + kStages * kTile;
  WeightsShared<C>& s = *reinterpret_cast<WeightsShared<C>*>(q_smem + 2 * kGroups * C::kQBytes);
  const AttendArgs& a = w.a;
  const int tid = threadIdx.x, warp = uniform(tid / 32), lane = tid % 32;

  if (tid < 2 * kGroups) *reinterpret_cast<uint64_t*>(s.rows[tid / kGroups][tid % kGroups].silent) = 0;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.k_full[i], 33);
      mbar_init(&s.k_empty[i], 5);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.q_full[i], kQueryWarps);
      mbar_init(&s.q_empty[i], 10);
      for (int j = 0; j < 2; ++j) {
        mbar_init(&s.s_full[i][j], 1);
        mbar_init(&s.s_empty[i][j], 4);
      }
    }
    s.stop = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tm_k);
  }
  pdl_wait();
  fence_proxy_async_global();  // earlier plain stores, before this kernel's bulk loads
  // Tensor memory is asked for only now, and later kernels of the stream may start
  // only once every CTA has it (see kv_attend_kernel).
  if (warp == 8) {
    tmem_alloc(&s.tmem, 512);
    tmem_relinquish();
  }
  // The share [lo, hi) of all tiles, and the item that it begins in.
  {
    const int B = a.c.B, per = (B + kThreads - 1) / kThreads;
    const int b0 = min(per * tid, B), b1 = min(b0 + per, B);
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) sum += sequence_of(a, b).tiles;
    int64_t before = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, before, d);
      if (lane >= d) before += v;
    }
    if (lane == 31) s.scan[warp] = before;
    __syncthreads();
    int64_t all = 0;
    before -= sum;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += s.scan[i];
      all += s.scan[i];
    }
    const int64_t total = all * a.c.Hkv;
    const int64_t lo = divide(total * blockIdx.x, gridDim.x), hi = divide(total * (blockIdx.x + 1), gridDim.x);
    if (tid == 0) {
      s.lo = lo;
      s.hi = hi;
      if (lo == hi) s.b = B;
    }
    int64_t at = before * a.c.Hkv;
    if (lo < hi && at <= lo && lo < at + sum * a.c.Hkv) {
      for (int b = b0; b < b1; ++b) {
        const int tiles = sequence_of(a, b).tiles;
        const int64_t units = static_cast<int64_t>(tiles) * a.c.Hkv;
        if (lo < at + units) {
          s.b = b;
          s.h = static_cast<int>((lo - at) / tiles);
          s.t = static_cast<int>((lo - at) % tiles);
          break;
        }
        at += units;
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  pdl_launch_dependents();

  const int n_groups = (a.n + a.qt - 1) / a.qt * a.split;  // of rows: a.qt queries, a.R heads
  const int passes = (n_groups + kGroups - 1) / kGroups;
  const int per_pass = min(n_groups, kGroups);

  if (warp < 8) {
    // ------------------------------------------------------- the weights
    const int wg = warp / 4, t = tid % 128;
    const uint32_t lane_addr = static_cast<uint32_t>(warp % 4 * 32) << 16;
    const uint32_t tm = uniform(s.tmem) + wg * 2 * kPlace + lane_addr;
    const int slot = t * PAR / a.c.block, off = t * PAR - slot * a.c.block;
    uint32_t g0 = 0, unit = 0, pc = 0;
    each_item<C>(a, s, [&](int b, const Sequence& q, int h, int t0, int part) {
      for (int pass = 0; pass < passes; ++pass, ++pc) {
        const uint32_t buf = pc & 1;
        // A tile may be the other warpgroup's in the next pass, which adds to what this
        // one stored.
        if (pass > 0) bar_sync(1, 256);
        wait_or_stop(&s.q_full[buf], (pc >> 1) & 1, &s.stop, a.status);
        const int groups = min(per_pass, n_groups - pass * kGroups);
        const int lo_pos = s.rows[buf][0].info.lo_pos;
        for (uint32_t g = g0 + ((g0 ^ wg) & 1); g < g0 + part; g += 2) {
          const uint32_t st = g % kStages;
          wait_or_stop(&s.k_full[st], (g / kStages) & 1, &s.stop, a.status);
          const int pos = ((t0 + static_cast<int>(g - g0)) << a.tile_log2) + t * PAR;
          float k_mul[PAR];
#pragma unroll
          for (int i = 0; i < PAR; ++i)
            k_mul[i] = __uint_as_float(static_cast<uint32_t>(s.ks[st][t * PAR + i]) << 16);
          const int64_t row0 = s.row0[st][slot];
          float* const at = w.weights + row0 + off;
          bool there[PAR];
          float old[PAR], acc[PAR];
#pragma unroll
          for (int i = 0; i < PAR; ++i) {
            there[i] = row0 >= 0 && pos + i < q.len;
            acc[i] = 0.0f;
            old[i] = pass == 0 && w.decay != 0.0f && pos + i < q.first ? s.old[st][t * PAR + i] * w.decay : 0.0f;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.k_empty[st]);
          if (pass > 0) {  // what the pass before left
#pragma unroll
            for (int i = 0; i < PAR; ++i)
              if (there[i]) old[i] = load_global(at + i);
          }
          for (int gr = 0; gr < groups; ++gr, ++unit) {
            const GroupRows<C>& rows = s.rows[buf][gr];
            const uint32_t place = unit & 1;
            wait_or_stop(&s.s_full[wg][place], (unit >> 1) & 1, &s.stop, a.status);
            __syncwarp();
            tc_fence_after_sync();
            // (A score that is not finite would leave NaN, not 0, of a silent row.)
            const bool masks = pos + PAR - 1 > lo_pos || *reinterpret_cast<const uint64_t*>(rows.silent) != 0;
            // A token's rows at a time, of three terms half of 32. (All the code of a
            // unit for each token in turn: it has to stay in the instruction caches.)
            constexpr int kPart = C::RR <= 16 || C::T == 2 ? C::RR : 16;
#pragma unroll 1
            for (int r0 = 0; r0 < RT; r0 += kPart) {
              float e[kPart];
              const int second = PAR == 2 && r0 >= C::RR, r1 = r0 - second * C::RR;  // of an operand row's tokens
              score_part<C, kPart>(tm + place * kPlace + second * C::NQ + r1, e);
              if (r0 + kPart == RT) {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.s_empty[wg][place]);
              }
              const float k = second ? k_mul[PAR - 1] : k_mul[0];
#pragma unroll
              for (int r = 0; r < kPart; r += 2) {
                const F2 y = f2(e[r], e[r + 1]) * f2(k, k);
                const F2 x = fma2(y, f2(rows.c[r1 + r], rows.c[r1 + r + 1]), f2(rows.nl[r1 + r], rows.nl[r1 + r + 1]));
                f2_get(x, e[r], e[r + 1]);
                e[r] = exp2_approx(e[r]);
                e[r + 1] = exp2_approx(e[r + 1]);
              }
              if (masks) {
#pragma unroll
                for (int r = 0; r < kPart; ++r)
                  if (pos + second > rows.info.row_pos[r1 + r]) e[r] = 0.0f;
              }
              F2 sum = f2(e[0], e[1]);
#pragma unroll
              for (int r = 2; r < kPart; r += 2) sum = sum + f2(e[r], e[r + 1]);
              float s0, s1;
              f2_get(sum, s0, s1);
              if (second) acc[PAR - 1] += s0 + s1;
              else acc[0] += s0 + s1;
            }
          }
#pragma unroll
          for (int i = 0; i < PAR; ++i)
            if (there[i]) at[i] = old[i] + acc[i];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.q_empty[buf]);
        g0 += part;
      }
    });
  } else if (warp >= kFirstProducer && warp < C::kFirstQuery) {
    // ------------------------------------------------------- keys, scales
    // Tiles p, p + kProducers, ... of the CTA: one warp's chain of instructions for
    // a tile takes longer (about 800 cycles) than the tile may.
    const int p = warp - kFirstProducer;
    const int spt = a.spt, per_batch = 32 / spt, my_k = lane / spt, my_slot = lane % spt;
    uint32_t g0 = 0;
    bool bad = false, ok = true;
    each_item<C>(a, s, [&](int b, const Sequence& q, int h, int t0, int part) {
      if (load_global(a.c.lens + b) > q.len) bad = true;  // longer than its page table
      const int32_t* const table = a.c.page_table + static_cast<int64_t>(b) * a.c.max_blocks;
      const int y = h * a.c.block / PAR, slab = a.c.block * C::HD;
      for (int pass = 0; pass < passes; ++pass, g0 += part) {
        const int own0 = static_cast<int>((p + kProducers - g0 % kProducers) % kProducers);
        const int own = part > own0 ? (part - own0 + kProducers - 1) / kProducers : 0;
        for (int k0 = 0; k0 < own; k0 += per_batch) {
          const int tiles = min(per_batch, own - k0);
          const int blk = (t0 + own0 + (k0 + my_k) * kProducers) * spt + my_slot;
          int page = -1;
          if (my_k < tiles && static_cast<int64_t>(blk) * a.c.block < q.len) {
            page = load_global(table + blk);
            if (page < 0 || page >= a.c.n_pages) {
              bad = true;
              page = -1;
            }
          }
          for (int i = 0; i < tiles; ++i) {
            const uint32_t g = g0 + own0 + (k0 + i) * kProducers, st = g % kStages;
            if (ok && g >= kStages) ok = wait_or_stop(&s.k_empty[st], ((g / kStages) & 1) ^ 1, &s.stop, a.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) continue;
            const uint32_t there = __ballot_sync(0xFFFFFFFFu, my_k == i && page >= 0);
            const int64_t row0 = page >= 0 ? (static_cast<int64_t>(page) * a.c.Hkv + h) * a.c.block : -1;
            // The rows go ahead of the elected lane's arrival, which publishes them: the
            // asynchronous arrivals below only stand for the copies ahead of them.
            if (my_k == i) s.row0[st][my_slot] = row0;
            __syncwarp();
            // Codes count as they are packed, half of a slab's bytes.
            if (elect_one()) mbar_arrive_expect_tx(&s.k_full[st], __popc(there) * (slab / 2));
            __syncwarp();
            // Each lane of the tile brings its own block's keys.
            if (my_k == i && page >= 0) tma_load_3d(ring + st * kTile + my_slot * slab, &tm_k, 0, y, page, &s.k_full[st]);
            // Scales and weights by 16-byte copies of all lanes: bulk copies of a
            // block's few bytes took 700 cycles a tile to issue.
            {
              const int t = lane * 8;
              const int64_t from = __shfl_sync(0xFFFFFFFFu, row0, (i * spt + t / a.c.block) & 31);
              if (from >= 0 && t < C::kTokens) copy16(&s.ks[st][t], a.c.k_scale4 + from + (t & (a.c.block - 1)));
            }
            if (pass == 0 && w.decay != 0.0f) {
#pragma unroll
              for (int x = 0; x < PAR; ++x) {
                const int t = x * 128 + lane * 4;
                const int64_t from = __shfl_sync(0xFFFFFFFFu, row0, (i * spt + t / a.c.block) & 31);
                if (from >= 0) copy16(&s.old[st][t], w.weights + from + (t & (a.c.block - 1)));
              }
            }
            copies_arrive(&s.k_full[st]);
          }
        }
      }
    });
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(a.status, kErrCacheIndex);
    if (!ok)  // let the copies in flight land before the CTA gives its memory back
      for (int i = p; i < kStages; i += kProducers)
        for (uint32_t parity = 0; parity < 2; ++parity) mbar_wait_bounded(&s.k_full[i], parity, 10000000ull);
  } else if (warp < kFirstProducer) {
    // ----------------------------------------------------------- products
    const int wg = warp - 8;
    const uint32_t tm = uniform(s.tmem) + wg * 2 * kPlace, ring_addr = smem_u32(ring), q_addr = smem_u32(q_smem);
    const bool leader = elect_one();
    uint32_t g0 = 0, pc = 0, unit = 0;
    each_item<C>(a, s, [&](int b, const Sequence& q, int h, int t0, int part) {
      for (int pass = 0; pass < passes; ++pass, ++pc) {
        const uint32_t buf = pc & 1;
        const int groups = min(per_pass, n_groups - pass * kGroups);
        wait_or_stop(&s.q_full[buf], (pc >> 1) & 1, &s.stop, a.status);
        for (uint32_t g = g0 + ((g0 ^ wg) & 1); g < g0 + part; g += 2) {
          const uint32_t st = g % kStages;
          wait_or_stop(&s.k_full[st], (g / kStages) & 1, &s.stop, a.status);
          for (int gr = 0; gr < groups; ++gr, ++unit) {
            const uint32_t place = unit & 1;
            if (unit >= 2) wait_or_stop(&s.s_empty[wg][place], ((unit >> 1) & 1) ^ 1, &s.stop, a.status);
            __syncwarp();
            tc_fence_after_sync();
            if (leader) {
              const uint64_t ka = smem_desc_rows<128>(ring_addr + st * kTile);
              const uint64_t qa = smem_desc_rows<C::HD>(q_addr + (buf * kGroups + gr) * C::kQBytes);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int ks = i % (C::HD / 32), half = i / (C::HD / 32);
                mma_f8_ss(tm + place * kPlace + half * C::NQ, ka + i * 2, qa + ks * 2, idesc_f8(C::NQ, false, true), ks > 0);
              }
              mma_commit(&s.s_full[wg][place]);
              if (gr == groups - 1) mma_commit(&s.k_empty[st]);
            }
            __syncwarp();
          }
        }
        if (leader) mma_commit(&s.q_empty[buf]);
        __syncwarp();
        g0 += part;
      }
    });
  } else {
    // ------------------------------------------------------------ queries
    uint32_t pc = 0;
    each_item<C>(a, s, [&](int b, const Sequence& q, int h, int t0, int part) {
      for (int pass = 0; pass < passes; ++pass, ++pc) {
        const uint32_t buf = pc & 1;
        if (pc >= 2) wait_or_stop(&s.q_empty[buf], ((pc >> 1) & 1) ^ 1, &s.stop, a.status);
        const int groups = min(per_pass, n_groups - pass * kGroups);
        // A warp's rows are of one group, and loaded together.
        constexpr int kRows = (kGroups * C::RR + kQueryWarps - 1) / kQueryWarps, kWarps = C::RR / kRows;
        static_assert(kWarps <= 8, "warps of a group");
        const int gr = (warp - C::kFirstQuery) / kWarps, r0 = (warp - C::kFirstQuery) % kWarps * kRows, r = r0 + lane;
        if (gr < groups) {
          GroupRows<C>& rows = s.rows[buf][gr];
          Entry en{};
          en.b = b;
          const int group = pass * kGroups + gr;
          const int item = h * a.split + group % a.split;  // its heads are item * a.R ..
          en.j0 = group / a.split * a.qt;
          en.nq = min(en.j0 + a.qt, q.n_new) - en.j0;
          en.first_pos = q.first + en.j0;
          // (A lane's row as query_rows has it.)
          const int row = r, j = row / a.R;
          const bool there = lane < kRows && row < a.qt * a.R && j < en.nq && en.first_pos + j >= 0;
          float lse = -INFINITY;
          if (there)
            lse = load_global(w.lse + (static_cast<int64_t>(b) * a.n + en.j0 + j) * a.Hq + item * a.R + (row - j * a.R));
          query_rows<C, kRows>(a, rows.info, q_smem + (buf * kGroups + gr) * C::kQBytes, en, item, r0, 1);
          __syncwarp();
          if (lane < kRows) {
            const bool gives = there && lse != -INFINITY;
            const float t = rows.info.row_mul[r];
            rows.c[r] = gives ? t * w.c : 0.0f;
            rows.nl[r] = gives ? lse * -1.4426950408889634f : -INFINITY;
            if (!gives) rows.info.row_pos[r] = -1;
          }
          // (Rows that are not there too: a group of them alone is masked as a silent one is.)
          const bool silent = __any_sync(0xFFFFFFFFu, lane < kRows && row < a.qt * a.R && en.j0 + j < a.n && lse == -INFINITY);
          if (lane == 0) rows.silent[(warp - C::kFirstQuery) % kWarps] = silent;
          __syncwarp();
        }
        // The first position that not all of the pass's rows see.
        if (warp == C::kFirstQuery && lane == 0) s.rows[buf][0].info.lo_pos = q.n_new > 0 ? max(q.first + pass * kGroups / a.split * a.qt, 0) : -1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.q_full[buf]);
      }
    });
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 8) tmem_dealloc(s.tmem, 512);
}

template <int D, int RT, int T>
cudaError_t weights_form(const CUtensorMap& tk, const WeightsArgs& w, int grid, int device, cudaStream_t stream) {
  using C = WeightsCfg<D, RT, T>;
  constexpr int smem = 1024 + C::kStages * kKvTile * 128 + 2 * C::kGroups * C::kQBytes + static_cast<int>(sizeof(WeightsShared<C>));
  static_assert(smem <= 227 * 1024, "shared memory");
  static_assert(C::NS <= kPlace, "tensor memory");
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << device;
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kv4_weights_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  const cudaError_t e = launch_pdl(kv4_weights_kernel<C>, dim3(grid), dim3(C::kThreads), smem, stream, tk, w);
  if (e == cudaSuccess) plan_add("kv4_weights_kernel");
  return e;
}

template <int D, int T>
cudaError_t weights_rows(int rt, const CUtensorMap& tk, const WeightsArgs& w, int grid, int device, cudaStream_t stream) {
  if (rt <= 8) return weights_form<D, 8, T>(tk, w, grid, device, stream);
  if (rt <= 16) return weights_form<D, 16, T>(tk, w, grid, device, stream);
  return weights_form<D, 32, T>(tk, w, grid, device, stream);
}

}  // namespace

cudaError_t launch_kv4_weights(const Kv4WeightsProblem& p, const DeviceInfo& dev, cudaStream_t stream) {
  WeightsArgs w{};
  AttendArgs& a = w.a;
  a.c = p.cache;
  a.q = p.q;
  a.status = dev.status_word;
  a.scale_log2 = 1.0f;
  a.n = p.n;
  a.Hq = p.Hq;
  a.R = p.Hq / p.cache.Hkv;
  a.bf16 = p.bf16;
  const int columns = 128 / p.cache.D;  // of a row: one for each token of an operand row
  a.tile_log2 = columns == 2 ? 8 : 7;
  a.spt = (1 << a.tile_log2) / p.cache.block;
  a.split = head_split(a.R, columns, 32);
  a.R /= a.split;
  a.qt = std::min(p.n, 32 / (a.R * columns));
  w.lse = p.lse;
  w.weights = p.weights;
  w.decay = p.decay;
  w.c = static_cast<float>(static_cast<double>(p.scale) * 1.4426950408889634);
  const int64_t most = static_cast<int64_t>(p.cache.B) * p.cache.Hkv * ((p.cache.max_blocks - 1) / a.spt + 1);
  const int grid = static_cast<int>(std::min<int64_t>(dev.sm_count, most));
  CUtensorMap tk;
  if (!encode_cache_map4(&tk, p.cache.k, p.cache)) return cudaErrorInvalidValue;
  const int rt = a.split > 1 ? 32 : a.qt * a.R * columns;
  if (p.cache.D == 64)
    return p.bf16 ? weights_rows<64, 2>(rt, tk, w, grid, dev.id, stream)
                  : weights_rows<64, 3>(rt, tk, w, grid, dev.id, stream);
  return p.bf16 ? weights_rows<128, 2>(rt, tk, w, grid, dev.id, stream)
                : weights_rows<128, 3>(rt, tk, w, grid, dev.id, stream);
}

}  // namespace qsa
