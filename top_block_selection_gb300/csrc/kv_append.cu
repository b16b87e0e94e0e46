// kv_append.cu - appending keys and values to the paged 8-bit cache.
//
// For each new token (position p) the key's rotated pairs are
//     x' = x cos[p] - y sin[p],  y' = y cos[p] + x sin[p]
// in fp32, each product and each sum rounded (no fused multiply-add), so the
// stored codes are a fixed function of the inputs. The new tokens of one
// (block, head) share one scale: the smallest power of two s with
// max|x| <= 448 s, and at least the block's scale so far when older tokens
// stand in the block; code = e4m3(x / s), round to nearest even. A power of
// two makes x / s exact and costs e4m3 no precision (its relative step does
// not depend on the scale), and when a block's scale grows the older codes
// are multiplied by a power of two: exact unless they fall below 2^-6, where
// they are rounded again.
// The block key is the mean of the block's stored keys, s * sum(codes) / n. A
// sum of up to 73 codes is a multiple of 2^-9 below 2^15, exact in fp32 in any
// order; a warp adds at most 40. The warps' sums are added as integers, in
// units of 2^-9, so that the sum of 128 codes is rounded once: it depends on
// the codes alone.
//
// What bounds it: bytes. One CTA owns one (block, head, K or V): it holds the
// block's new values in registers between the maximum and the rounding, so
// each input byte is read once and each code written once, and nobody else
// writes the block's scale. 4,096 tokens, 8 KV heads, 32 query heads, D = 128
// take 20.8 us (4.5 TB/s, 68% of a plain copy's rate), one token of each of 64
// requests 5.0 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_internal.h"
#include "qsa_device.cuh"

namespace qsa {
namespace {

constexpr int kHeadsPerThread = 2;  // query heads of a thread (4: 3% to 18% slower, 8: 30%)

struct AppendArgs {
  KvCacheArgs c;
  KvRows k, v, q;
  const float* cos;
  const float* sin;
  void* q_out;
  uint16_t* kb;
  uint32_t* status;
  int64_t units;
  int32_t n, Hq, rot, max_pos, blocks_per_seq;
};

__device__ __forceinline__ uint4 load8(const void* base, int64_t off) {
  return load_global(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off));
}

template <bool BF16>
__device__ __forceinline__ void unpack8(uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* base, int64_t off, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + off) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread holds two runs of 8 elements of one row. In the rotated part they
// are the two members of 8 half-split pairs, or 4 + 4 interleaved pairs.
struct Lane {
  int off0, off1;  // element offsets of the two runs
  int ang0, ang1;  // offsets of the angles (half-split: 8 at ang0; interleaved: 4 at each)
  bool turns;
};

template <int TPT>
__device__ __forceinline__ Lane lane_of(int sub, int rot, bool interleaved) {
  Lane l;
  l.turns = sub < rot / 16;
  if (l.turns) {
    l.off0 = 8 * sub;
    l.off1 = rot / 2 + 8 * sub;
    l.ang0 = interleaved ? 4 * sub : 8 * sub;
    l.ang1 = rot / 4 + 4 * sub;
  } else {
    l.off0 = rot + 16 * (sub - rot / 16);
    l.off1 = l.off0 + 8;
    l.ang0 = l.ang1 = 0;
  }
  return l;
}

__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float u = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = u;
}

// Rotates a thread's two runs by the angles of row `row` of the tables, four
// pairs at a time.
template <bool PAIRS>
__device__ __forceinline__ void rotate(const float* cos, const float* sin, int64_t row, const Lane& l, float (&x)[8],
                                       float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t at = row + (i == 0 ? l.ang0 : (PAIRS ? l.ang1 : l.ang0 + 4));
    const float4 c = load_global(reinterpret_cast<const float4*>(cos + at));
    const float4 s = load_global(reinterpret_cast<const float4*>(sin + at));
    if (PAIRS) {
      float(&z)[8] = i == 0 ? x : y;
      turn(z[0], z[1], c.x, s.x);
      turn(z[2], z[3], c.y, s.y);
      turn(z[4], z[5], c.z, s.z);
      turn(z[6], z[7], c.w, s.w);
    } else {
      turn(x[4 * i], y[4 * i], c.x, s.x);
      turn(x[4 * i + 1], y[4 * i + 1], c.y, s.y);
      turn(x[4 * i + 2], y[4 * i + 2], c.z, s.z);
      turn(x[4 * i + 3], y[4 * i + 3], c.w, s.w);
    }
  }
}

__device__ __forceinline__ uint2 encode8(const float (&x)[8], float s, float inv, bool pow2) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = pow2 ? x[i] * inv : __fdiv_rn(x[i], s);
  uint2 r;
  r.x = e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16);
  r.y = e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16);
  return r;
}

__device__ __forceinline__ void decode8(uint2 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x & 0xFFFFu, u.x >> 16, u.y & 0xFFFFu, u.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = e4m3x2_to_float2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// Rotates the queries: TPT threads a row, each for kHeadsPerThread heads.
template <int TPT, int THREADS, bool BF16, bool PAIRS>
__device__ __forceinline__ void rotate_queries(const AppendArgs& a) {
  const int sub = threadIdx.x % TPT;
  const int chunks = (a.Hq + kHeadsPerThread - 1) / kHeadsPerThread;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) - a.units) * (THREADS / TPT) + threadIdx.x / TPT;
  if (row >= static_cast<int64_t>(a.c.B) * a.n * chunks) return;
  const int64_t token = row / chunks;
  const int h0 = static_cast<int>(row - token * chunks) * kHeadsPerThread;
  const int b = static_cast<int>(token / a.n), j = static_cast<int>(token - static_cast<int64_t>(b) * a.n);
  const Lane l = lane_of<TPT>(sub, a.rot, PAIRS);
  const int64_t in = b * a.q.sb + j * a.q.sn;
  const Span sp = span_of(a.c, b, a.n);
  uint4 u[kHeadsPerThread][2];
#pragma unroll
  for (int i = 0; i < kHeadsPerThread; ++i)
    if (h0 + i < a.Hq) {
      u[i][0] = load8(a.q.data, in + (h0 + i) * a.q.sh + l.off0);
      u[i][1] = load8(a.q.data, in + (h0 + i) * a.q.sh + l.off1);
    }
  const int64_t pos = static_cast<int64_t>(sp.first) + j;
  bool there = j < sp.n_new && pos >= 0;
  if (there && a.rot > 0 && pos >= a.max_pos) {
    if (sub == 0) atomicOr(a.status, kErrCacheIndex);
    there = false;
  }
#pragma unroll
  for (int i = 0; i < kHeadsPerThread; ++i) {
    if (h0 + i >= a.Hq) break;
    const int64_t to = (token * a.Hq + h0 + i) * (TPT * 16);
    float x[8], y[8];
    unpack8<BF16>(there ? u[i][0] : make_uint4(0, 0, 0, 0), x);
    unpack8<BF16>(there ? u[i][1] : make_uint4(0, 0, 0, 0), y);
    if (there && l.turns) rotate<PAIRS>(a.cos, a.sin, pos * (a.rot / 2), l, x, y);
    store8<BF16>(a.q_out, to + l.off0, x);
    store8<BF16>(a.q_out, to + l.off1, y);
  }
}

// TPT threads a token (D = 16 TPT), THREADS / TPT tokens a pass, the new tokens
// of a block in at most PASSES passes, held in registers.
// (1,024 threads an SM: 64 registers and a spill of a few words, against 80 and
// none at 768, take 22.2 us instead of 23.3 for 4,096 tokens, 32 + 16 heads; a
// form of four passes would spill its values.)
template <int TPT, int PASSES, int THREADS, bool BF16, bool PAIRS>
__global__ void __launch_bounds__(THREADS, (PASSES < 4 ? 1024 : 768) / THREADS) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  pdl_wait();
  pdl_launch_dependents();  // after the wait: at most one kernel ahead of the one that runs
  if (static_cast<int64_t>(blockIdx.x) >= a.units) {
    rotate_queries<TPT, THREADS, BF16, PAIRS>(a);
    return;
  }
  constexpr int D = 16 * TPT;
  constexpr int kTokens = THREADS / TPT;  // tokens of one pass
  __shared__ uint32_t s_max[THREADS / 32];
  __shared__ float s_sum[THREADS / 32][D];

  uint32_t u = blockIdx.x;
  const bool is_v = u & 1;
  u >>= 1;
  const uint32_t bi = u / a.c.Hkv;
  const int h = static_cast<int>(u - bi * a.c.Hkv);
  const int b = static_cast<int>(bi / a.blocks_per_seq), i = static_cast<int>(bi - b * a.blocks_per_seq);

  const Span sp = span_of(a.c, b, a.n);
  const int p0 = max(sp.first, 0);
  if (sp.len <= p0) return;  // no new token
  const int64_t blk64 = static_cast<int64_t>(p0 / a.c.block) + i;
  const int64_t start64 = blk64 * a.c.block;
  if (start64 >= sp.len) return;
  int64_t end64 = min(start64 + a.c.block, static_cast<int64_t>(sp.len));
  if (a.rot > 0 && end64 > a.max_pos) {  // positions past the angles are left out
    if (threadIdx.x == 0) atomicOr(a.status, kErrCacheIndex);
    end64 = a.max_pos;
    if (end64 <= max(static_cast<int64_t>(p0), start64)) return;
  }
  int page = -1;
  if (blk64 < a.c.max_blocks) page = load_global(a.c.page_table + static_cast<int64_t>(b) * a.c.max_blocks + blk64);

  // The new tokens: from `from` on, one to a group of TPT threads.
  const int start = static_cast<int>(start64), end = static_cast<int>(end64);
  const int from = max(p0, start), n_old = from - start, held = end - start, fresh = end - from;
  const KvRows& src = is_v ? a.v : a.k;
  const int64_t in = b * src.sb + h * src.sh;
  const int sub = threadIdx.x % TPT, tok = threadIdx.x / TPT;
  const Lane l = lane_of<TPT>(sub, is_v ? 0 : a.rot, PAIRS);
  uint4 raw[PASSES][2];
#pragma unroll
  for (int t = 0; t < PASSES; ++t)
    if (t * kTokens + tok < fresh) {
      const int64_t row = in + (static_cast<int64_t>(from) + t * kTokens + tok - sp.first) * src.sn;
      raw[t][0] = load8(src.data, row + l.off0);
      raw[t][1] = load8(src.data, row + l.off1);
    }
  if (page < 0 || page >= a.c.n_pages) {
    if (threadIdx.x == 0) atomicOr(a.status, kErrCacheIndex);
    return;
  }
  float* const scale_at = (is_v ? a.c.v_scale : a.c.k_scale) + static_cast<int64_t>(page) * a.c.Hkv + h;
  const float s_old = n_old > 0 ? load_global(scale_at) : 0.0f;
  uint8_t* const codes = (is_v ? a.c.v : a.c.k) + page * a.c.page_stride + static_cast<int64_t>(h) * a.c.block * D;

  float x[PASSES][8], y[PASSES][8], m = 0.0f;
#pragma unroll
  for (int t = 0; t < PASSES; ++t)
    if (t * kTokens + tok < fresh) {
      unpack8<BF16>(raw[t][0], x[t]);
      unpack8<BF16>(raw[t][1], y[t]);
      if (l.turns)
        rotate<PAIRS>(a.cos, a.sin, (static_cast<int64_t>(from) + t * kTokens + tok) * (a.rot / 2), l, x[t], y[t]);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(fabsf(x[t][e]), fabsf(y[t][e])));
    }
  // Non-negative floats order as their bits.
  const uint32_t wm = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
  if (threadIdx.x % 32 == 0) s_max[threadIdx.x / 32] = wm;
  __syncthreads();
  uint32_t bm = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) bm = max(bm, s_max[w]);
  const float s_new = pow2_scale(__uint_as_float(bm));
  const float s = n_old > 0 ? fmaxf(s_old, s_new) : s_new;
  const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0;
  const float inv = pow2 ? __uint_as_float((254u << 23) - __float_as_uint(s)) : 0.0f;
  const float ratio = n_old > 0 ? __fdiv_rn(s_old, s) : 1.0f;
  const bool want_kb = a.kb != nullptr && !is_v;
  if (threadIdx.x == 0) *scale_at = s;

  float acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
  auto add = [&](uint2 c0, uint2 c1) {
    float f[8];
    decode8(c0, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += f[e];
    decode8(c1, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[8 + e] += f[e];
  };
#pragma unroll
  for (int t = 0; t < PASSES; ++t) {
    const int slot = n_old + t * kTokens + tok;
    if (slot >= held) continue;
    const uint2 c0 = encode8(x[t], s, inv, pow2), c1 = encode8(y[t], s, inv, pow2);
    *reinterpret_cast<uint2*>(codes + slot * D + l.off0) = c0;
    *reinterpret_cast<uint2*>(codes + slot * D + l.off1) = c1;
    if (want_kb) add(c0, c1);
  }
  // The older tokens: rounded again where the scale grew, added to the mean.
  if (n_old > 0 && (want_kb || ratio != 1.0f)) {
#pragma unroll 4
    for (int slot = tok; slot < n_old; slot += kTokens) {
      uint2* const at0 = reinterpret_cast<uint2*>(codes + slot * D + l.off0);
      uint2* const at1 = reinterpret_cast<uint2*>(codes + slot * D + l.off1);
      uint2 c0 = *at0, c1 = *at1;
      if (ratio != 1.0f) {
        float f[8];
        decode8(c0, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= ratio;
        c0 = encode8(f, 1.0f, 1.0f, true);
        decode8(c1, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= ratio;
        c1 = encode8(f, 1.0f, 1.0f, true);
        *at0 = c0;
        *at1 = c1;
      }
      if (want_kb) add(c0, c1);
    }
  }
  if (!want_kb) return;
#pragma unroll
  for (int d = TPT; d < 32; d *= 2)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] += __shfl_xor_sync(0xFFFFFFFFu, acc[e], d);
  if (threadIdx.x % 32 < TPT) {
    float* const row = s_sum[threadIdx.x / 32];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      row[l.off0 + e] = acc[e];
      row[l.off1 + e] = acc[8 + e];
    }
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float total = 0.0f;
    int units = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      const float part = s_sum[w][threadIdx.x];
      total += part;
      units += __float2int_rn(part * 512.0f);
    }
    if (!isnan(total)) total = __int2float_rn(units) * 0.001953125f;
    const float mean = __fdiv_rn(__fmul_rn(total, s), static_cast<float>(held));
    const int64_t at = ((static_cast<int64_t>(b) * a.c.Hkv + h) * a.c.max_blocks + blk64) * D + threadIdx.x;
    a.kb[at] = __half_as_ushort(__float2half_rn(mean));
    // A scorer next on the stream may start early and reads block keys by bulk
    // copies, without a fence between these plain stores and its copies.
    fence_proxy_async_global();
  }
}

template <int TPT, int PASSES, int THREADS>
cudaError_t launch_form(const AppendArgs& a, bool bf16, bool pairs, unsigned grid, cudaStream_t stream) {
  // Programmatic dependent launch: the CTAs are there when the work before them
  // on the stream ends (pdl_wait), which saves about 2 us of a step's calls.
  cudaError_t e;
  if (bf16) {
    e = pairs ? launch_pdl(kv_append_kernel<TPT, PASSES, THREADS, true, true>, dim3(grid), dim3(THREADS), 0, stream, a)
              : launch_pdl(kv_append_kernel<TPT, PASSES, THREADS, true, false>, dim3(grid), dim3(THREADS), 0, stream, a);
  } else {
    e = pairs ? launch_pdl(kv_append_kernel<TPT, PASSES, THREADS, false, true>, dim3(grid), dim3(THREADS), 0, stream, a)
              : launch_pdl(kv_append_kernel<TPT, PASSES, THREADS, false, false>, dim3(grid), dim3(THREADS), 0, stream, a);
  }
  if (e != cudaSuccess) return e;
  plan_add("kv_append_kernel");
  return cudaSuccess;
}

// With few new tokens a sequence (a decode step) a CTA's work is a chain of
// loads, and what counts is that all CTAs run at once: 128 threads. Otherwise
// 256, for the bytes in flight.
int append_threads(const KvAppendProblem& p) { return p.n * (p.cache.D / 16) <= 128 ? 128 : 256; }

}  // namespace

int64_t kv_append_grid(const KvAppendProblem& p, int64_t* units, int32_t* blocks_per_seq) {
  // n tokens that begin anywhere in a block reach at most this many blocks.
  const int64_t per_seq = (static_cast<int64_t>(p.n) + p.cache.block - 2) / p.cache.block + 1;
  *blocks_per_seq = static_cast<int32_t>(per_seq);
  *units = per_seq * p.cache.B * p.cache.Hkv * 2;
  if (!p.q.data) return *units;
  const int64_t rows =
      static_cast<int64_t>(p.cache.B) * p.n * ((p.Hq + kHeadsPerThread - 1) / kHeadsPerThread);
  const int per_cta = append_threads(p) / (p.cache.D / 16);
  return *units + (rows + per_cta - 1) / per_cta;
}

cudaError_t launch_kv_append(const KvAppendProblem& p, const DeviceInfo& dev, cudaStream_t stream) {
  AppendArgs a{};
  a.c = p.cache;
  a.k = p.k;
  a.v = p.v;
  a.q = p.q;
  a.cos = p.cos;
  a.sin = p.sin;
  a.q_out = p.q_out;
  a.kb = p.kb;
  a.status = dev.status_word;
  a.n = p.n;
  a.Hq = p.Hq;
  a.rot = p.rot;
  a.max_pos = p.max_pos;
  const unsigned grid = static_cast<unsigned>(kv_append_grid(p, &a.units, &a.blocks_per_seq));
  const bool few = append_threads(p) == 128;
  if (p.cache.D == 128) {
    if (few) return launch_form<8, 1, 128>(a, p.bf16, p.interleaved, grid, stream);
    if (p.cache.block <= 32) return launch_form<8, 1, 256>(a, p.bf16, p.interleaved, grid, stream);
    if (p.cache.block <= 64) return launch_form<8, 2, 256>(a, p.bf16, p.interleaved, grid, stream);
    return launch_form<8, 4, 256>(a, p.bf16, p.interleaved, grid, stream);
  }
  if (few) return launch_form<4, 1, 128>(a, p.bf16, p.interleaved, grid, stream);
  if (p.cache.block <= 64) return launch_form<4, 1, 256>(a, p.bf16, p.interleaved, grid, stream);
  return launch_form<4, 2, 256>(a, p.bf16, p.interleaved, grid, stream);
}

}  // namespace qsa
