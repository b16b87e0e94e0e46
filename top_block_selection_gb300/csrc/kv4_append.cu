// kv4_append.cu - writing the paged 4-bit cache and reading it back.
//
// Each new token's key (rotated as in kv_append.cu) and value have, for each KV
// head, a scale of their own, the smallest bf16 s with max|x| <= 6 s, and the
// codes e2m1(x / s), the quotient rounded to fp32 first. That changes no code:
// a border T between two codes is a number of at most three bits, and s T is an
// fp32 number, so that x / s is T itself, exactly, or off by more than half an
// fp32 step: x differs from s T by a step of its own, and the 8 bits of s keep its
// mantissa below 2 - 2^-7. The quotient is x times the reciprocal of s, corrected
// by its remainder (Markstein): within 2^-47 before its one rounding, at two
// operations more than the product (a division each took 2 us more for 4,096
// tokens). A token's codes depend on that token
// alone: nothing that is in the cache is touched again.
//
// The block key is the mean of the block's stored keys. Products of a code and
// its scale are exact in fp32 (10 bits); they are added slot by slot in an
// order that depends on the slots alone (slot i in the sum i % kTokens, these
// in a tree), so that appending together or one by one gives the same bits.
//
// One CTA owns one (block, head, K or V): scales and codes of a block are contiguous
// there. What bounds it: for chunks, instructions beside bytes (4,096 tokens, 8 heads
// of 128 dimensions and 32 of queries, 19.6 us, 4.4 TB/s of what has to be moved, issue
// slots 67% busy: rotation, maximum, quotients, conversions); for few tokens a chain of
// dependent loads (lengths, page, codes of the begun block), 5.8 us for a token of
// each of 64 requests. Reading the 4,096 tokens back takes 6.7 us.
#include "kv4_codes.cuh"
#include "kv_rows.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 128;
// One token of a thread at a time and 8 CTAs an SM: 4,096 tokens 19.6 us, a token of
// each of 64 requests 5.8 (two tokens in flight, which spills, 19.6 and 6.4, at 6
// CTAs an SM 21.2 and 5.5; four and 6, with divisions, 23.8 and 7.9).
constexpr int kCtasPerSm = 8;

// inv is 1 / s, rounded.
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], float s, float inv) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = x[i] * inv;
    y[i] = copysignf(fmaf(fmaf(-q, s, x[i]), inv, q), x[i]);  // (the sign of a zero)
  }
  return e2m1x8(y);
}

template <int TPT, bool BF16, bool PAIRS>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv4_append_kernel(const __grid_constant__ AppendArgs a) {
  pdl_wait();
  pdl_launch_dependents();  // after the wait: at most one kernel ahead of the one that runs
  if (static_cast<int64_t>(blockIdx.x) >= a.units) {
    rotate_queries<TPT, kThreads, BF16, PAIRS>(a);
    return;
  }
  constexpr int D = 16 * TPT;
  constexpr int kTokens = kThreads / TPT;  // tokens of one pass
  __shared__ float s_sum[kThreads / 32][D];

  uint32_t u = blockIdx.x;
  const bool is_v = u & 1;
  u >>= 1;
  const uint32_t bi = u / a.c.Hkv;
  const int h = static_cast<int>(u - bi * a.c.Hkv);
  const int b = static_cast<int>(bi / a.blocks_per_seq), i = static_cast<int>(bi - b * a.blocks_per_seq);

  const Span sp = span_of(a.c, b, a.n);
  const int64_t ahead = a.offset ? load_global(a.offset + b) : 0;
  const int p0 = max(sp.first, 0);
  if (sp.len <= p0) return;  // no new token
  const int64_t blk64 = static_cast<int64_t>(p0 / a.c.block) + i;
  const int64_t start64 = blk64 * a.c.block;
  if (start64 >= sp.len) return;
  int64_t end64 = min(start64 + a.c.block, static_cast<int64_t>(sp.len));
  // Tokens whose positions are not in the angle tables are left out.
  if (a.rot > 0 && (ahead < 0 || end64 + ahead > a.max_pos)) {
    if (threadIdx.x == 0) atomicOr(a.status, kErrCacheIndex);
    end64 = ahead < 0 ? 0 : a.max_pos - ahead;
    if (end64 <= max(static_cast<int64_t>(p0), start64)) return;
  }
  int page = -1;
  if (blk64 < a.c.max_blocks) page = load_global(a.c.page_table + static_cast<int64_t>(b) * a.c.max_blocks + blk64);

  const int start = static_cast<int>(start64), held = static_cast<int>(end64) - start;
  const int n_old = max(p0 - start, 0);
  const KvRows& src = is_v ? a.v : a.k;
  const int64_t in = b * src.sb + h * src.sh + (static_cast<int64_t>(start) - sp.first) * src.sn;
  const int sub = threadIdx.x % TPT, tok = threadIdx.x / TPT;
  const Lane l = lane_of<TPT>(sub, is_v ? 0 : a.rot, PAIRS);
  const bool want_kb = a.kb != nullptr && !is_v;

  float acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
  auto add = [&](uint32_t c0, uint32_t c1, float s) {
    float x[8], y[8];
    e2m1x8_to_float(c0, x);
    e2m1x8_to_float(c1, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      acc[e] = fmaf(x[e], s, acc[e]);
      acc[8 + e] = fmaf(y[e], s, acc[8 + e]);
    }
  };
  uint8_t* codes = nullptr;
  uint16_t* scales = nullptr;
  auto found = [&]() {
    const bool there = page >= 0 && page < a.c.n_pages;
    if (!there && threadIdx.x == 0) atomicOr(a.status, kErrCacheIndex);
    codes = (is_v ? a.c.v : a.c.k) + page * a.c.page_stride + static_cast<int64_t>(h) * a.c.block * (D / 2);
    scales = (is_v ? a.c.v_scale4 : a.c.k_scale4) + (static_cast<int64_t>(page) * a.c.Hkv + h) * a.c.block;
    return there;
  };
  // The older tokens, for the block key: the loads of four go out together.
  if (want_kb && n_old > 0) {
    if (!found()) return;
#pragma unroll 1
    for (int s0 = tok; s0 < n_old; s0 += 4 * kTokens) {
      uint32_t c0[4], c1[4];
      float s[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int slot = min(s0 + t * kTokens, n_old - 1);
        c0[t] = load_global(reinterpret_cast<const uint32_t*>(codes + slot * (D / 2) + l.off0 / 2));
        c1[t] = load_global(reinterpret_cast<const uint32_t*>(codes + slot * (D / 2) + l.off1 / 2));
        s[t] = load_scale(scales + slot);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (s0 + t * kTokens < n_old) add(c0[t], c1[t], s[t]);
    }
  }
  for (int slot = n_old / kTokens * kTokens + tok; slot - tok < held; slot += kTokens) {
    const bool fresh = slot >= n_old && slot < held;
    uint4 raw0, raw1;
    if (fresh) {
      const int64_t row = in + static_cast<int64_t>(slot) * src.sn;
      raw0 = load8(src.data, row + l.off0);
      raw1 = load8(src.data, row + l.off1);
    }
    // The page is waited for only now, with the new tokens on their way.
    if (!codes && !found()) return;
    uint32_t c0 = 0, c1 = 0, top = 0;
    float s = 0.0f, x[8], y[8];
    if (fresh) {
      unpack8<BF16>(raw0, x);
      unpack8<BF16>(raw1, y);
      if (l.turns) rotate<PAIRS>(a.cos, a.sin, (ahead + start + slot) * (a.rot / 2), l, x, y);
      // Magnitudes order as their bits, NaN above all.
#pragma unroll
      for (int e = 0; e < 8; ++e)
        top = max(top, max(__float_as_uint(x[e]) & 0x7FFFFFFFu, __float_as_uint(y[e]) & 0x7FFFFFFFu));
    }
#pragma unroll
    for (int d = 1; d < TPT; d *= 2) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    if (fresh) {
      s = token_scale(top);
      if (top == 0x7F800000u) {  // infinities to the largest finite float: code 6
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = fminf(fmaxf(x[e], -3.402823466e38f), 3.402823466e38f);
          y[e] = fminf(fmaxf(y[e], -3.402823466e38f), 3.402823466e38f);
        }
      }
      const float inv = __frcp_rn(s);
      c0 = isnan(s) ? 0u : encode8(x, s, inv);
      c1 = isnan(s) ? 0u : encode8(y, s, inv);
      *reinterpret_cast<uint32_t*>(codes + slot * (D / 2) + l.off0 / 2) = c0;
      *reinterpret_cast<uint32_t*>(codes + slot * (D / 2) + l.off1 / 2) = c1;
      if (sub == 0) scales[slot] = static_cast<uint16_t>(__float_as_uint(s) >> 16);
      if (want_kb) add(c0, c1, s);
    }
  }
  // An attention next on the stream may start early and reads codes by bulk
  // copies, without a fence between these plain stores and its copies.
  fence_proxy_async_global();
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
    const float total = (s_sum[0][threadIdx.x] + s_sum[1][threadIdx.x]) + (s_sum[2][threadIdx.x] + s_sum[3][threadIdx.x]);
    const float mean = __fdiv_rn(total, static_cast<float>(held));
    const int64_t at = ((static_cast<int64_t>(b) * a.c.Hkv + h) * a.c.max_blocks + blk64) * D + threadIdx.x;
    a.kb[at] = __half_as_ushort(__float2half_rn(mean));
    // A scorer next on the stream reads block keys by bulk copies too.
    fence_proxy_async_global();
  }
}

struct ReadArgs {
  KvCacheArgs c;
  void* k;
  void* v;
  uint32_t* status;
  int64_t rows;
  int32_t n;
};

// TPT threads a row (token, head, K or V), of 16 elements each; a row's code
// times scale is exact in fp32 and rounded once. 4,096 tokens take twice the time of
// their bytes at a plain copy's rate (6.6 us, 3.1): each thread has one chain of loads
// (lengths, page, codes), and no unit is above 45% (issue slots 55%).
template <int TPT, bool BF16>
__global__ void __launch_bounds__(256) kv4_read_kernel(const __grid_constant__ ReadArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int D = 16 * TPT;
  const int sub = threadIdx.x % TPT;
  int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / TPT) + threadIdx.x / TPT;
  if (row >= 2 * a.rows) return;
  const bool is_v = row >= a.rows;
  if (is_v) row -= a.rows;
  const int64_t token = row / a.c.Hkv;
  const int h = static_cast<int>(row - token * a.c.Hkv);
  const int b = static_cast<int>(token / a.n), j = static_cast<int>(token - static_cast<int64_t>(b) * a.n);
  const Span sp = span_of(a.c, b, a.n);
  const int64_t slot = static_cast<int64_t>(sp.first) + j;
  uint2 codes = make_uint2(0, 0);
  float s = 0.0f;
  if (j < sp.n_new && slot >= 0) {
    const int blk = static_cast<int>(slot / a.c.block), off = static_cast<int>(slot - static_cast<int64_t>(blk) * a.c.block);
    int page = -1;
    if (blk < a.c.max_blocks) page = load_global(a.c.page_table + static_cast<int64_t>(b) * a.c.max_blocks + blk);
    if (page < 0 || page >= a.c.n_pages) {
      if (sub == 0) atomicOr(a.status, kErrCacheIndex);
    } else {
      codes = load_global(reinterpret_cast<const uint2*>((is_v ? a.c.v : a.c.k) + page * a.c.page_stride +
                                                         (static_cast<int64_t>(h) * a.c.block + off) * (D / 2) + sub * 8));
      s = load_scale((is_v ? a.c.v_scale4 : a.c.k_scale4) + (static_cast<int64_t>(page) * a.c.Hkv + h) * a.c.block + off);
    }
  }
  float x[8], y[8];
  e2m1x8_to_float(codes.x, x);
  e2m1x8_to_float(codes.y, y);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] *= s;
    y[e] *= s;
  }
  void* const out = is_v ? a.v : a.k;
  store8<BF16>(out, row * D + sub * 16, x);
  store8<BF16>(out, row * D + sub * 16 + 8, y);
}

template <int TPT>
cudaError_t launch_form(const AppendArgs& a, bool bf16, bool pairs, unsigned grid, cudaStream_t stream) {
  cudaError_t e;
  if (bf16) {
    e = pairs ? launch_pdl(kv4_append_kernel<TPT, true, true>, dim3(grid), dim3(kThreads), 0, stream, a)
              : launch_pdl(kv4_append_kernel<TPT, true, false>, dim3(grid), dim3(kThreads), 0, stream, a);
  } else {
    e = pairs ? launch_pdl(kv4_append_kernel<TPT, false, true>, dim3(grid), dim3(kThreads), 0, stream, a)
              : launch_pdl(kv4_append_kernel<TPT, false, false>, dim3(grid), dim3(kThreads), 0, stream, a);
  }
  if (e == cudaSuccess) plan_add("kv4_append_kernel");
  return e;
}

}  // namespace

int64_t kv4_append_grid(const KvAppendProblem& p, int64_t* units, int32_t* blocks_per_seq) {
  // n tokens that begin anywhere in a block reach at most this many blocks.
  const int64_t per_seq = (static_cast<int64_t>(p.n) + p.cache.block - 2) / p.cache.block + 1;
  *blocks_per_seq = static_cast<int32_t>(per_seq);
  *units = per_seq * p.cache.B * p.cache.Hkv * 2;
  if (!p.q.data) return *units;
  const int64_t rows =
      static_cast<int64_t>(p.cache.B) * p.n * ((p.Hq + kHeadsPerThread - 1) / kHeadsPerThread);
  const int per_cta = kThreads / (p.cache.D / 16);
  return *units + (rows + per_cta - 1) / per_cta;
}

cudaError_t launch_kv4_append(const KvAppendProblem& p, const DeviceInfo& dev, cudaStream_t stream) {
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
  a.offset = p.offset;
  const unsigned grid = static_cast<unsigned>(kv4_append_grid(p, &a.units, &a.blocks_per_seq));
  if (p.cache.D == 128) return launch_form<8>(a, p.bf16, p.interleaved, grid, stream);
  return launch_form<4>(a, p.bf16, p.interleaved, grid, stream);
}

int64_t kv4_read_grid(const KvCacheArgs& c, int32_t n) {
  const int per_cta = 256 / (c.D / 16);
  return (2 * static_cast<int64_t>(c.B) * n * c.Hkv + per_cta - 1) / per_cta;
}

cudaError_t launch_kv4_read(const KvCacheArgs& c, int32_t n, bool bf16, void* k, void* v, const DeviceInfo& dev,
                            cudaStream_t stream) {
  const ReadArgs a{c, k, v, dev.status_word, static_cast<int64_t>(c.B) * n * c.Hkv, n};
  const dim3 grid(static_cast<unsigned>(kv4_read_grid(c, n)));
  cudaError_t e;
  if (c.D == 128)
    e = bf16 ? launch_pdl(kv4_read_kernel<8, true>, grid, dim3(256), 0, stream, a)
             : launch_pdl(kv4_read_kernel<8, false>, grid, dim3(256), 0, stream, a);
  else
    e = bf16 ? launch_pdl(kv4_read_kernel<4, true>, grid, dim3(256), 0, stream, a)
             : launch_pdl(kv4_read_kernel<4, false>, grid, dim3(256), 0, stream, a);
  if (e == cudaSuccess) plan_add("kv4_read_kernel");
  return e;
}

}  // namespace qsa
