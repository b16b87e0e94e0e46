// kv_rows.cuh - rows of 16-bit floats as the appends read them: eight elements
// at a time, rotated by position, and the rotation of the queries.
#pragma once

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
  const int32_t* offset;  // positions of a sequence's tokens beyond their slots, or null
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
  const int64_t slot = static_cast<int64_t>(sp.first) + j;
  const int64_t pos = slot + (a.offset ? load_global(a.offset + b) : 0);
  bool there = j < sp.n_new && slot >= 0;
  if (there && a.rot > 0 && (pos >= a.max_pos || pos < slot)) {
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

}  // namespace
}  // namespace qsa
