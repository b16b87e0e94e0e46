// qsa_api.cpp - the C ABI (include/qsa.h): host-side validation, block
// partition, and stream-ordered launches. Arguments are checked before any
// CUDA call, so a bad call returns a status without touching the device.
#include "qsa.h"

#include <cstdint>
#include <cstdio>
#include <cuda_runtime.h>

#include "kv_internal.h"
#include "qsa_internal.h"

namespace qsa {
void plan_begin();
void plan_add(const char* kernel);
}  // namespace qsa

namespace {

using qsa::DeviceInfo;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool supported_heads(int32_t H) {
  return H == 1 || H == 2 || H == 4 || H == 8 || H == 16 || H == 32;
}

cudaStream_t as_cuda(qsa_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

thread_local const char* t_last_cuda_error = "no error";

// The kernels the last call on this thread launched, in order (static names).
constexpr int kPlanMax = 8;
thread_local const char* t_plan[kPlanMax];
thread_local int t_plan_n = 0;
thread_local bool t_plan_any = false;

qsa_status cuda_fail(cudaError_t e) {
  t_last_cuda_error = cudaGetErrorString(e);
  return QSA_ERR_CUDA;
}

qsa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QSA_OK : cuda_fail(e); }

// Returns the current device's info, or an error status. Entry points that
// launch pass launching = true, which starts this thread's plan record.
qsa_status device_or_error(const DeviceInfo** out, bool launching = true) {
  cudaError_t e = cudaSuccess;
  const DeviceInfo* d = qsa::current_device(&e);
  if (!d) return cuda_fail(e);
  if (!d->supported) return QSA_ERR_UNSUPPORTED_ARCH;
  *out = d;
  if (launching) qsa::plan_begin();
  return QSA_OK;
}

struct Geometry {
  int64_t nb = 0, n_full = 0;
  bool has_tail = false;
};

// Checks shared by every scoring entry point; fills g on success.
qsa_status check_scores(const uint16_t* q, const uint16_t* kb, int32_t nq, int32_t H, int32_t D,
                        int64_t n_kv, int32_t block, const float* scores, Geometry* g) {
  if (nq < 0 || n_kv < 0 || block < 1 || H < 1 || D < 1) return QSA_ERR_INVALID_ARG;
  if (!supported_heads(H) || D % 16 != 0 || D < 16 || D > 256) return QSA_ERR_UNSUPPORTED_GEOMETRY;
  g->nb = n_kv / block + (n_kv % block != 0 ? 1 : 0);
  g->n_full = n_kv / block;
  g->has_tail = (n_kv % block) != 0;
  if (g->nb > 0x7FFFFFFFLL || static_cast<int64_t>(nq) * H > 0x7FFFFFFFLL)
    return QSA_ERR_UNSUPPORTED_GEOMETRY;
  if (nq == 0 || g->nb == 0) return QSA_OK;
  if (!q || !kb || !scores) return QSA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kb, 16) || !aligned(scores, 16)) return QSA_ERR_MISALIGNED;
  return QSA_OK;
}

qsa_status check_select(const float* scores, int32_t nq, int64_t nb, int32_t k,
                        const int32_t* ids) {
  if (nq < 0 || nb < 0 || k < 1) return QSA_ERR_INVALID_ARG;
  if (k > qsa::kMaxSelectK || nb > qsa::kMaxSelectNb) return QSA_ERR_UNSUPPORTED_GEOMETRY;
  if (nq == 0) return QSA_OK;
  if (!ids || (nb > 0 && !scores)) return QSA_ERR_INVALID_ARG;
  if (!aligned(ids, 4) || !aligned(scores, 4)) return QSA_ERR_MISALIGNED;
  return QSA_OK;
}

qsa_status run_scores(const uint16_t* q, const uint16_t* kb, int32_t nq, int32_t H, int32_t D,
                      const Geometry& g, float* scores, const DeviceInfo& dev,
                      cudaStream_t stream, bool skip_tail = false) {
  if (nq == 0 || g.nb == 0) return QSA_OK;
  qsa::ScoreProblem p{q, kb, scores, nq, H, D, g.nb, g.n_full, g.has_tail, skip_tail};
  return from_cuda(qsa::launch_scores(p, dev, stream));
}

// The single-batch steps run either the one fused cluster kernel or the
// separate stages (convert, score + tail, select) chained by programmatic
// dependent launch. Fused wins while its CTAs fit in a few waves (it saves the
// scores round trip and the launch gaps); past that the separate score kernel,
// which tiles 128 key blocks per MMA against many queries, does less work per
// score. Both write identical scores and ids.
bool use_separate(int32_t nq, int32_t H, const DeviceInfo& dev) {
  return qsa::fused_blocks(nq, H, dev) > 4LL * dev.sm_count;
}

// With many rows the select kernel scores the tail column itself (one launch
// fewer; the same pinned fp32 order, so the same bits).
qsa_status run_separate(const uint16_t* q, const uint16_t* kb, int32_t nq, int32_t H, int32_t D,
                        const Geometry& g, int32_t k, float* scores, int32_t* ids,
                        const DeviceInfo& dev, cudaStream_t stream) {
  const int32_t nb = static_cast<int32_t>(g.nb);
  const bool tail_in_select = g.has_tail && qsa::select_scores_tail(nq, nb, k);
  qsa_status st = run_scores(q, kb, nq, H, D, g, scores, dev, stream, tail_in_select);
  if (st != QSA_OK) return st;
  if (!tail_in_select) return from_cuda(qsa::launch_select(scores, nq, nb, k, ids, dev, stream));
  const qsa::TailInfo t{q, kb + (g.nb - 1) * D, H, D};
  return from_cuda(qsa::launch_select(scores, nq, nb, k, ids, dev, stream, &t));
}

// Batches with their own kb: past a few waves of the fused kernel the chain
// (persistent scores over every batch's tiles, then one select over every
// batch's rows, the tail block scored there) does the same work with less
// per score, when the persistent kernel and the row select can take it.
bool batched_chain_ok(int32_t n_batches, int32_t nq, int32_t H, int32_t D, const Geometry& g, int32_t k,
                      int64_t kb_batch_stride, const DeviceInfo& dev) {
  if (n_batches < 2 || g.nb == 0 || g.n_full == 0) return false;
  const int64_t rows = static_cast<int64_t>(n_batches) * nq;
  if (rows > 0x7FFFFFFFLL) return false;
  if (static_cast<int64_t>(n_batches) * qsa::fused_blocks(nq, H, dev) <= 4LL * dev.sm_count) return false;
  qsa::ScoreProblem sp{nullptr, nullptr, nullptr, nq, H, D, g.nb, g.n_full, g.has_tail, g.has_tail};
  sp.n_batches = n_batches;
  sp.kb_batch_stride = kb_batch_stride;
  if (!qsa::scores_persistent(sp, dev)) return false;
  return !g.has_tail || qsa::select_scores_tail(static_cast<int32_t>(rows), static_cast<int32_t>(g.nb), k);
}

qsa_status run_batched_chain(const uint16_t* q, const uint16_t* kb, int64_t kb_batch_stride,
                             int32_t n_batches, int32_t nq, int32_t H, int32_t D, const Geometry& g,
                             int32_t k, float* scores, int32_t* ids, const DeviceInfo& dev,
                             cudaStream_t stream) {
  qsa::ScoreProblem sp{q, kb, scores, nq, H, D, g.nb, g.n_full, g.has_tail, g.has_tail};
  sp.n_batches = n_batches;
  sp.kb_batch_stride = kb_batch_stride;
  qsa_status st = from_cuda(qsa::launch_scores(sp, dev, stream));
  if (st != QSA_OK) return st;
  const int32_t rows = n_batches * nq, nb = static_cast<int32_t>(g.nb);
  if (!g.has_tail) return from_cuda(qsa::launch_select(scores, rows, nb, k, ids, dev, stream));
  qsa::TailInfo t{q, kb + (g.nb - 1) * D, H, D};
  t.kb_batch_stride = kb_batch_stride;
  t.nq_per_batch = nq;
  return from_cuda(qsa::launch_select(scores, rows, nb, k, ids, dev, stream, &t));
}

}  // namespace

namespace qsa {
void plan_begin() {
  t_plan_n = 0;
  t_plan_any = true;
}
void plan_add(const char* kernel) {
  if (t_plan_n < kPlanMax) t_plan[t_plan_n++] = kernel;
}
}  // namespace qsa

// -------------------------------------------------------- the paged caches
// Sizes of a cache and the batch; nothing is dereferenced but *c. `bits` of an
// element, pages and their stride in units of `unit` bytes.
template <class Cache>
static qsa_status check_cache_sizes(const Cache* c, int32_t n, int bits, int unit) {
  if (!c) return QSA_ERR_INVALID_ARG;
  if (c->B < 0 || n < 0 || c->n_pages < 0 || c->max_blocks < 0 || c->Hkv < 1 || c->block < 1 || c->D < 1)
    return QSA_ERR_INVALID_ARG;
  if ((c->D != 64 && c->D != 128) ||
      (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) || c->Hkv > 65535)
    return QSA_ERR_UNSUPPORTED_GEOMETRY;
  if (static_cast<int64_t>(c->max_blocks) * c->block > (1 << 30) ||
      static_cast<int64_t>(c->B) * n > 0x7FFFFFFFLL)
    return QSA_ERR_UNSUPPORTED_GEOMETRY;
  if (c->page_stride < static_cast<int64_t>(c->Hkv) * c->block * c->D * bits / 8) return QSA_ERR_INVALID_ARG;
  if (c->page_stride >= (1LL << 40)) return QSA_ERR_UNSUPPORTED_GEOMETRY;
  if (c->page_stride % unit != 0) return QSA_ERR_MISALIGNED;
  return QSA_OK;
}
static qsa_status check_cache_sizes(const qsa_kv_cache* c, int32_t n) { return check_cache_sizes(c, n, 8, 16); }
static qsa_status check_cache_sizes(const qsa_kv4_cache* c, int32_t n) { return check_cache_sizes(c, n, 4, 32); }

// Codes on `unit` bytes, scales on `scale_unit`; values and their scales need
// not be there where `values` is false.
template <class Cache>
static qsa_status check_cache_pointers(const Cache* c, uintptr_t unit, uintptr_t scale_unit, bool values) {
  if (!c->lens || (c->max_blocks > 0 && !c->page_table)) return QSA_ERR_INVALID_ARG;
  if (c->n_pages > 0 && (!c->k || !c->k_scale || (values && (!c->v || !c->v_scale)))) return QSA_ERR_INVALID_ARG;
  if (!aligned(c->k, unit) || !aligned(c->v, unit) || !aligned(c->k_scale, scale_unit) ||
      !aligned(c->v_scale, scale_unit) || !aligned(c->page_table, 4) || !aligned(c->lens, 4) || !aligned(c->n_new, 4))
    return QSA_ERR_MISALIGNED;
  return QSA_OK;
}
static qsa_status check_cache_pointers(const qsa_kv_cache* c) { return check_cache_pointers(c, 16, 4, true); }
static qsa_status check_cache_pointers(const qsa_kv4_cache* c, bool values = true) {
  return check_cache_pointers(c, 32, 16, values);
}

// Rows of 16-bit floats read by 16-byte loads.
static qsa_status check_rows(const qsa_rows* r) {
  if (!r || !r->data) return QSA_ERR_INVALID_ARG;
  if (r->stride_b < 0 || r->stride_n < 0 || r->stride_h < 0) return QSA_ERR_INVALID_ARG;
  if (!aligned(r->data, 16) || r->stride_b % 8 != 0 || r->stride_n % 8 != 0 || r->stride_h % 8 != 0)
    return QSA_ERR_MISALIGNED;
  return QSA_OK;
}

static qsa::KvCacheArgs cache_args(const qsa_kv_cache* c) {
  return qsa::KvCacheArgs{c->k,     c->v,       c->k_scale,    c->v_scale, c->page_table, c->lens,
                          c->n_new, c->page_stride, c->n_pages, c->max_blocks, c->B, c->Hkv,
                          c->block, c->D};
}
static qsa::KvCacheArgs cache_args(const qsa_kv4_cache* c) {
  return qsa::KvCacheArgs{c->k,     c->v,       nullptr,    nullptr, c->page_table, c->lens,
                          c->n_new, c->page_stride, c->n_pages, c->max_blocks, c->B, c->Hkv,
                          c->block, c->D,       c->k_scale, c->v_scale};
}

static qsa::KvRows row_args(const qsa_rows* r) {
  return r ? qsa::KvRows{r->data, r->stride_b, r->stride_n, r->stride_h} : qsa::KvRows{nullptr, 0, 0, 0};
}

// Both appends: `grid` and `launch` are the cache's own.
template <class Cache, class Grid, class Launch>
static qsa_status run_append(const Cache* cache, const qsa_rows* k, const qsa_rows* v, const qsa_rows* q, int32_t n,
                             int32_t Hq, qsa_dtype dtype, const float* cos, const float* sin, int32_t rot,
                             int32_t max_pos, int32_t interleaved, const int32_t* offset, void* q_out, uint16_t* kb,
                             qsa_stream_t stream, Grid grid, Launch launch) {
  qsa_status st = check_cache_sizes(cache, n);
  if (st != QSA_OK) return st;
  if (rot < 0 || max_pos < 0 || (q && Hq < 1)) return QSA_ERR_INVALID_ARG;
  if (dtype != QSA_F16 && dtype != QSA_BF16) return QSA_ERR_INVALID_ARG;
  if (rot % 16 != 0 || rot > cache->D) return QSA_ERR_UNSUPPORTED_GEOMETRY;
  qsa::KvAppendProblem p{};
  p.cache = cache_args(cache);
  p.q = row_args(q);
  p.n = n;
  p.Hq = q ? Hq : 0;
  if (cache->B == 0 || n == 0) return QSA_OK;
  int64_t units = 0;
  int32_t per_seq = 0;
  if (grid(p, &units, &per_seq) > 0x7FFFFFFFLL) return QSA_ERR_UNSUPPORTED_GEOMETRY;
  if ((st = check_cache_pointers(cache)) != QSA_OK) return st;
  if ((st = check_rows(k)) != QSA_OK || (st = check_rows(v)) != QSA_OK) return st;
  if (q && ((st = check_rows(q)) != QSA_OK)) return st;
  if ((q != nullptr) != (q_out != nullptr)) return QSA_ERR_INVALID_ARG;
  if (rot > 0 && (!cos || !sin)) return QSA_ERR_INVALID_ARG;
  if (!aligned(q_out, 16) || !aligned(kb, 2) || !aligned(cos, 16) || !aligned(sin, 16) || !aligned(offset, 4))
    return QSA_ERR_MISALIGNED;
  p.k = row_args(k);
  p.v = row_args(v);
  p.rot = rot;
  p.max_pos = max_pos;
  p.bf16 = dtype == QSA_BF16;
  p.interleaved = interleaved != 0;
  p.cos = cos;
  p.sin = sin;
  p.q_out = q_out;
  p.kb = kb;
  p.offset = offset;
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  return from_cuda(launch(p, *dev, as_cuda(stream)));
}

// Both attentions.
template <class Cache, class Bytes, class Launch>
static qsa_status run_attend(const Cache* cache, const qsa_rows* q, int32_t n, int32_t Hq, qsa_dtype dtype,
                             float scale, const int32_t* ids, int32_t n_lists, int32_t k, void* out, float* lse,
                             void* workspace, size_t workspace_bytes, qsa_stream_t stream, Bytes bytes,
                             Launch launch) {
  qsa_status st = check_cache_sizes(cache, n);
  if (st != QSA_OK) return st;
  if (Hq < 1 || (dtype != QSA_F16 && dtype != QSA_BF16)) return QSA_ERR_INVALID_ARG;
  if (Hq % cache->Hkv != 0) return QSA_ERR_INVALID_ARG;
  if (ids && (k < 1 || (n_lists != 1 && n_lists != cache->Hkv))) return QSA_ERR_INVALID_ARG;
  if (Hq / cache->Hkv > qsa::kKvMaxGroup || (ids && k > (1 << 20))) return QSA_ERR_UNSUPPORTED_GEOMETRY;
  if (cache->B == 0 || n == 0) return QSA_OK;
  if (!(scale - scale == 0.0f)) return QSA_ERR_INVALID_ARG;
  if ((st = check_cache_pointers(cache)) != QSA_OK) return st;
  if (cache->n_pages < 1 || cache->max_blocks < 1) return QSA_ERR_INVALID_ARG;
  if ((st = check_rows(q)) != QSA_OK) return st;
  if (!out || !workspace || workspace_bytes < bytes(cache->B, n, Hq, cache->Hkv, cache->D)) return QSA_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(ids, 4) || !aligned(workspace, 16))
    return QSA_ERR_MISALIGNED;
  qsa::KvAttendProblem p{};
  p.cache = cache_args(cache);
  p.q = row_args(q);
  p.n = n;
  p.Hq = Hq;
  p.bf16 = dtype == QSA_BF16;
  p.scale = scale;
  p.ids = ids;
  p.n_lists = ids ? n_lists : 1;
  p.k = ids ? k : 0;
  p.out = out;
  p.lse = lse;
  p.workspace = workspace;
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  return from_cuda(launch(p, *dev, as_cuda(stream)));
}

extern "C" {

int qsa_abi_version(void) { return QSA_ABI_VERSION; }

const char* qsa_last_cuda_error(void) { return t_last_cuda_error; }

const char* qsa_status_str(qsa_status s) {
  switch (s) {
    case QSA_OK: return "QSA_OK";
    case QSA_ERR_INVALID_ARG: return "QSA_ERR_INVALID_ARG";
    case QSA_ERR_UNSUPPORTED_GEOMETRY: return "QSA_ERR_UNSUPPORTED_GEOMETRY";
    case QSA_ERR_UNSUPPORTED_ARCH: return "QSA_ERR_UNSUPPORTED_ARCH";
    case QSA_ERR_MISALIGNED: return "QSA_ERR_MISALIGNED";
    case QSA_ERR_CUDA: return "QSA_ERR_CUDA";
    case QSA_ERR_TIMEOUT: return "QSA_ERR_TIMEOUT";
  }
  return "QSA_ERR_UNKNOWN";
}

const char* qsa_arm(void) {
  thread_local char buf[1024];
  int n = snprintf(buf, sizeof buf,
                   "sm_103a: TMA + tcgen05.mma kind::f16 (M128, fp32 in TMEM) scorer with fused "
                   "ReLU/head-sum epilogue; fp32 pinned-order tail (+1e9); exact top-k select "
                   "(one warp for rows of <= 64 blocks, threshold + rank for k <= 128, radix "
                   "select otherwise; "
                   "block-index tie-break); cvt.rn fp32->fp16 stage | last call on this thread: ");
  if (!t_plan_any) {
    snprintf(buf + n, sizeof buf - n, "none");
  } else if (t_plan_n == 0) {
    snprintf(buf + n, sizeof buf - n, "no launch");
  } else {
    n += snprintf(buf + n, sizeof buf - n, "%d launch%s: ", t_plan_n, t_plan_n == 1 ? "" : "es");
    for (int i = 0; i < t_plan_n && n < static_cast<int>(sizeof buf); ++i)
      n += snprintf(buf + n, sizeof buf - n, "%s%s", i ? " -> " : "", t_plan[i]);
  }
  return buf;
}

int64_t qsa_num_blocks(int64_t n_kv, int32_t block) {
  if (n_kv < 0 || block < 1) return -1;
  return n_kv / block + (n_kv % block != 0 ? 1 : 0);
}

qsa_status qsa_f32_to_f16(const float* src, uint16_t* dst, int64_t n, qsa_stream_t stream) {
  if (n < 0) return QSA_ERR_INVALID_ARG;
  if (n == 0) return QSA_OK;
  if (!src || !dst) return QSA_ERR_INVALID_ARG;
  if (!aligned(src, 4) || !aligned(dst, 2)) return QSA_ERR_MISALIGNED;
  const DeviceInfo* dev = nullptr;
  qsa_status st = device_or_error(&dev);
  if (st != QSA_OK) return st;
  return from_cuda(qsa::launch_convert(src, dst, n, *dev, as_cuda(stream)));
}

qsa_status qsa_block_scores(const uint16_t* q, const uint16_t* kb, int32_t nq, int32_t H,
                            int32_t D, int64_t n_kv, int32_t block, float* scores,
                            qsa_stream_t stream) {
  Geometry g;
  qsa_status st = check_scores(q, kb, nq, H, D, n_kv, block, scores, &g);
  if (st != QSA_OK || nq == 0 || g.nb == 0) return st;
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  return run_scores(q, kb, nq, H, D, g, scores, *dev, as_cuda(stream));
}

qsa_status qsa_select(const float* scores, int32_t nq, int32_t nb, int32_t k, int32_t* ids,
                      qsa_stream_t stream) {
  qsa_status st = check_select(scores, nq, nb, k, ids);
  if (st != QSA_OK || nq == 0) return st;
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  return from_cuda(qsa::launch_select(scores, nq, nb, k, ids, *dev, as_cuda(stream)));
}

qsa_status qsa_score_select(const uint16_t* q, const uint16_t* kb, int32_t nq, int32_t H,
                            int32_t D, int64_t n_kv, int32_t block, int32_t k, float* scores,
                            int32_t* ids, qsa_stream_t stream) {
  Geometry g;
  qsa_status st = check_scores(q, kb, nq, H, D, n_kv, block, scores, &g);
  if (st != QSA_OK) return st;
  if ((st = check_select(scores, nq, g.nb, k, ids)) != QSA_OK) return st;
  if (nq == 0) return QSA_OK;
  if (g.nb > 0 && (!q || !kb)) return QSA_ERR_INVALID_ARG;
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  if (g.nb > 0 && use_separate(nq, H, *dev))
    return run_separate(q, kb, nq, H, D, g, k, scores, ids, *dev, as_cuda(stream));
  qsa::FusedProblem p{nullptr, q,       nullptr,  kb, scores, ids, nq, H, D, g.nb, g.n_full,
                      g.has_tail, k, 1, 0};
  return from_cuda(qsa::launch_fused(p, *dev, as_cuda(stream)));
}

qsa_status qsa_select_step(const float* q32, uint16_t* q16, const uint16_t* kb, int32_t nq,
                           int32_t H, int32_t D, int64_t n_kv, int32_t block, int32_t k,
                           float* scores, int32_t* ids, qsa_stream_t stream) {
  Geometry g;
  // q16 is optional here; the scoring checks see the (aligned) q32 in its place.
  qsa_status st = check_scores(reinterpret_cast<const uint16_t*>(q32), kb, nq, H, D, n_kv, block,
                               scores, &g);
  if (st != QSA_OK) return st;
  if ((st = check_select(scores, nq, g.nb, k, ids)) != QSA_OK) return st;
  if (nq == 0) return QSA_OK;
  if (!q32) return QSA_ERR_INVALID_ARG;
  if (!aligned(q32, 16) || !aligned(q16, 16)) return QSA_ERR_MISALIGNED;
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  if (q16 && g.nb > 0 && use_separate(nq, H, *dev)) {
    cudaStream_t s = as_cuda(stream);
    const int64_t n = static_cast<int64_t>(nq) * H * D;
    if ((st = from_cuda(qsa::launch_convert(q32, q16, n, *dev, s))) != QSA_OK) return st;
    return run_separate(q16, kb, nq, H, D, g, k, scores, ids, *dev, s);
  }
  qsa::FusedProblem p{q32, nullptr, q16, kb, scores, ids, nq, H, D, g.nb, g.n_full,
                      g.has_tail, k, 1, 0};
  return from_cuda(qsa::launch_fused(p, *dev, as_cuda(stream)));
}

int32_t qsa_select_step_launches(int32_t nq, int32_t H, int32_t D, int64_t n_kv, int32_t block,
                                 int32_t k, int32_t with_q16) {
  if (nq < 0 || n_kv < 0 || block < 1 || H < 1 || D < 1 || k < 1) return -1;
  if (!supported_heads(H) || D % 16 != 0 || D < 16 || D > 256 || k > qsa::kMaxSelectK) return -1;
  const int64_t nb = n_kv / block + (n_kv % block != 0 ? 1 : 0);
  if (nb > qsa::kMaxSelectNb || static_cast<int64_t>(nq) * H > 0x7FFFFFFFLL) return -1;
  if (nq == 0 || nb == 0) return 0;
  const DeviceInfo* dev = nullptr;
  if (device_or_error(&dev, false) != QSA_OK) return -1;
  if (!with_q16 || !use_separate(nq, H, *dev)) return 1;
  // convert (nq * H * D is a multiple of 8: one vector launch), the score
  // kernel when there are full blocks, the tail kernel when there is a tail
  // that the select does not score itself, and the select.
  const bool tail_kernel = n_kv % block != 0 && !qsa::select_scores_tail(nq, static_cast<int32_t>(nb), k);
  return 1 + (n_kv / block > 0 ? 1 : 0) + (tail_kernel ? 1 : 0) + 1;
}

// Shared by the two batched entry points: batch count and kb stride rules.
static qsa_status check_batches(int32_t n_batches, int64_t kb_batch_stride, int64_t nb, int32_t D) {
  if (n_batches < 0 || kb_batch_stride < 0) return QSA_ERR_INVALID_ARG;
  if (kb_batch_stride != 0 && kb_batch_stride < nb * D) return QSA_ERR_INVALID_ARG;
  if (kb_batch_stride % 8 != 0) return QSA_ERR_MISALIGNED;
  return QSA_OK;
}

qsa_status qsa_score_select_batched(const uint16_t* q, const uint16_t* kb, int64_t kb_batch_stride,
                                    int32_t n_batches, int32_t nq, int32_t H, int32_t D,
                                    int64_t n_kv, int32_t block, int32_t k, float* scores,
                                    int32_t* ids, qsa_stream_t stream) {
  Geometry g;
  qsa_status st = check_scores(q, kb, nq, H, D, n_kv, block, scores, &g);
  if (st != QSA_OK) return st;
  if ((st = check_select(scores, nq, g.nb, k, ids)) != QSA_OK) return st;
  if ((st = check_batches(n_batches, kb_batch_stride, g.nb, D)) != QSA_OK) return st;
  if (nq == 0 || n_batches == 0) return QSA_OK;
  if (static_cast<int64_t>(n_batches) * nq * H > 0x7FFFFFFFLL) return QSA_ERR_UNSUPPORTED_GEOMETRY;
  if (g.nb > 0 && (!q || !kb)) return QSA_ERR_INVALID_ARG;
  // Batches sharing one kb: one step over n_batches * nq queries.
  if (kb_batch_stride == 0)
    return qsa_score_select(q, kb, n_batches * nq, H, D, n_kv, block, k, scores, ids, stream);
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  if (batched_chain_ok(n_batches, nq, H, D, g, k, kb_batch_stride, *dev))
    return run_batched_chain(q, kb, kb_batch_stride, n_batches, nq, H, D, g, k, scores, ids, *dev,
                             as_cuda(stream));
  qsa::FusedProblem p{nullptr, q,       nullptr,  kb, scores, ids, nq, H, D, g.nb, g.n_full,
                      g.has_tail, k, n_batches, kb_batch_stride};
  return from_cuda(qsa::launch_fused(p, *dev, as_cuda(stream)));
}

qsa_status qsa_select_step_batched(const float* q32, uint16_t* q16, const uint16_t* kb,
                                   int64_t kb_batch_stride, int32_t n_batches, int32_t nq,
                                   int32_t H, int32_t D, int64_t n_kv, int32_t block, int32_t k,
                                   float* scores, int32_t* ids, qsa_stream_t stream) {
  Geometry g;
  qsa_status st = check_scores(reinterpret_cast<const uint16_t*>(q32), kb, nq, H, D, n_kv, block,
                               scores, &g);
  if (st != QSA_OK) return st;
  if ((st = check_select(scores, nq, g.nb, k, ids)) != QSA_OK) return st;
  if ((st = check_batches(n_batches, kb_batch_stride, g.nb, D)) != QSA_OK) return st;
  if (nq == 0 || n_batches == 0) return QSA_OK;
  if (static_cast<int64_t>(n_batches) * nq * H > 0x7FFFFFFFLL) return QSA_ERR_UNSUPPORTED_GEOMETRY;
  if (!q32) return QSA_ERR_INVALID_ARG;
  if (!aligned(q32, 16) || !aligned(q16, 16)) return QSA_ERR_MISALIGNED;
  // Batches sharing one kb are one step over n_batches * nq queries (the
  // buffers are laid out as such): it takes the single-step plan, the chain
  // of separate kernels when it is large and q16 is given.
  if (kb_batch_stride == 0)
    return qsa_select_step(q32, q16, kb, n_batches * nq, H, D, n_kv, block, k, scores, ids, stream);
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  if (q16 && batched_chain_ok(n_batches, nq, H, D, g, k, kb_batch_stride, *dev)) {
    cudaStream_t s = as_cuda(stream);
    const int64_t n = static_cast<int64_t>(n_batches) * nq * H * D;
    if ((st = from_cuda(qsa::launch_convert(q32, q16, n, *dev, s))) != QSA_OK) return st;
    return run_batched_chain(q16, kb, kb_batch_stride, n_batches, nq, H, D, g, k, scores, ids, *dev, s);
  }
  qsa::FusedProblem p{q32, nullptr, q16, kb, scores, ids, nq, H, D, g.nb, g.n_full,
                      g.has_tail, k, n_batches, kb_batch_stride};
  return from_cuda(qsa::launch_fused(p, *dev, as_cuda(stream)));
}

qsa_status qsa_select_step_host(const float* q32_host, const uint16_t* kb_host, int32_t nq,
                                int32_t H, int32_t D, int64_t n_kv, int32_t block, int32_t k,
                                float* scores_host, int32_t* ids_host, float* q32_dev,
                                uint16_t* q16_dev, uint16_t* kb_dev, float* scores_dev,
                                int32_t* ids_dev, qsa_stream_t stream) {
  Geometry g;
  qsa_status st = check_scores(reinterpret_cast<const uint16_t*>(q32_dev), kb_dev, nq, H, D, n_kv,
                               block, scores_dev, &g);
  if (st != QSA_OK) return st;
  if ((st = check_select(scores_dev, nq, g.nb, k, ids_dev)) != QSA_OK) return st;
  if (nq == 0) return QSA_OK;
  if (!q32_host || !ids_host || !q32_dev || !ids_dev) return QSA_ERR_INVALID_ARG;
  if (g.nb > 0 && !kb_host) return QSA_ERR_INVALID_ARG;
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  cudaStream_t s = as_cuda(stream);
  const size_t q_bytes = static_cast<size_t>(nq) * H * D * sizeof(float);
  const size_t kb_bytes = static_cast<size_t>(g.nb) * D * sizeof(uint16_t);
  const size_t s_bytes = static_cast<size_t>(nq) * g.nb * sizeof(float);
  const size_t id_bytes = static_cast<size_t>(nq) * k * sizeof(int32_t);
  if (cudaMemcpyAsync(q32_dev, q32_host, q_bytes, cudaMemcpyHostToDevice, s) != cudaSuccess)
    return cuda_fail(cudaGetLastError());
  if (kb_bytes &&
      cudaMemcpyAsync(kb_dev, kb_host, kb_bytes, cudaMemcpyHostToDevice, s) != cudaSuccess)
    return cuda_fail(cudaGetLastError());
  st = qsa_select_step(q32_dev, q16_dev, kb_dev, nq, H, D, n_kv, block, k, scores_dev, ids_dev,
                       stream);
  if (st != QSA_OK) return st;
  if (s_bytes && scores_host &&
      cudaMemcpyAsync(scores_host, scores_dev, s_bytes, cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return cuda_fail(cudaGetLastError());
  if (cudaMemcpyAsync(ids_host, ids_dev, id_bytes, cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return cuda_fail(cudaGetLastError());
  return QSA_OK;
}

qsa_status qsa_select_step_host_packed(const void* in_host, int32_t nq, int32_t H, int32_t D,
                                       int64_t n_kv, int32_t block, int32_t k, void* out_host,
                                       int32_t with_scores, void* in_dev, uint16_t* q16_dev,
                                       void* out_dev, qsa_stream_t stream) {
  if (nq < 0 || H < 1 || D < 1) return QSA_ERR_INVALID_ARG;
  const int64_t nb = qsa_num_blocks(n_kv, block);
  if (nb < 0) return QSA_ERR_INVALID_ARG;
  const size_t q_bytes = static_cast<size_t>(nq) * H * D * sizeof(float);
  const size_t kb_bytes = static_cast<size_t>(nb) * D * sizeof(uint16_t);
  const size_t s_bytes = static_cast<size_t>(nq) * nb * sizeof(float);
  const size_t id_bytes = static_cast<size_t>(nq) * (k > 0 ? k : 0) * sizeof(int32_t);
  char* in_d = static_cast<char*>(in_dev);
  char* out_d = static_cast<char*>(out_dev);
  float* q32_dev = reinterpret_cast<float*>(in_d);
  uint16_t* kb_dev = in_d ? reinterpret_cast<uint16_t*>(in_d + q_bytes) : nullptr;
  float* scores_dev = reinterpret_cast<float*>(out_d);
  int32_t* ids_dev = out_d ? reinterpret_cast<int32_t*>(out_d + s_bytes) : nullptr;
  Geometry g;
  qsa_status st = check_scores(reinterpret_cast<const uint16_t*>(q32_dev), kb_dev, nq, H, D, n_kv,
                               block, scores_dev, &g);
  if (st != QSA_OK) return st;
  if ((st = check_select(scores_dev, nq, g.nb, k, ids_dev)) != QSA_OK) return st;
  if (nq == 0) return QSA_OK;
  if (!in_host || !out_host || !in_dev || !out_dev) return QSA_ERR_INVALID_ARG;
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  cudaStream_t s = as_cuda(stream);
  // One copy in (queries then keys), one copy out (scores then ids, or ids).
  if (cudaMemcpyAsync(in_dev, in_host, q_bytes + kb_bytes, cudaMemcpyHostToDevice, s) != cudaSuccess)
    return cuda_fail(cudaGetLastError());
  st = qsa_select_step(q32_dev, q16_dev, kb_dev, nq, H, D, n_kv, block, k, scores_dev, ids_dev,
                       stream);
  if (st != QSA_OK) return st;
  const void* src = with_scores ? static_cast<const void*>(scores_dev) : static_cast<const void*>(ids_dev);
  const size_t out_bytes = with_scores ? s_bytes + id_bytes : id_bytes;
  if (cudaMemcpyAsync(out_host, src, out_bytes, cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return cuda_fail(cudaGetLastError());
  return QSA_OK;
}

// Shape rules of the split reduce; fills *ws with the workspace it needs.
static qsa_status check_split(int32_t G, int32_t R, int32_t B, int32_t C, size_t* ws) {
  if (G < 0 || R < 1 || B < 1 || C < 1) return QSA_ERR_INVALID_ARG;
  if (R > qsa::kSrMaxRows || C % 4 != 0 || C < 4 || G > 65535 ||
      static_cast<int64_t>(R) * C > 4LL * qsa::kSrMaxQuadsPerThread * 256)
    return QSA_ERR_UNSUPPORTED_GEOMETRY;
  *ws = qsa::split_reduce_workspace_bytes(G, R, B, C);
  return QSA_OK;
}

size_t qsa_split_reduce_workspace_bytes(int32_t G, int32_t R, int32_t B, int32_t C) {
  size_t ws = 0;
  return check_split(G, R, B, C, &ws) == QSA_OK ? ws : 0;
}

qsa_status qsa_split_reduce(const float* partial_max, const float* partial_sum,
                            const uint16_t* partial_out, int32_t G, int32_t R, int32_t B,
                            int32_t C, float* out, void* workspace, size_t workspace_bytes,
                            qsa_stream_t stream) {
  size_t need = 0;
  qsa_status st = check_split(G, R, B, C, &need);
  if (st != QSA_OK) return st;
  if (G == 0) return QSA_OK;
  if (!partial_max || !partial_sum || !partial_out || !out) return QSA_ERR_INVALID_ARG;
  if (need > 0 && (!workspace || workspace_bytes < need)) return QSA_ERR_INVALID_ARG;
  if (!aligned(partial_max, 4) || !aligned(partial_sum, 4) || !aligned(partial_out, 8) ||
      !aligned(out, 16) || (need > 0 && !aligned(workspace, 16)))
    return QSA_ERR_MISALIGNED;
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  qsa::SplitReduceProblem p{partial_max, partial_sum, partial_out, out, workspace, G, R, B, C};
  return from_cuda(qsa::launch_split_reduce(p, *dev, as_cuda(stream)));
}

qsa_status qsa_split_reduce_static(const float* partial_max, const float* partial_sum,
                                   const uint16_t* partial_out, int32_t G, int32_t R, int32_t B,
                                   int32_t C, float* out, qsa_stream_t stream) {
  size_t need = 0;
  qsa_status st = check_split(G, R, B, C, &need);
  if (st != QSA_OK) return st;
  if (need > QSA_SPLIT_STATIC_SCRATCH_BYTES) return QSA_ERR_UNSUPPORTED_GEOMETRY;
  if (G == 0) return QSA_OK;
  if (!partial_max || !partial_sum || !partial_out || !out) return QSA_ERR_INVALID_ARG;
  if (!aligned(partial_max, 4) || !aligned(partial_sum, 4) || !aligned(partial_out, 8) ||
      !aligned(out, 16))
    return QSA_ERR_MISALIGNED;
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  cudaError_t e = cudaSuccess;
  void* scratch = qsa::split_static_scratch(&e);
  if (!scratch) return cuda_fail(e);
  cudaStream_t s = as_cuda(stream);
  if (need > 0) {
    // The counters lead the workspace layout and must be zero; an earlier
    // call of another shape may have left partials where they now sit.
    const size_t counters = (static_cast<size_t>(G) * R * sizeof(uint32_t) + 15) & ~static_cast<size_t>(15);
    if ((e = cudaMemsetAsync(scratch, 0, counters, s)) != cudaSuccess) return cuda_fail(e);
  }
  qsa::SplitReduceProblem p{partial_max, partial_sum, partial_out, out, scratch, G, R, B, C};
  return from_cuda(qsa::launch_split_reduce(p, *dev, s));
}

// -------------------------------------------------------- the paged caches
qsa_status qsa_kv_append(const qsa_kv_cache* cache, const qsa_rows* k, const qsa_rows* v, const qsa_rows* q,
                         int32_t n, int32_t Hq, qsa_dtype dtype, const float* cos, const float* sin,
                         int32_t rot, int32_t max_pos, int32_t interleaved, void* q_out, uint16_t* kb,
                         qsa_stream_t stream) {
  return run_append(cache, k, v, q, n, Hq, dtype, cos, sin, rot, max_pos, interleaved, nullptr, q_out, kb, stream,
                    qsa::kv_append_grid, qsa::launch_kv_append);
}

qsa_status qsa_kv4_append(const qsa_kv4_cache* cache, const qsa_rows* k, const qsa_rows* v, const qsa_rows* q,
                          int32_t n, int32_t Hq, qsa_dtype dtype, const float* cos, const float* sin,
                          int32_t rot, int32_t max_pos, int32_t interleaved, const int32_t* offset, void* q_out,
                          uint16_t* kb, qsa_stream_t stream) {
  return run_append(cache, k, v, q, n, Hq, dtype, cos, sin, rot, max_pos, interleaved, offset, q_out, kb, stream,
                    qsa::kv4_append_grid, qsa::launch_kv4_append);
}

qsa_status qsa_kv4_read(const qsa_kv4_cache* cache, int32_t n, qsa_dtype dtype, void* k_out, void* v_out,
                        qsa_stream_t stream) {
  qsa_status st = check_cache_sizes(cache, n);
  if (st != QSA_OK) return st;
  if (dtype != QSA_F16 && dtype != QSA_BF16) return QSA_ERR_INVALID_ARG;
  if (cache->B == 0 || n == 0) return QSA_OK;
  const qsa::KvCacheArgs c = cache_args(cache);
  if (qsa::kv4_read_grid(c, n) > 0x7FFFFFFFLL) return QSA_ERR_UNSUPPORTED_GEOMETRY;
  if ((st = check_cache_pointers(cache)) != QSA_OK) return st;
  if (!k_out || !v_out) return QSA_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return QSA_ERR_MISALIGNED;
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  return from_cuda(qsa::launch_kv4_read(c, n, dtype == QSA_BF16, k_out, v_out, *dev, as_cuda(stream)));
}

size_t qsa_kv_attend_workspace_bytes(int32_t B, int32_t n, int32_t Hq, int32_t Hkv, int32_t D) {
  return qsa::kv_attend_workspace_bytes(B, n, Hq, Hkv, D);
}
size_t qsa_kv4_attend_workspace_bytes(int32_t B, int32_t n, int32_t Hq, int32_t Hkv, int32_t D) {
  return qsa::kv4_attend_workspace_bytes(B, n, Hq, Hkv, D);
}

qsa_status qsa_kv_attend(const qsa_kv_cache* cache, const qsa_rows* q, int32_t n, int32_t Hq, qsa_dtype dtype,
                         float scale, const int32_t* ids, int32_t n_lists, int32_t k, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, qsa_stream_t stream) {
  return run_attend(cache, q, n, Hq, dtype, scale, ids, n_lists, k, out, lse, workspace, workspace_bytes, stream,
                    qsa::kv_attend_workspace_bytes, qsa::launch_kv_attend);
}

qsa_status qsa_kv4_attend(const qsa_kv4_cache* cache, const qsa_rows* q, int32_t n, int32_t Hq, qsa_dtype dtype,
                          float scale, const int32_t* ids, int32_t n_lists, int32_t k, void* out, float* lse,
                          void* workspace, size_t workspace_bytes, qsa_stream_t stream) {
  return run_attend(cache, q, n, Hq, dtype, scale, ids, n_lists, k, out, lse, workspace, workspace_bytes, stream,
                    qsa::kv4_attend_workspace_bytes, qsa::launch_kv4_attend);
}

qsa_status qsa_kv4_weights(const qsa_kv4_cache* cache, const qsa_rows* q, int32_t n, int32_t Hq, qsa_dtype dtype,
                           float scale, const float* lse, float decay, float* weights, qsa_stream_t stream) {
  qsa_status st = check_cache_sizes(cache, n);
  if (st != QSA_OK) return st;
  if (Hq < 1 || (dtype != QSA_F16 && dtype != QSA_BF16)) return QSA_ERR_INVALID_ARG;
  if (Hq % cache->Hkv != 0) return QSA_ERR_INVALID_ARG;
  if (Hq / cache->Hkv > qsa::kKvMaxGroup) return QSA_ERR_UNSUPPORTED_GEOMETRY;
  if (cache->B == 0 || n == 0) return QSA_OK;
  if (!(scale - scale == 0.0f) || !(decay - decay == 0.0f) || decay < 0.0f) return QSA_ERR_INVALID_ARG;
  if ((st = check_cache_pointers(cache, false)) != QSA_OK) return st;
  if (cache->n_pages < 1 || cache->max_blocks < 1) return QSA_ERR_INVALID_ARG;
  if ((st = check_rows(q)) != QSA_OK) return st;
  if (!lse || !weights) return QSA_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(weights, 16)) return QSA_ERR_MISALIGNED;
  const qsa::Kv4WeightsProblem p{cache_args(cache), row_args(q), n, Hq, dtype == QSA_BF16, scale, decay, lse, weights};
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  return from_cuda(qsa::launch_kv4_weights(p, *dev, as_cuda(stream)));
}

size_t qsa_kv4_evict_workspace_bytes(int32_t B, int32_t Hkv, int32_t budget) {
  return qsa::kv4_evict_workspace_bytes(B, Hkv, budget);
}

qsa_status qsa_kv4_evict(const qsa_kv4_cache* cache, float* weights, int32_t budget, int32_t sink, int32_t recent,
                         int32_t* lens_out, int32_t* offset, void* workspace, size_t workspace_bytes,
                         qsa_stream_t stream) {
  qsa_status st = check_cache_sizes(cache, 1);
  if (st != QSA_OK) return st;
  if (budget < 1 || sink < 0 || recent < 0 || static_cast<int64_t>(sink) + recent > budget) return QSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(cache->B) * cache->Hkv > (1 << 27)) return QSA_ERR_UNSUPPORTED_GEOMETRY;
  if (cache->B == 0) return QSA_OK;
  if ((st = check_cache_pointers(cache)) != QSA_OK) return st;
  if (cache->n_pages < 1 || cache->max_blocks < 1) return QSA_ERR_INVALID_ARG;
  if (!weights || !lens_out) return QSA_ERR_INVALID_ARG;
  // (No sequence is longer than its page table.)
  if (budget < cache->max_blocks * cache->block &&
      (!workspace || workspace_bytes < qsa::kv4_evict_workspace_bytes(cache->B, cache->Hkv, budget)))
    return QSA_ERR_INVALID_ARG;
  if (!aligned(weights, 16) || !aligned(lens_out, 4) || !aligned(offset, 4) || !aligned(workspace, 16))
    return QSA_ERR_MISALIGNED;
  // Each sequence's length is read while others' are written.
  const uintptr_t ints[3] = {reinterpret_cast<uintptr_t>(cache->lens), reinterpret_cast<uintptr_t>(lens_out),
                             reinterpret_cast<uintptr_t>(offset)};
  for (int i = 0; i < 3; ++i) {
    const uintptr_t x = ints[i], y = ints[(i + 1) % 3];
    if (x && y && (x > y ? x - y : y - x) < sizeof(int32_t) * static_cast<uintptr_t>(cache->B)) return QSA_ERR_INVALID_ARG;
  }
  const qsa::Kv4EvictProblem p{cache_args(cache), weights,  budget, sink,
                               recent,            lens_out, offset, static_cast<int32_t*>(workspace)};
  const DeviceInfo* dev = nullptr;
  if ((st = device_or_error(&dev)) != QSA_OK) return st;
  return from_cuda(qsa::launch_kv4_evict(p, *dev, as_cuda(stream)));
}

qsa_status qsa_selftest_bounded_wait(uint64_t timeout_ns, qsa_stream_t stream) {
  if (timeout_ns == 0 || timeout_ns > 1000000000ull) return QSA_ERR_INVALID_ARG;
  const DeviceInfo* dev = nullptr;
  qsa_status st = device_or_error(&dev);
  if (st != QSA_OK) return st;
  return from_cuda(qsa::launch_selftest_wait(*dev, timeout_ns, as_cuda(stream)));
}

qsa_status qsa_device_status(int clear, uint32_t* bits, qsa_stream_t stream) {
  const DeviceInfo* dev = nullptr;
  qsa_status st = device_or_error(&dev, false);
  if (st != QSA_OK) return st;
  cudaError_t e = cudaStreamSynchronize(as_cuda(stream));
  if (e != cudaSuccess) return cuda_fail(e);
  uint32_t v = 0;
  if ((e = cudaMemcpy(&v, dev->status_word, sizeof(v), cudaMemcpyDeviceToHost)) != cudaSuccess)
    return cuda_fail(e);
  if (bits) *bits = v;
  if (v != 0 && clear) {
    if ((e = cudaMemset(dev->status_word, 0, sizeof(uint32_t))) != cudaSuccess ||
        (e = cudaDeviceSynchronize()) != cudaSuccess)
      return cuda_fail(e);
  }
  if (v == qsa::kKvIndexBit) return QSA_ERR_INVALID_ARG;
  return v == 0 ? QSA_OK : QSA_ERR_TIMEOUT;
}

}  // extern "C"
