// C entry points of libress.so: argument validation on the host, then kernel launches on
// the caller's stream.  Validation happens before any CUDA call, so a bad argument is
// reported without touching the device.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/ress.h"
#include "ress_common.cuh"
#include "ress_internal.h"

using ress::Dims;

namespace {

constexpr int32_t kAbiVersion = 5;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shape checks shared by every entry point.  On success fills d; *empty = true means
// there is no work (B = 0 or N = 0).
ress_status check_shape(const ress_shape *s, Dims *d, bool *empty) {
  if (s == nullptr) return RESS_ERR_INVALID_ARG;
  if (s->batch < 0 || s->seq_len < 0 || s->heads < 1) return RESS_ERR_INVALID_ARG;
  if (s->head_dim != ress::kHeadDim || s->block != ress::kBlock) return RESS_ERR_UNSUPPORTED;
  if (s->key_block != 0 && s->key_block != ress::kBlock && s->key_block != ress::kBlock / 2)
    return RESS_ERR_UNSUPPORTED;
  if (s->heads > ress::kMaxHeads) return RESS_ERR_UNSUPPORTED;
  d->B = s->batch;
  d->H = s->heads;
  d->N = s->seq_len;
  d->kb = s->key_block == 0 ? ress::kBlock : s->key_block;
  d->nq = (s->seq_len + ress::kBlock - 1) / ress::kBlock;
  d->nk = (s->seq_len + d->kb - 1) / d->kb;
  d->nb = d->nq;
  if (d->nk > ress::kMaxBlocks) return RESS_ERR_UNSUPPORTED;
  if (d->BH() > 65535) return RESS_ERR_UNSUPPORTED;  // grid.y limit of the block kernels
  if (d->BH() * d->nq * (long long)d->nk > 0x7fffffffffffll) return RESS_ERR_UNSUPPORTED;
  if (d->BH() * d->nq > 0x7fffffffll) return RESS_ERR_UNSUPPORTED;
  *empty = (d->B == 0 || d->N == 0);
  return RESS_OK;
}

bool ptr_ok(const void *p) { return p != nullptr && aligned16(p); }

ress_status from_cuda(cudaError_t e) { return e == cudaSuccess ? RESS_OK : RESS_ERR_CUDA; }

// Query rows of ress_masked_attn: the grid's limit, and the limits of check_shape for rows.
bool queries_ok(const Dims &d, int32_t q_len) {
  const long long nq = (1ll * q_len + ress::kBlock - 1) / ress::kBlock;
  return nq <= ress::kMaxBlocks && d.BH() * nq <= 0x7fffffffll;
}

bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// ------------------------------------------------------------ checks of the token operators
constexpr int32_t kMaxTokenHeads = 65536;

size_t dtype_bytes(int32_t dtype) {
  return dtype == RESS_BF16 || dtype == RESS_FP16 ? 2 : (dtype == RESS_FP32 ? 4 : 0);
}

bool plan_ok(const ress_rope_plan *r) {
  if (r == nullptr || r->head_dim < 2 || r->head_dim > RESS_MAX_TOKEN_DIM) return false;
  if (r->axes < 1 || r->axes > 3 || r->rot_dim < 2 || r->rot_dim > r->head_dim) return false;
  if (r->rot_dim % (2 * r->axes) != 0) return false;
  if (r->layout != RESS_ROPE_HALF && r->layout != RESS_ROPE_INTERLEAVED) return false;
  return r->amplitude > 0.f && !std::isinf(r->amplitude);
}

bool positions_ok(const ress_rope_plan *r, const int32_t *positions, int64_t stride_b) {
  if (positions == nullptr) return r->axes == 1;
  return aligned_to(positions, 4) && stride_b >= 0;
}

bool rows_ok(const ress_rows *r, size_t size) {
  return r != nullptr && r->ptr != nullptr && aligned_to(r->ptr, size) && r->stride_b >= 0 &&
         r->stride_h >= 0 && r->stride_t >= 0;
}

// An output view: its rows of `dim` elements must not overlap.  Taken from the smallest
// stride up, each stride has to reach past everything that the smaller ones span.
bool out_rows_ok(const ress_rows *r, size_t size, int64_t batch, int64_t heads, int64_t tokens,
                 int64_t dim) {
  if (!rows_ok(r, size)) return false;
  struct Axis {
    int64_t stride, count;
  } ax[3] = {{r->stride_b, batch}, {r->stride_h, heads}, {r->stride_t, tokens}};
  std::sort(ax, ax + 3, [](const Axis &x, const Axis &y) { return x.stride < y.stride; });
  int64_t span = dim;
  for (const Axis &x : ax) {
    if (x.count == 1) continue;
    if (x.stride < span || x.stride > ((int64_t)1 << 60) / x.count) return false;
    span += x.stride * (x.count - 1);
  }
  return true;
}

// Two views of one pointer that name the same rows (strides of single entries do not count).
bool same_rows(const ress_rows *x, const ress_rows *y, int64_t batch, int64_t heads, int64_t tokens) {
  return (batch == 1 || x->stride_b == y->stride_b) && (heads == 1 || x->stride_h == y->stride_h) &&
         (tokens == 1 || x->stride_t == y->stride_t);
}

}  // namespace

extern "C" {

int32_t ress_abi_version(void) { return kAbiVersion; }

const char *ress_status_string(ress_status status) {
  switch (status) {
    case RESS_OK: return "RESS_OK";
    case RESS_ERR_INVALID_ARG: return "RESS_ERR_INVALID_ARG";
    case RESS_ERR_UNSUPPORTED: return "RESS_ERR_UNSUPPORTED";
    case RESS_ERR_CUDA: return "RESS_ERR_CUDA";
    case RESS_ERR_DEVICE_BOUNDS: return "RESS_ERR_DEVICE_BOUNDS";
    case RESS_ERR_DEVICE_TIMEOUT: return "RESS_ERR_DEVICE_TIMEOUT";
  }
  return "RESS_ERR_UNKNOWN";
}

ress_status ress_head_gram(const ress_shape *shape, int32_t d_model, const float *w_o,
                           float *gram, ress_stream_t stream) {
  Dims d;
  bool empty;
  ress_status st = check_shape(shape, &d, &empty);
  if (st != RESS_OK) return st;
  if (d_model < 1 || !ptr_ok(w_o) || !ptr_ok(gram)) return RESS_ERR_INVALID_ARG;
  return from_cuda(ress::launch_head_gram(d.H, d_model, w_o, gram, (cudaStream_t)stream));
}

ress_status ress_token_gather(const ress_shape *shape, int32_t views, int32_t specials,
                              int32_t inverse, const void *src, void *dst, ress_stream_t stream) {
  Dims d;
  bool empty;
  ress_status st = check_shape(shape, &d, &empty);
  if (st != RESS_OK) return st;
  if (views < 1 || (d.N > 0 && d.N % views != 0)) return RESS_ERR_INVALID_ARG;
  if (specials < 0 || specials > d.N / views) return RESS_ERR_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return RESS_ERR_INVALID_ARG;
  if (empty) return RESS_OK;
  if (!ptr_ok(src) || !ptr_ok(dst) || src == dst) return RESS_ERR_INVALID_ARG;
  return from_cuda(ress::launch_token_gather(d, views, specials, inverse != 0, src, dst,
                                             (cudaStream_t)stream));
}

ress_status ress_pool_blocks(const ress_shape *shape, const void *q, const void *k,
                             const void *v, float *q_pool, float *k_pool, float *v_pool,
                             ress_stream_t stream) {
  Dims d;
  bool empty;
  ress_status st = check_shape(shape, &d, &empty);
  if (st != RESS_OK) return st;
  if (empty) return RESS_OK;
  if (!ptr_ok(q) || !ptr_ok(k) || !ptr_ok(v) || !ptr_ok(q_pool) || !ptr_ok(k_pool) ||
      !ptr_ok(v_pool))
    return RESS_ERR_INVALID_ARG;
  return from_cuda(ress::launch_pool(d, q, k, v, q_pool, k_pool, v_pool, (cudaStream_t)stream));
}

ress_status ress_block_scores(const ress_shape *shape, const float *q_pool, const float *k_pool,
                              const float *v_pool, float scale, float *P, float *v_bar,
                              ress_stream_t stream) {
  Dims d;
  bool empty;
  ress_status st = check_shape(shape, &d, &empty);
  if (st != RESS_OK) return st;
  if (empty) return RESS_OK;
  if (!ptr_ok(q_pool) || !ptr_ok(k_pool) || !ptr_ok(v_pool) || !ptr_ok(P) || !ptr_ok(v_bar))
    return RESS_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale != scale) return RESS_ERR_INVALID_ARG;
  return from_cuda(
      ress::launch_block_scores(d, q_pool, k_pool, v_pool, scale, P, v_bar, (cudaStream_t)stream));
}

size_t ress_drift_workspace_bytes(const ress_shape *shape) {
  Dims d;
  bool empty;
  if (check_shape(shape, &d, &empty) != RESS_OK || empty) return 0;
  return ress::drift_workspace_bytes(d);
}

ress_status ress_drift_scores(const ress_shape *shape, const float *P, const float *v_pool,
                              const float *v_bar, const float *gram, float *s, void *workspace,
                              size_t workspace_bytes, ress_stream_t stream) {
  Dims d;
  bool empty;
  ress_status st = check_shape(shape, &d, &empty);
  if (st != RESS_OK) return st;
  if (empty) return RESS_OK;
  if (!ptr_ok(P) || !ptr_ok(v_pool) || !ptr_ok(v_bar) || !ptr_ok(gram) || !ptr_ok(s) ||
      !ptr_ok(workspace))
    return RESS_ERR_INVALID_ARG;
  if (workspace_bytes < ress::drift_workspace_bytes(d)) return RESS_ERR_INVALID_ARG;
  return from_cuda(
      ress::launch_drift(d, P, v_pool, v_bar, gram, s, workspace, (cudaStream_t)stream));
}

ress_status ress_select_blocks(const ress_shape *shape, const ress_select_params *params,
                               const float *P, const float *s, const float *v_pool,
                               const float *v_bar, const float *gram, int32_t *kv_idx,
                               int32_t *kv_cnt, uint8_t *mask, int32_t *dev_err,
                               ress_stream_t stream) {
  Dims d;
  bool empty;
  ress_status st = check_shape(shape, &d, &empty);
  if (st != RESS_OK) return st;
  if (params == nullptr || params->budgets == nullptr) return RESS_ERR_INVALID_ARG;
  const int m = params->method;
  if (m != RESS_SELECT_MASS && m != RESS_SELECT_DRIFT && m != RESS_SELECT_RANDOM &&
      m != RESS_SELECT_CDF)
    return RESS_ERR_INVALID_ARG;
  if (m == RESS_SELECT_CDF && !(params->top_p > 0.f && params->top_p <= 1.f)) return RESS_ERR_INVALID_ARG;
  for (int h = 0; h < d.H; ++h)
    if (params->budgets[h] < 0 || params->budgets[h] > d.nk) return RESS_ERR_INVALID_ARG;
  const int obj = params->objective;
  if (obj != RESS_DRIFT_MINIMISE && obj != RESS_DRIFT_MAXIMISE_SWAPS && obj != RESS_DRIFT_MAXIMISE_FULL)
    return RESS_ERR_INVALID_ARG;
  if (obj != RESS_DRIFT_MINIMISE && m != RESS_SELECT_DRIFT) return RESS_ERR_INVALID_ARG;
  const bool want_drift = params->drift != nullptr;
  if (m == RESS_SELECT_DRIFT) {
    if (params->rounds < 0 || params->rounds > 64) return RESS_ERR_INVALID_ARG;
    if (!(params->rho > 0.f) || !(params->rho <= 1.f)) return RESS_ERR_INVALID_ARG;
  }
  if ((m == RESS_SELECT_DRIFT || want_drift) && !(params->eps > 0.f)) return RESS_ERR_INVALID_ARG;
  if (empty) return RESS_OK;
  if (!ptr_ok(P) || !ptr_ok(kv_idx) || !ptr_ok(kv_cnt)) return RESS_ERR_INVALID_ARG;
  if (mask != nullptr && !aligned16(mask)) return RESS_ERR_INVALID_ARG;
  if (dev_err != nullptr && (reinterpret_cast<uintptr_t>(dev_err) & 3u)) return RESS_ERR_INVALID_ARG;
  const bool restore = m == RESS_SELECT_DRIFT && params->rounds > 0;
  const bool state = restore || want_drift;  // the kernel tracks g, K and J
  if (m == RESS_SELECT_DRIFT && !ptr_ok(s)) return RESS_ERR_INVALID_ARG;
  if (state && (!ptr_ok(v_pool) || !ptr_ok(v_bar) || !ptr_ok(gram))) return RESS_ERR_INVALID_ARG;
  if (want_drift && !aligned16(params->drift)) return RESS_ERR_INVALID_ARG;
  ress::SelectLaunch a;
  a.method = m;
  a.rounds = m == RESS_SELECT_DRIFT ? params->rounds : 0;
  a.rho = params->rho;
  a.eps = (m == RESS_SELECT_DRIFT || want_drift) ? params->eps : 1e-4f;
  a.objective = obj;
  a.top_p = params->top_p;
  a.drift = params->drift;
  a.seed = params->seed;
  a.budgets = params->budgets;
  a.keep_k = params->keep_k;
  a.dense_q = params->dense_q;
  a.P = P;
  a.s = m == RESS_SELECT_DRIFT ? s : nullptr;
  a.vp = state ? v_pool : nullptr;
  a.vbar = state ? v_bar : nullptr;
  a.gram = state ? gram : nullptr;
  a.kv_idx = kv_idx;
  a.kv_cnt = kv_cnt;
  a.mask = mask;
  a.dev_err = dev_err;
  cudaError_t e = ress::launch_select(d, a, (cudaStream_t)stream);
  if (e == cudaErrorNotSupported) return RESS_ERR_UNSUPPORTED;
  return from_cuda(e);
}

ress_status ress_scores_select(const ress_shape *shape, const ress_select_params *params,
                               const float *q_pool, const float *k_pool, const float *v_pool,
                               float scale, float *P, float *v_bar, int32_t *kv_idx,
                               int32_t *kv_cnt, uint8_t *mask, int32_t *dev_err,
                               ress_stream_t stream) {
  Dims d;
  bool empty;
  ress_status st = check_shape(shape, &d, &empty);
  if (st != RESS_OK) return st;
  if (params == nullptr || params->budgets == nullptr) return RESS_ERR_INVALID_ARG;
  const int m = params->method;
  if (m == RESS_SELECT_DRIFT) return RESS_ERR_UNSUPPORTED;
  if (m != RESS_SELECT_MASS && m != RESS_SELECT_RANDOM && m != RESS_SELECT_CDF) return RESS_ERR_INVALID_ARG;
  if (m == RESS_SELECT_CDF && !(params->top_p > 0.f && params->top_p <= 1.f)) return RESS_ERR_INVALID_ARG;
  if (params->objective != RESS_DRIFT_MINIMISE || params->drift != nullptr) return RESS_ERR_INVALID_ARG;
  for (int h = 0; h < d.H; ++h)
    if (params->budgets[h] < 0 || params->budgets[h] > d.nk) return RESS_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale != scale) return RESS_ERR_INVALID_ARG;
  if (empty) return RESS_OK;
  if (!ptr_ok(q_pool) || !ptr_ok(k_pool) || !ptr_ok(kv_idx) || !ptr_ok(kv_cnt)) return RESS_ERR_INVALID_ARG;
  if (P != nullptr && !aligned16(P)) return RESS_ERR_INVALID_ARG;
  if (v_bar != nullptr && (!aligned16(v_bar) || !ptr_ok(v_pool))) return RESS_ERR_INVALID_ARG;
  if (mask != nullptr && !aligned16(mask)) return RESS_ERR_INVALID_ARG;
  if (dev_err != nullptr && (reinterpret_cast<uintptr_t>(dev_err) & 3u)) return RESS_ERR_INVALID_ARG;
  ress::ScoresSelectLaunch a;
  a.method = m;
  a.seed = params->seed;
  a.top_p = params->top_p;
  a.budgets = params->budgets;
  a.keep_k = params->keep_k;
  a.dense_q = params->dense_q;
  a.qp = q_pool;
  a.kp = k_pool;
  a.vp = v_bar ? v_pool : nullptr;
  a.scale = scale;
  a.P = P;
  a.vbar = v_bar;
  a.kv_idx = kv_idx;
  a.kv_cnt = kv_cnt;
  a.mask = mask;
  return from_cuda(ress::launch_scores_select(d, a, (cudaStream_t)stream));
}

size_t ress_drift_select_workspace_bytes(const ress_shape *shape) {
  Dims d;
  bool empty;
  if (check_shape(shape, &d, &empty) != RESS_OK) return 0;
  return ress::drift_select_workspace_bytes(d);
}

ress_status ress_drift_select(const ress_shape *shape, const ress_select_params *params,
                              const float *q_pool, const float *k_pool, const float *v_pool,
                              const float *gram, float scale, float *P, float *v_bar, float *s,
                              int32_t *kv_idx, int32_t *kv_cnt, uint8_t *mask, int32_t *dev_err,
                              void *workspace, size_t workspace_bytes, ress_stream_t stream) {
  Dims d;
  bool empty;
  ress_status st = check_shape(shape, &d, &empty);
  if (st != RESS_OK) return st;
  if (params == nullptr || params->budgets == nullptr) return RESS_ERR_INVALID_ARG;
  if (params->method != RESS_SELECT_DRIFT) return RESS_ERR_INVALID_ARG;
  for (int h = 0; h < d.H; ++h)
    if (params->budgets[h] < 0 || params->budgets[h] > d.nk) return RESS_ERR_INVALID_ARG;
  const int obj = params->objective;
  if (obj != RESS_DRIFT_MINIMISE && obj != RESS_DRIFT_MAXIMISE_SWAPS && obj != RESS_DRIFT_MAXIMISE_FULL)
    return RESS_ERR_INVALID_ARG;
  if (params->rounds < 0 || params->rounds > 64) return RESS_ERR_INVALID_ARG;
  if (!(params->rho > 0.f) || !(params->rho <= 1.f) || !(params->eps > 0.f)) return RESS_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale != scale) return RESS_ERR_INVALID_ARG;
  if (empty) return RESS_OK;
  if (!ptr_ok(q_pool) || !ptr_ok(k_pool) || !ptr_ok(v_pool) || !ptr_ok(gram) || !ptr_ok(kv_idx) ||
      !ptr_ok(kv_cnt) || !ptr_ok(workspace))
    return RESS_ERR_INVALID_ARG;
  if (workspace_bytes < ress::drift_select_workspace_bytes(d)) return RESS_ERR_INVALID_ARG;
  for (const void *o : {(const void *)P, (const void *)v_bar, (const void *)s, (const void *)mask,
                        (const void *)params->drift})
    if (o != nullptr && !aligned16(o)) return RESS_ERR_INVALID_ARG;
  if (dev_err != nullptr && (reinterpret_cast<uintptr_t>(dev_err) & 3u)) return RESS_ERR_INVALID_ARG;
  ress::DriftSelectLaunch a;
  a.sel.method = RESS_SELECT_DRIFT;
  a.sel.rounds = params->rounds;
  a.sel.rho = params->rho;
  a.sel.eps = params->eps;
  a.sel.objective = obj;
  a.sel.top_p = params->top_p;
  a.sel.drift = params->drift;
  a.sel.seed = params->seed;
  a.sel.budgets = params->budgets;
  a.sel.keep_k = params->keep_k;
  a.sel.dense_q = params->dense_q;
  a.sel.P = nullptr;
  a.sel.s = nullptr;
  a.sel.vp = v_pool;
  a.sel.vbar = nullptr;
  a.sel.gram = gram;
  a.sel.kv_idx = kv_idx;
  a.sel.kv_cnt = kv_cnt;
  a.sel.mask = mask;
  a.sel.dev_err = dev_err;
  a.qp = q_pool;
  a.kp = k_pool;
  a.scale = scale;
  a.P_out = P;
  a.s_out = s;
  a.vbar_out = v_bar;
  a.ws = workspace;
  cudaError_t e = ress::launch_drift_select(d, a, (cudaStream_t)stream);
  if (e == cudaErrorNotSupported) return RESS_ERR_UNSUPPORTED;
  return from_cuda(e);
}

ress_status ress_attn_schedule(const ress_shape *shape, const int32_t *kv_cnt, int32_t *work_order,
                               ress_stream_t stream) {
  Dims d;
  bool empty;
  ress_status st = check_shape(shape, &d, &empty);
  if (st != RESS_OK) return st;
  if (empty) return RESS_OK;
  if (!ptr_ok(kv_cnt) || !ptr_ok(work_order)) return RESS_ERR_INVALID_ARG;
  return from_cuda(ress::launch_schedule(d, kv_cnt, work_order, (cudaStream_t)stream));
}

ress_status ress_block_sparse_attn(const ress_shape *shape, const void *q, const void *k,
                                   const void *v, const int32_t *kv_idx, const int32_t *kv_cnt,
                                   const int32_t *work_order, float scale, void *out, float *lse,
                                   int32_t *dev_err, ress_stream_t stream) {
  Dims d;
  bool empty;
  ress_status st = check_shape(shape, &d, &empty);
  if (st != RESS_OK) return st;
  if (empty) return RESS_OK;
  if (!ptr_ok(q) || !ptr_ok(k) || !ptr_ok(v) || !ptr_ok(kv_idx) || !ptr_ok(kv_cnt) || !ptr_ok(out))
    return RESS_ERR_INVALID_ARG;
  if (work_order != nullptr && !aligned16(work_order)) return RESS_ERR_INVALID_ARG;
  if (lse != nullptr && !aligned16(lse)) return RESS_ERR_INVALID_ARG;
  if (dev_err != nullptr && (reinterpret_cast<uintptr_t>(dev_err) & 3u)) return RESS_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale != scale) return RESS_ERR_INVALID_ARG;
  ress::AttnLaunch a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.kv_idx = kv_idx;
  a.kv_cnt = kv_cnt;
  a.order = work_order;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.dev_err = dev_err;
  cudaError_t e = ress::launch_attn(d, a, (cudaStream_t)stream);
  if (e == cudaErrorNotSupported) return RESS_ERR_CUDA;
  return from_cuda(e);
}

ress_status ress_debug_attn_forced_timeout(const ress_shape *shape, const void *q, const void *k,
                                           const void *v, const int32_t *kv_idx,
                                           const int32_t *kv_cnt, float scale, void *out,
                                           int32_t *dev_err, int64_t limit_cycles,
                                           ress_stream_t stream) {
  if (limit_cycles <= 0 || limit_cycles > (int64_t)1 << 32) return RESS_ERR_INVALID_ARG;
  if (dev_err == nullptr || (reinterpret_cast<uintptr_t>(dev_err) & 3u)) return RESS_ERR_INVALID_ARG;
  Dims d;
  bool empty;
  ress_status st = check_shape(shape, &d, &empty);
  if (st != RESS_OK) return st;
  if (empty) return RESS_OK;
  if (!ptr_ok(q) || !ptr_ok(k) || !ptr_ok(v) || !ptr_ok(kv_idx) || !ptr_ok(kv_cnt) || !ptr_ok(out))
    return RESS_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale != scale) return RESS_ERR_INVALID_ARG;
  ress::AttnLaunch a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.kv_idx = kv_idx;
  a.kv_cnt = kv_cnt;
  a.order = nullptr;
  a.scale = scale;
  a.out = out;
  a.lse = nullptr;
  a.dev_err = dev_err;
  a.stall_cycles = (long long)limit_cycles;
  cudaError_t e = ress::launch_attn(d, a, (cudaStream_t)stream);
  if (e == cudaErrorNotSupported) return RESS_ERR_CUDA;
  return from_cuda(e);
}

// ------------------------------------------------------------------- token operators
ress_status ress_rope_init(ress_rope_plan *plan, int32_t head_dim, int32_t rot_dim, int32_t axes,
                           int32_t layout, double theta, int32_t scaling, double factor,
                           int32_t original_len, double beta_fast, double beta_slow) {
  if (plan == nullptr || !(theta > 1.0 && theta <= 1e12)) return RESS_ERR_INVALID_ARG;
  if (scaling < RESS_ROPE_PLAIN || scaling > RESS_ROPE_YARN) return RESS_ERR_INVALID_ARG;
  if (scaling != RESS_ROPE_PLAIN && !(factor >= 1.0 && factor <= 1e6)) return RESS_ERR_INVALID_ARG;
  if (scaling == RESS_ROPE_YARN &&
      (original_len < 1 || !(beta_slow > 0.0) || !(beta_slow < beta_fast) || std::isinf(beta_fast)))
    return RESS_ERR_INVALID_ARG;
  ress_rope_plan r = {};
  r.head_dim = head_dim;
  r.rot_dim = rot_dim;
  r.axes = axes;
  r.layout = layout;
  r.amplitude = scaling == RESS_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  if (!plan_ok(&r)) return RESS_ERR_INVALID_ARG;
  const int d = rot_dim / axes;
  if (scaling == RESS_ROPE_NTK && d <= 2) return RESS_ERR_INVALID_ARG;
  const long double pi2 = 6.28318530717958647692528676655900577L;
  long double base = theta;
  if (scaling == RESS_ROPE_NTK) base *= powl((long double)factor, (long double)d / (d - 2));
  // YaRN: pair index at which a pair turns `turns` times within the trained length
  auto pair_of = [&](double turns) {
    return d * std::log(original_len / (turns * (double)pi2)) / (2.0 * std::log(theta));
  };
  double low = 0.0, high = 0.0;
  if (scaling == RESS_ROPE_YARN) {
    low = std::max(std::floor(pair_of(beta_fast)), 0.0);
    high = std::min(std::ceil(pair_of(beta_slow)), d - 1.0);
  }
  for (int i = 0; i < d / 2; ++i) {
    long double f = powl(base, -2.0L * i / d);
    if (scaling == RESS_ROPE_LINEAR) f /= factor;
    if (scaling == RESS_ROPE_YARN) {
      const double ramp = std::min(std::max((i - low) / std::max(high - low, 0.001), 0.0), 1.0);
      f = f / factor * ramp + f * (1.0 - ramp);
    }
    // f <= 1 radian per position: a fraction of a turn below 0.16
    r.phase[i] = (uint64_t)roundl(f / pi2 * 18446744073709551616.0L);
  }
  *plan = r;
  return RESS_OK;
}

ress_status ress_rope(const ress_rope_plan *plan, int32_t batch, int32_t heads, int32_t tokens,
                      int32_t dtype, const ress_rows *x, const int32_t *positions,
                      int64_t pos_stride_b, int32_t inverse, const ress_rows *out,
                      ress_stream_t stream) {
  if (!plan_ok(plan) || batch < 0 || heads < 0 || tokens < 0) return RESS_ERR_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return RESS_ERR_INVALID_ARG;
  const size_t size = dtype_bytes(dtype);
  if (size == 0) return RESS_ERR_INVALID_ARG;
  if (heads > kMaxTokenHeads) return RESS_ERR_UNSUPPORTED;
  if (batch == 0 || heads == 0 || tokens == 0) return RESS_OK;
  if (!positions_ok(plan, positions, pos_stride_b)) return RESS_ERR_INVALID_ARG;
  if (!rows_ok(x, size) || !out_rows_ok(out, size, batch, heads, tokens, plan->head_dim))
    return RESS_ERR_INVALID_ARG;
  if (x->ptr == out->ptr && !same_rows(x, out, batch, heads, tokens)) return RESS_ERR_INVALID_ARG;
  ress::TokensLaunch a = {};
  a.parts = 1;
  a.batch = batch;
  a.tokens = tokens;
  a.head_dim = plan->head_dim;
  a.dtype = dtype;
  a.norm = RESS_NORM_NONE;
  a.rope = plan;
  a.inverse = inverse != 0;
  a.positions = positions;
  a.pos_stride_b = pos_stride_b;
  a.views = 1;
  a.part[0] = {x, out, heads, true, nullptr, nullptr};
  return from_cuda(ress::launch_tokens(a, (cudaStream_t)stream));
}

ress_status ress_qk_norm_rope(const ress_qk_params *params, const ress_rows *q,
                              const ress_rows *k, const ress_rows *v, const ress_rows *q_out,
                              const ress_rows *k_out, const ress_rows *v_out,
                              ress_stream_t stream) {
  if (params == nullptr) return RESS_ERR_INVALID_ARG;
  const ress_qk_params &p = *params;
  if (p.batch < 0 || p.tokens < 0 || p.q_heads < 1 || p.kv_heads < 1) return RESS_ERR_INVALID_ARG;
  if (p.head_dim < 2 || p.head_dim > RESS_MAX_TOKEN_DIM) return RESS_ERR_INVALID_ARG;
  const size_t size = dtype_bytes(p.dtype);
  if (size == 0) return RESS_ERR_INVALID_ARG;
  if (p.norm < RESS_NORM_NONE || p.norm > RESS_NORM_LAYER) return RESS_ERR_INVALID_ARG;
  if (!(p.eps >= 0.f) || std::isinf(p.eps)) return RESS_ERR_INVALID_ARG;
  for (const float *w : {p.q_weight, p.q_bias, p.k_weight, p.k_bias})
    if (!aligned_to(w, 4)) return RESS_ERR_INVALID_ARG;
  if (p.rope != nullptr && (!plan_ok(p.rope) || p.rope->head_dim != p.head_dim)) return RESS_ERR_INVALID_ARG;
  if (p.views < 1 || p.specials < 0 || p.tokens % p.views != 0 || p.specials > p.tokens / p.views)
    return RESS_ERR_INVALID_ARG;
  if ((v == nullptr) != (v_out == nullptr)) return RESS_ERR_INVALID_ARG;
  if (p.q_heads > kMaxTokenHeads || p.kv_heads > kMaxTokenHeads) return RESS_ERR_UNSUPPORTED;
  if (p.batch == 0 || p.tokens == 0) return RESS_OK;
  if (p.rope != nullptr && !positions_ok(p.rope, p.positions, p.pos_stride_b)) return RESS_ERR_INVALID_ARG;
  const bool moves = p.specials > 0 && p.specials < p.tokens / p.views;  // some token's place changes
  const ress_rows *in[3] = {q, k, v}, *out[3] = {q_out, k_out, v_out};
  const int heads[3] = {p.q_heads, p.kv_heads, p.kv_heads};
  const int parts = v != nullptr ? 3 : 2;
  for (int i = 0; i < parts; ++i) {
    if (!rows_ok(in[i], size) || !out_rows_ok(out[i], size, p.batch, heads[i], p.tokens, p.head_dim))
      return RESS_ERR_INVALID_ARG;
    for (int j = 0; j < parts; ++j) {
      if (in[j] == nullptr || in[j]->ptr != out[i]->ptr) continue;
      if (i != j || moves || !same_rows(in[i], out[i], p.batch, heads[i], p.tokens))
        return RESS_ERR_INVALID_ARG;
    }
    for (int j = 0; j < i; ++j)
      if (out[i]->ptr == out[j]->ptr) return RESS_ERR_INVALID_ARG;
  }
  ress::TokensLaunch a = {};
  a.parts = parts;
  a.batch = p.batch;
  a.tokens = p.tokens;
  a.head_dim = p.head_dim;
  a.dtype = p.dtype;
  a.norm = p.norm;
  a.eps = p.eps;
  a.rope = p.rope;
  a.positions = p.positions;
  a.pos_stride_b = p.pos_stride_b;
  a.views = p.views;
  a.specials = p.specials;
  a.part[0] = {q, q_out, heads[0], true, p.q_weight, p.q_bias};
  a.part[1] = {k, k_out, heads[1], true, p.k_weight, p.k_bias};
  a.part[2] = {v, v_out, heads[2], false, nullptr, nullptr};
  return from_cuda(ress::launch_tokens(a, (cudaStream_t)stream));
}

// ------------------------------------------------------- attention with changed scores
size_t ress_masked_attn_workspace_bytes(const ress_shape *shape, int32_t q_len) {
  Dims d;
  bool empty;
  if (check_shape(shape, &d, &empty) != RESS_OK || empty || q_len < 1) return 0;
  if (!queries_ok(d, q_len)) return 0;
  return ress::masked_attn_workspace_bytes(d, q_len);
}

ress_status ress_masked_attn(const ress_shape *shape, const ress_attn_mods *mods, const void *q,
                             const void *k, const void *v, const int32_t *kv_idx,
                             const int32_t *kv_cnt, const int32_t *work_order, float scale,
                             void *out, float *lse, void *workspace, size_t workspace_bytes,
                             int32_t *dev_err, ress_stream_t stream) {
  Dims d;
  bool empty;
  ress_status st = check_shape(shape, &d, &empty);
  if (st != RESS_OK) return st;
  ress_attn_mods m = {};
  m.q_len = d.N;
  if (mods != nullptr) m = *mods;
  if (m.q_len < 0 || !(m.softcap >= 0.f)) return RESS_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale <= 1e30f) || !(m.softcap <= 1e30f)) return RESS_ERR_INVALID_ARG;
  if (m.softcap > 0.f && !(scale / m.softcap >= 1e-20f && scale / m.softcap <= 1e20f)) return RESS_ERR_INVALID_ARG;
  if (d.N > 0 && m.q_len > 0 && d.B > 0) {  // (an array without elements may be NULL)
    if ((m.q_pos == nullptr) != (m.k_pos == nullptr) || (m.q_doc == nullptr) != (m.k_doc == nullptr) ||
        (m.q_order == nullptr) != (m.k_order == nullptr) || (kv_idx == nullptr) != (kv_cnt == nullptr))
      return RESS_ERR_INVALID_ARG;
    if (m.slopes != nullptr && m.q_pos == nullptr) return RESS_ERR_INVALID_ARG;
  }
  for (const void *x : {(const void *)m.slopes, (const void *)m.q_pos, (const void *)m.k_pos, (const void *)m.q_doc,
                        (const void *)m.k_doc, (const void *)m.q_order, (const void *)m.k_order, (const void *)lse,
                        (const void *)dev_err})
    if (!aligned_to(x, 4)) return RESS_ERR_INVALID_ARG;
  if (!queries_ok(d, m.q_len)) return RESS_ERR_UNSUPPORTED;
  if (d.B == 0 || m.q_len == 0) return RESS_OK;
  if (!ptr_ok(out)) return RESS_ERR_INVALID_ARG;
  if (d.N > 0) {
    const size_t need = ress::masked_attn_workspace_bytes(d, m.q_len);
    if (!ptr_ok(q) || !ptr_ok(k) || !ptr_ok(v) || !aligned16(workspace)) return RESS_ERR_INVALID_ARG;
    if (workspace_bytes < need || (need > 0 && workspace == nullptr)) return RESS_ERR_INVALID_ARG;
    if (!aligned16(kv_idx) || !aligned16(kv_cnt) || !aligned16(work_order)) return RESS_ERR_INVALID_ARG;
  }
  ress::MaskedAttnLaunch a;
  a.mods = m;
  a.q = q;
  a.k = k;
  a.v = v;
  a.kv_idx = kv_idx;
  a.kv_cnt = kv_cnt;
  a.order = work_order;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  a.dev_err = dev_err;
  return from_cuda(ress::launch_masked_attn(d, a, (cudaStream_t)stream));
}

}  // extern "C"

// ---------------------------------------------------------------------------------------
// ress_drift_scores_static: the drift score for callers that cannot allocate device
// memory.  Its scratch is this file's static device array; the host looks up the array's
// device address once per device (the array's name in host code is only a stand-in).
#include <mutex>

namespace {

constexpr size_t kDriftStaticBytes = (size_t)8 << 20;  // 8 MiB, see include/ress.h
static __device__ __align__(256) unsigned char g_drift_static_scratch[kDriftStaticBytes];

constexpr int kMaxDevices = 64;
void *g_drift_static_addr[kMaxDevices] = {};
std::mutex g_drift_static_mu;

// Device address of the static scratch on the current device; looked up on the first
// call per device, with that device current.
cudaError_t drift_static_address(void **out) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_drift_static_mu);
  if (g_drift_static_addr[dev] == nullptr) {
    void *p = nullptr;
    e = cudaGetSymbolAddress(&p, g_drift_static_scratch);
    if (e != cudaSuccess) return e;
    g_drift_static_addr[dev] = p;
  }
  *out = g_drift_static_addr[dev];
  return cudaSuccess;
}

}  // namespace

extern "C" ress_status ress_drift_scores_static(const ress_shape *shape, const float *P,
                                                const float *v_pool, const float *v_bar,
                                                const float *gram, float *s,
                                                ress_stream_t stream) {
  Dims d;
  bool empty;
  ress_status st = check_shape(shape, &d, &empty);
  if (st != RESS_OK) return st;
  if (empty) return RESS_OK;
  if (!ptr_ok(P) || !ptr_ok(v_pool) || !ptr_ok(v_bar) || !ptr_ok(gram) || !ptr_ok(s))
    return RESS_ERR_INVALID_ARG;
  if (ress::drift_workspace_bytes(d) > kDriftStaticBytes) return RESS_ERR_UNSUPPORTED;
  void *scratch = nullptr;
  if (drift_static_address(&scratch) != cudaSuccess) return RESS_ERR_CUDA;
  return from_cuda(ress::launch_drift(d, P, v_pool, v_bar, gram, s, scratch, (cudaStream_t)stream));
}
