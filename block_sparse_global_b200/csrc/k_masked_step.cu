// Attention with changed scores for few query rows over a cache, one new token above all (see
// k_masked_attn.cu for the mathematics): one row at a time on the FMA pipes, since a
// tensor-core tile of 128 rows would hold one.
//
// What bounds it: HBM for one token.  Every visible key and value is read once, 256 bytes for
// 128 FMAs; hidden ones are never read.  A cluster of up to eight CTAs shares a row: its
// warps take 16 keys in turn (eight lanes hold a key, 16 bytes each, so a lane group has four
// keys and their values in registers, and the next keys load while the weights of these are
// computed), keep an online softmax per lane group in fp32, and join over lanes, warps and,
// through distributed shared memory, the cluster.  One launch, no workspace.
//
// Measured, one token over 10992, in a CUDA graph: 16 heads (45 MB) 14.4 us, 128 heads (360 MB)
// 59 us = 6.1 TB/s.  About 6 us of each are launch and joins.  Two CTAs of 384 threads an SM: a
// cluster of eight CTAs that fill an SM each does not fit every GPC beside the others (512
// threads, one an SM: 18 us); a ring of asynchronous copies in shared memory was slower (19 us).
#include <cooperative_groups.h>

#include <algorithm>

#include "k_attn.cuh"
#include "k_masked.cuh"

namespace ress {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 4;  // keys of a lane group in flight

struct StepParams {
  const __nv_bfloat16 *q, *k, *v;
  const int32_t *kv_idx, *kv_cnt;
  const int32_t *q_pos, *k_pos, *q_doc, *k_doc, *q_order, *k_order;
  const float *slopes;
  __nv_bfloat16 *out;
  float *lse;
  int32_t *dev_err;
  int H, N, Nq, nq, nk, kb_log2, parts;
  float scale_log2, cap_log2, cap_in;  // cap_in = 0: no cap
};

// Eight bf16 values as four pairs of fp32.
RESS_DEV void unpack8(const uint4 &raw, uint64_t (&x)[4]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = ((uint64_t)(w[i] & 0xffff0000u) << 32) | (w[i] << 16);
}

__global__ void __launch_bounds__(kThreads, 2) step_kernel(const __grid_constant__ StepParams p) {
  __shared__ float2 warp_ml[kWarps];
  __shared__ float warp_o[kWarps][64];
  __shared__ float2 part_ml;
  __shared__ float part_o[64];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / (unsigned)p.parts, part = blockIdx.x - row * p.parts;
  const int bh = row / p.Nq, t = row - bh * p.Nq, b = bh / p.H;
  const long long item = (long long)bh * p.nq + (t >> 7);
  const int cnt = p.kv_cnt ? p.kv_cnt[item] : p.nk;
  const int32_t *list = p.kv_idx ? p.kv_idx + item * p.nk : nullptr;
  bool bad = cnt < 0 || cnt > p.nk;
  if (list && !bad)
    for (int j = tid; j < cnt; j += kThreads) bad |= list[j] < 0 || list[j] >= p.nk;
  if (list) bad = __syncthreads_or(bad);  // the same for every CTA of the row
  if (bad && tid == 0 && part == 0) report_error(p.dev_err, RESS_ERR_DEVICE_BOUNDS);

  const int group = lane >> 3, own = lane & 7;  // key of a load, elements 8 own ..
  uint64_t q[4];
  unpack8(*reinterpret_cast<const uint4 *>(p.q + ((long long)bh * p.Nq + t) * 64 + 8 * own), q);
  const int doc = p.q_doc ? p.q_doc[(long long)b * p.Nq + t] : 0;
  const int order = p.q_order ? p.q_order[(long long)b * p.Nq + t] : 0;
  const int pos = p.slopes ? p.q_pos[(long long)b * p.Nq + t] : 0;
  const float slope = p.slopes ? -p.slopes[bh - b * p.H] * kLog2e : 0.f;
  float m = kNoMax, l = 0.f;
  uint64_t o[4] = {};
  const __nv_bfloat16 *kp = p.k + (long long)bh * p.N * 64 + 8 * own;
  const __nv_bfloat16 *vp = p.v + (long long)bh * p.N * 64 + 8 * own;
  const long long tokens = (long long)b * p.N;
  const int units = bad || doc < 0 ? 0 : cnt << (p.kb_log2 - 4);  // of 16 keys
  const int step = p.parts * kWarps;
  // this lane group's first key of unit i, and which of its keys the query sees
  auto first_key = [&](int i) {
    const int entry = i >> (p.kb_log2 - 4), in_block = (i << 4) & ((1 << p.kb_log2) - 1);
    return ((list ? list[entry] : entry) << p.kb_log2) + in_block + group;
  };
  auto seen = [&](int u0) {
    uint32_t bits = 0;
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      const int u = u0 + 4 * j;
      bool vis = u < p.N;
      if (vis && p.q_doc) vis = p.k_doc[tokens + u] == doc;
      if (vis && p.q_order) vis = p.k_order[tokens + u] <= order;
      bits |= (uint32_t)vis << j;
    }
    return bits;
  };
  uint4 kr[kKeys], vr[kKeys];
  auto load = [&](uint4 (&raw)[kKeys], const __nv_bfloat16 *src, int u0, uint32_t vis) {
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      raw[j] = make_uint4(0, 0, 0, 0);
      if (vis >> j & 1) raw[j] = *reinterpret_cast<const uint4 *>(src + (long long)(u0 + 4 * j) * 64);
    }
  };
  int i = part * kWarps + warp, u0 = 0;
  uint32_t vis = 0;
  if (i < units) {
    u0 = first_key(i);
    vis = seen(u0);
    load(kr, kp, u0, vis);
    load(vr, vp, u0, vis);
  }
  for (; i < units; i += step) {
    float s[kKeys];
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      uint64_t x[4];
      unpack8(kr[j], x);
      uint64_t a = fmul2(q[0], x[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) a = ffma2(q[e], x[e], a);
      s[j] = f2lo(a) + f2hi(a);
    }
    // the next unit's keys load while this one's weights are computed
    const int u_now = u0;
    const uint32_t now = vis;
    if (i + step < units) {
      u0 = first_key(i + step);
      vis = seen(u0);
      load(kr, kp, u0, vis);
    }
    // sums of eight lanes, four keys at once: lane `own` ends with the sum of key own & 3
    static_assert(kKeys == 4, "the exchange below");
    const bool hi1 = own & 1, hi2 = own & 2;
    const float a0 = (hi1 ? s[1] : s[0]) + __shfl_xor_sync(0xffffffffu, hi1 ? s[0] : s[1], 1);
    const float a1 = (hi1 ? s[3] : s[2]) + __shfl_xor_sync(0xffffffffu, hi1 ? s[2] : s[3], 1);
    float z = (hi2 ? a1 : a0) + __shfl_xor_sync(0xffffffffu, hi2 ? a0 : a1, 2);
    z += __shfl_xor_sync(0xffffffffu, z, 4);
    const int key = own & 3;
    const bool mine = now >> key & 1;
    z = p.cap_in > 0.f ? p.cap_log2 * tanh_any(z * p.cap_in) : z * p.scale_log2;
    if (p.slopes && mine) {
      const float far = fabsf((float)((long long)pos - p.k_pos[tokens + u_now + 4 * key]));
      z = fmaf(slope, far, z);
    }
    float top = mine ? fmaxf(m, z) : m;
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float alpha = ex2_approx(m - top), w_own = mine ? ex2_approx(z - top) : 0.f;
    m = top;
    l *= alpha;
    const uint64_t al2 = f2(alpha, alpha);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = fmul2(o[e], al2);
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      const float w = __shfl_sync(0xffffffffu, w_own, (lane & 24) + j);
      if (!(now >> j & 1)) continue;
      uint64_t x[4];
      unpack8(vr[j], x);
      l += w;
      const uint64_t w2 = f2(w, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = ffma2(w2, x[e], o[e]);
    }
    if (i + step < units) load(vr, vp, u0, vis);
  }
  // the four lane groups, then the warps, then the cluster
#pragma unroll
  for (int d = 8; d < 32; d <<= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, d), l2 = __shfl_xor_sync(0xffffffffu, l, d);
    const float top = fmaxf(m, m2), a = ex2_approx(m - top), a2 = ex2_approx(m2 - top);
    l = l * a + l2 * a2;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lo = __shfl_xor_sync(0xffffffffu, f2lo(o[e]), d), hi = __shfl_xor_sync(0xffffffffu, f2hi(o[e]), d);
      o[e] = ffma2(f2(lo, hi), f2(a2, a2), fmul2(o[e], f2(a, a)));
    }
    m = top;
  }
  if (lane == 0) warp_ml[warp] = make_float2(m, l);
  if (group == 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<float2 *>(&warp_o[warp][8 * own + 2 * e]) = make_float2(f2lo(o[e]), f2hi(o[e]));
  }
  __syncthreads();
  if (tid < 64) {
    float top = kNoMax;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, warp_ml[w].x);
    float ls = 0.f, os = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float a = ex2_approx(warp_ml[w].x - top);
      ls += a * warp_ml[w].y;
      os += a * warp_o[w][tid];
    }
    part_o[tid] = os;
    if (tid == 0) part_ml = make_float2(top, ls);
  }
  cluster.sync();
  if (part == 0 && tid < 64 && !bad) {
    float top = kNoMax;
    for (int r = 0; r < p.parts; ++r) top = fmaxf(top, cluster.map_shared_rank(&part_ml, r)->x);
    float ls = 0.f, os = 0.f;
    for (int r = 0; r < p.parts; ++r) {
      const float2 ml = *cluster.map_shared_rank(&part_ml, r);
      const float a = ex2_approx(ml.x - top);
      ls += a * ml.y;
      os += a * *cluster.map_shared_rank(&part_o[tid], r);
    }
    const long long at = (long long)bh * p.Nq + t;
    p.out[at * 64 + tid] = __float2bfloat16_rn(ls == 0.f ? 0.f : os / ls);
    if (p.lse && tid == 0) p.lse[at] = ls == 0.f ? -INFINITY : (top + __log2f(ls)) * kLn2;
  }
  cluster.sync();  // nobody leaves while its sums are read
}

constexpr int kSlots = 2 * 148;  // resident CTAs

// CTAs of a row's cluster: enough for the card, each with at least 512 keys.
int step_parts(long long rows, int N) {
  int parts = 1;
  while (parts < 8 && rows * parts < 256 && N >= 512 * parts) parts *= 2;
  return parts;
}

}  // namespace

// Which form takes a call.  Measured: this one takes 6 us and about 8.1 ns for every key that
// a resident CTA walks; the tensor-core form 16 us and what the keys and values of all heads
// take at 6 TB/s, whatever the queries of a block.  (16 heads, in a CUDA graph, this form
// against the other: one token over 10992 keys 14 against 19 us, over 43968 46 against 41; 2
// tokens over 10992 15 against 19, 3 tokens 25 against 18; 16 tokens over 1000 keys 12 and 12,
// back to back from the host 13 against 18; 128 heads, one token over 10992 59 against 76.)
bool masked_step_fits(const Dims &d, int q_len) {
  const long long rows = d.BH() * q_len;
  const int parts = step_parts(rows, d.N);
  const long long walked = (rows * parts + kSlots - 1) / kSlots * ((d.N + parts - 1) / parts);
  return walked * 81 <= 100000 + d.BH() * d.N * 256 / 600;  // in 0.1 ns
}

cudaError_t launch_masked_step(const Dims &d, const MaskedAttnLaunch &a, cudaStream_t st) {
  const ress_attn_mods &m = a.mods;
  StepParams p = {};
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.k = static_cast<const __nv_bfloat16 *>(a.k);
  p.v = static_cast<const __nv_bfloat16 *>(a.v);
  p.kv_idx = a.kv_idx;
  p.kv_cnt = a.kv_cnt;
  if (m.slopes) {
    p.slopes = m.slopes;
    p.q_pos = m.q_pos;
    p.k_pos = m.k_pos;
  }
  p.q_doc = m.q_doc;
  p.k_doc = m.k_doc;
  p.q_order = m.q_order;
  p.k_order = m.k_order;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.lse = a.lse;
  p.dev_err = a.dev_err;
  p.H = d.H;
  p.N = d.N;
  p.Nq = m.q_len;
  p.nq = (m.q_len + 127) / 128;
  p.nk = d.nk;
  p.kb_log2 = d.kb == 64 ? 6 : 7;
  const long long rows = d.BH() * m.q_len;
  p.parts = step_parts(rows, d.N);
  p.scale_log2 = a.scale * kLog2e;
  p.cap_log2 = m.softcap * kLog2e;
  p.cap_in = m.softcap > 0.f ? a.scale / m.softcap : 0.f;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)p.parts;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * p.parts));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, step_kernel, p);
}

}  // namespace ress
