// Token operators in front of the attention: rotary positions, and the per-head norm of
// queries and keys with the rotation in the same pass.
//
// Mathematics.  A row x is the D elements of one (token, head).  The norm is
//   RMS    y = x / sqrt(mean(x^2) + eps) * w + b
//   LAYER  y = (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps) * w + b
// and the rotation turns pair p of the row by the angle pos * f_p:
//   (a, b) -> amplitude * (a cos - b sin, b cos + a sin).
// Both are evaluated in fp32 from the stored type and rounded once, to the stored type, at
// the end; the two-pass form of the layer norm keeps rows with a large mean exact.
//
// Angles.  The plan holds f_p / (2 pi), the turns per position, as a 64-bit fraction F of
// a turn.  pos * F modulo 2^64 (one integer multiply) is the angle's fraction of a turn
// with an error of |pos| * 2^-65 turns, so that the range reduction is exact for far
// positions where an fp32 product pos * f_p has lost the fraction altogether.  The nearest
// quarter turn is taken off as an integer too, so that only an angle of at most pi / 4 is
// rounded to fp32 (an error of 2^-25 relative, against 2^-24 pi for a whole turn).
//
// What bounds it: HBM.  Every element is read and written once.  A warp takes one token:
// its angles are the same for every head, so they are computed once per token, by lanes
// in parallel, and stay in registers while the warp walks the token's heads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ress_common.cuh"
#include "ress_internal.h"

namespace ress {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxDim = 256;
constexpr int kMaxPairs = kMaxDim / 2;

template <typename T>
RESS_DEV float to_f32(T v);
template <>
RESS_DEV float to_f32(float v) { return v; }
template <>
RESS_DEV float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
RESS_DEV float to_f32(__half v) { return __half2float(v); }

template <typename T>
RESS_DEV T from_f32(float v);
template <>
RESS_DEV float from_f32(float v) { return v; }
template <>
RESS_DEV __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <>
RESS_DEV __half from_f32(float v) { return __float2half_rn(v); }

// One tensor of the call: `heads` rows per token, read from and written to strided views.
struct Part {
  const void *in;
  void *out;
  long long in_b, in_h, in_t, out_b, out_h, out_t;  // strides in elements
  int heads;
  int work;  // 1: norm and rotate, 0: move only
  const float *weight, *bias;
};

struct TokenParams {
  Part part[3];
  int parts;
  int B, N, D;
  int norm;  // ress_norm
  float eps;
  int rot, axes, layout;  // rot = 0: no rotation
  float amplitude, sign;
  const int32_t *positions;  // [B or 1][N][axes], or null: the token's index
  long long pos_b;
  int views, specials, view_tokens;  // view_tokens = 0: rows keep their places
  int groups;                        // warps that share a token's heads
  long long tasks;                   // B * N * groups
  uint64_t phase[kMaxPairs];         // turns per position of each pair of a section
};

// Row that token t goes to: patch tokens first, special tokens behind them.
RESS_DEV int target_row(const TokenParams &p, int t) {
  if (p.view_tokens == 0) return t;
  const int v = t / p.view_tokens, r = t - v * p.view_tokens;
  const int patch = p.view_tokens - p.specials;
  return r >= p.specials ? v * patch + r - p.specials : p.views * patch + v * p.specials + r;
}

// (amplitude cos, amplitude sin) of every pair of a token, in section order.
RESS_DEV void token_angles(const TokenParams &p, const uint64_t *phase, int b, int t, int lane,
                           float2 *cs) {
  const int pairs = p.rot >> 1, per = pairs / p.axes;
  for (int i = lane; i < pairs; i += 32) {
    const int a = i / per;
    const long long pos =
        p.positions ? (long long)__ldg(p.positions + b * p.pos_b + (long long)t * p.axes + a) : t;
    const uint64_t turn = (uint64_t)pos * phase[i - a * per];
    const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);
    const long long rest = (long long)(turn - ((uint64_t)quarter << 62));
    float s, c;
    sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);
    if (quarter & 1) {
      const float t = s;
      s = c;
      c = -t;
    }
    if (quarter & 2) {
      s = -s;
      c = -c;
    }
    cs[i] = make_float2(p.amplitude * c, p.sign * p.amplitude * s);
  }
}

RESS_DEV float row_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ------------------------------------------------------------------- 16-byte form
// A row is D * sizeof(T) / 16 lanes (a power of two up to 32), one 16-byte chunk each, so a
// warp holds several heads of a token at a time; a lane keeps the same chunk of the row for
// every head, and with it the same angles.  Pairs of the interleaved layout lie inside a
// chunk; pairs of the half layout lie in chunks half a section apart and meet by shuffle.
template <typename T>
__global__ void __launch_bounds__(kThreads) token_vec_kernel(const __grid_constant__ TokenParams p) {
  constexpr int V = 16 / sizeof(T);
  constexpr int U = 4;  // loads in flight per lane
  __shared__ uint64_t phase[kMaxPairs];
  __shared__ __align__(16) float wb[4][kMaxDim];
  __shared__ float2 cs_all[kWarps][kMaxPairs];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pairs = p.rot >> 1;
  if (pairs > 0)
    for (int i = tid; i < pairs / p.axes; i += kThreads) phase[i] = p.phase[i];
  for (int i = tid; i < p.D; i += kThreads) {
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      wb[2 * a][i] = p.part[a].weight ? p.part[a].weight[i] : 1.f;
      wb[2 * a + 1][i] = p.part[a].bias ? p.part[a].bias[i] : 0.f;
    }
  }
  __syncthreads();
  const int lpr = p.D / V, rpw = 32 / lpr;  // lanes per row, rows per warp
  const int sub = lane / lpr, chunk = lane - sub * lpr;
  float2 *cs = cs_all[warp];
  // iterations of each part: rpw heads at a time
  const int it1 = (p.part[0].heads + rpw - 1) / rpw;
  const int it2 = it1 + (p.parts > 1 ? (p.part[1].heads + rpw - 1) / rpw : 0);
  const int its = it2 + (p.parts > 2 ? (p.part[2].heads + rpw - 1) / rpw : 0);
  // this lane's pairs: shuffle partner and first pair (half layout)
  const bool half = p.layout == RESS_ROPE_HALF;
  int partner = lane, pair0 = chunk * V / 2;
  bool second = false, turned = chunk * V < p.rot;
  if (half && turned) {
    const int hl = p.rot / p.axes / (2 * V);  // chunks in half a section
    const int sec = chunk / (2 * hl), at = chunk - sec * 2 * hl;
    second = at >= hl;
    partner = second ? lane - hl : lane + hl;
    pair0 = (sec * hl + (second ? at - hl : at)) * V;
  }
  const long long stride = (long long)gridDim.x * kWarps;
  for (long long task = (long long)blockIdx.x * kWarps + warp; task < p.tasks; task += stride) {
    const long long token = task / p.groups;
    const int group = (int)(task - token * p.groups);
    const int b = (int)(token / p.N), t = (int)(token - (long long)b * p.N);
    const int t_out = target_row(p, t);
    float c[V], s[V];
    if (pairs > 0) {
      __syncwarp();
      token_angles(p, phase, b, t, lane, cs);
      __syncwarp();
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int at = half ? pair0 + e : pair0 + (e >> 1);
        const float2 v = turned && at < pairs ? cs[at] : make_float2(1.f, 0.f);
        c[e] = v.x;
        s[e] = v.y;
      }
    }
    const int i0 = (int)((long long)its * group / p.groups);
    const int i1 = (int)((long long)its * (group + 1) / p.groups);
    for (int i = i0; i < i1; i += U) {
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = i + u;
        if (k < i1) {
          const int which = k < it1 ? 0 : (k < it2 ? 1 : 2);
          const Part &q = p.part[which];
          const int h = (k - (which == 0 ? 0 : (which == 1 ? it1 : it2))) * rpw + sub;
          raw[u] = make_uint4(0, 0, 0, 0);
          if (h < q.heads)
            raw[u] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(q.in) + b * q.in_b +
                                                      h * q.in_h + t * q.in_t + chunk * V);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = i + u;
        if (k >= i1) break;
        const int which = k < it1 ? 0 : (k < it2 ? 1 : 2);
        const Part &q = p.part[which];
        const int h = (k - (which == 0 ? 0 : (which == 1 ? it1 : it2))) * rpw + sub;
        if (q.work) {
          T *e_ = reinterpret_cast<T *>(&raw[u]);
          float x[V];
#pragma unroll
          for (int e = 0; e < V; ++e) x[e] = to_f32<T>(e_[e]);
          if (p.norm != RESS_NORM_NONE) {
            float mean = 0.f;
            if (p.norm == RESS_NORM_LAYER) {
              float m = 0.f;
#pragma unroll
              for (int e = 0; e < V; ++e) m += x[e];
              mean = row_sum(m, lpr) / p.D;
            }
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) {
              x[e] -= mean;
              ss += x[e] * x[e];
            }
            const float r = rsqrtf(row_sum(ss, lpr) / p.D + p.eps);
            const float *w = wb[2 * which] + chunk * V, *bb = wb[2 * which + 1] + chunk * V;
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] = x[e] * r * w[e] + bb[e];
          }
          if (pairs > 0) {
            if (half) {
#pragma unroll
              for (int e = 0; e < V; ++e) {
                const float y = __shfl_sync(0xffffffffu, x[e], partner);
                if (turned) x[e] = second ? x[e] * c[e] + y * s[e] : x[e] * c[e] - y * s[e];
              }
            } else {
#pragma unroll
              for (int e = 0; e < V; e += 2) {
                if (chunk * V + e < p.rot) {
                  const float a = x[e], d = x[e + 1];
                  x[e] = a * c[e] - d * s[e];
                  x[e + 1] = d * c[e] + a * s[e];
                }
              }
            }
          }
#pragma unroll
          for (int e = 0; e < V; ++e) e_[e] = from_f32<T>(x[e]);
        }
        if (h < q.heads)
          *reinterpret_cast<uint4 *>(static_cast<T *>(q.out) + b * q.out_b + h * q.out_h +
                                     t_out * q.out_t + chunk * V) = raw[u];
      }
    }
  }
}

// ------------------------------------------------------------------- element form
// Any head size up to 256, any strides, any even split of the rotated part: a warp takes
// the rows of a token one after another, elements spread over its lanes.
template <typename T>
__global__ void __launch_bounds__(kThreads) token_elem_kernel(const __grid_constant__ TokenParams p) {
  constexpr int R = kMaxDim / 32;
  __shared__ uint64_t phase[kMaxPairs];
  __shared__ float2 cs_all[kWarps][kMaxPairs];
  __shared__ float row_all[kWarps][kMaxDim];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pairs = p.rot >> 1;
  if (pairs > 0)
    for (int i = tid; i < pairs / p.axes; i += kThreads) phase[i] = p.phase[i];
  __syncthreads();
  float2 *cs = cs_all[warp];
  float *row = row_all[warp];
  const int rows = p.part[0].heads + (p.parts > 1 ? p.part[1].heads : 0) + (p.parts > 2 ? p.part[2].heads : 0);
  const int sec = p.rot > 0 ? p.rot / p.axes : 1;
  const long long stride = (long long)gridDim.x * kWarps;
  for (long long task = (long long)blockIdx.x * kWarps + warp; task < p.tasks; task += stride) {
    const long long token = task / p.groups;
    const int group = (int)(task - token * p.groups);
    const int b = (int)(token / p.N), t = (int)(token - (long long)b * p.N);
    const int t_out = target_row(p, t);
    __syncwarp();
    if (pairs > 0) token_angles(p, phase, b, t, lane, cs);
    const int r0 = (int)((long long)rows * group / p.groups);
    const int r1 = (int)((long long)rows * (group + 1) / p.groups);
    for (int r = r0; r < r1; ++r) {
      int which = 0, h = r;
      while (h >= p.part[which].heads) h -= p.part[which++].heads;
      const Part &q = p.part[which];
      const T *src = static_cast<const T *>(q.in) + b * q.in_b + h * q.in_h + t * q.in_t;
      T *dst = static_cast<T *>(q.out) + b * q.out_b + h * q.out_h + t_out * q.out_t;
      if (!q.work) {
        T v[R];
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (lane + 32 * i < p.D) v[i] = src[lane + 32 * i];
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (lane + 32 * i < p.D) dst[lane + 32 * i] = v[i];
        continue;
      }
      float x[R];
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        x[i] = lane + 32 * i < p.D ? to_f32<T>(src[lane + 32 * i]) : 0.f;
        sum += x[i];
      }
      if (p.norm != RESS_NORM_NONE) {
        const float mean = p.norm == RESS_NORM_LAYER ? row_sum(sum, 32) / p.D : 0.f;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (lane + 32 * i < p.D) {
            x[i] -= mean;
            ss += x[i] * x[i];
          }
        const float rs = rsqrtf(row_sum(ss, 32) / p.D + p.eps);
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (lane + 32 * i < p.D)
            x[i] = x[i] * rs * (q.weight ? __ldg(q.weight + lane + 32 * i) : 1.f) +
                   (q.bias ? __ldg(q.bias + lane + 32 * i) : 0.f);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (lane + 32 * i < p.rot) row[lane + 32 * i] = x[i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int e = lane + 32 * i;
        if (e >= p.D) continue;
        float y = x[i];
        if (e < p.rot) {
          const int a = e / sec, at = e - a * sec;
          int other, pair;
          bool second;
          if (p.layout == RESS_ROPE_HALF) {
            second = at >= sec / 2;
            other = second ? e - sec / 2 : e + sec / 2;
            pair = a * (sec / 2) + (second ? at - sec / 2 : at);
          } else {
            second = at & 1;
            other = e ^ 1;
            pair = e >> 1;
          }
          const float2 v = cs[pair];
          y = second ? y * v.x + row[other] * v.y : y * v.x - row[other] * v.y;
        }
        dst[e] = from_f32<T>(y);
      }
    }
  }
}

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

template <typename T>
cudaError_t launch_typed(TokenParams &p, int sms, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  // the 16-byte form: chunks fill a power-of-two share of a warp, every row starts on a
  // 16-byte boundary, and the pairs of the half layout lie whole chunks apart
  const int lpr = p.D / V;
  bool vec = p.D % V == 0 && lpr <= 32 && (lpr & (lpr - 1)) == 0;
  if (p.rot > 0 && p.layout == RESS_ROPE_HALF) vec = vec && (p.rot / p.axes) % (2 * V) == 0;
  int rows = 0;
  for (int i = 0; i < p.parts; ++i) {
    const Part &q = p.part[i];
    vec = vec && aligned(q.in, 16) && aligned(q.out, 16);
    for (long long s : {q.in_b, q.in_h, q.in_t, q.out_b, q.out_h, q.out_t}) vec = vec && s % V == 0;
    rows += vec ? (q.heads + 32 / lpr - 1) / (32 / lpr) : q.heads;
  }
  if (!vec) {
    rows = 0;
    for (int i = 0; i < p.parts; ++i) rows += p.part[i].heads;
  }
  const long long tokens = (long long)p.B * p.N;
  // few tokens: spread a token's heads over warps until the card has some for every
  // scheduler; each then computes the token's angles again
  const long long want = (long long)sms * 16;
  p.groups = (int)(tokens >= want ? 1 : (want + tokens - 1) / tokens);
  if (p.groups > rows) p.groups = rows;
  p.tasks = tokens * p.groups;
  long long ctas = (p.tasks + kWarps - 1) / kWarps;
  if (ctas > (long long)sms * 8) ctas = (long long)sms * 8;
  if (vec)
    token_vec_kernel<T><<<(unsigned)ctas, kThreads, 0, st>>>(p);
  else
    token_elem_kernel<T><<<(unsigned)ctas, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tokens(const TokensLaunch &a, cudaStream_t st) {
  TokenParams p = {};
  p.parts = a.parts;
  for (int i = 0; i < a.parts; ++i) {
    const TokensPart &s = a.part[i];
    Part &q = p.part[i];
    q.in = s.in->ptr;
    q.out = s.out->ptr;
    q.in_b = s.in->stride_b;
    q.in_h = s.in->stride_h;
    q.in_t = s.in->stride_t;
    q.out_b = s.out->stride_b;
    q.out_h = s.out->stride_h;
    q.out_t = s.out->stride_t;
    q.heads = s.heads;
    q.work = s.work;
    q.weight = s.weight;
    q.bias = s.bias;
  }
  p.B = a.batch;
  p.N = a.tokens;
  p.D = a.head_dim;
  p.norm = a.norm;
  p.eps = a.eps;
  p.sign = a.inverse ? -1.f : 1.f;
  if (a.rope != nullptr) {
    p.rot = a.rope->rot_dim;
    p.axes = a.rope->axes;
    p.layout = a.rope->layout;
    p.amplitude = a.rope->amplitude;
    for (int i = 0; i < p.rot / 2 / p.axes; ++i) p.phase[i] = a.rope->phase[i];
  } else {
    p.axes = 1;
  }
  p.positions = a.positions;
  p.pos_b = a.pos_stride_b;
  p.views = a.views;
  p.specials = a.specials;
  p.view_tokens = a.specials > 0 && a.specials < a.tokens / a.views ? a.tokens / a.views : 0;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  switch (a.dtype) {
    case RESS_BF16: return launch_typed<__nv_bfloat16>(p, sms, st);
    case RESS_FP16: return launch_typed<__half>(p, sms, st);
    default: return launch_typed<float>(p, sms, st);
  }
}

}  // namespace ress
