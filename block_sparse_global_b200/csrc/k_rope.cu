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
// What bounds it: HBM.  Every element is read and written once.  The angles of a token are
// the same for every head, so a CTA takes some tokens with all their heads, computes their
// angles once into shared memory, and its warps then walk (heads, token) pieces.
//
// Measured on one B200 (in a CUDA graph): rotation of 16 heads x 137400 tokens x 64, fp16
// (563 MB) 111 us = 5.1 TB/s; layer norm, two-axis rotation and values of 3 x 16 heads x
// 137400 tokens, bf16 (1.69 GB) 338 us = 5.0 TB/s, of 10992 tokens (135 MB) 33 us.
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
  int groups;                        // element form: warps that share a token's heads
  long long tasks;                   // element form: B * N * groups
  int tile, tiles;                   // chunk form: tokens of a CTA, CTAs of a batch entry
  uint64_t phase[kMaxPairs];         // turns per position of each pair of a section
};

// Row that token t goes to: patch tokens first, special tokens behind them.
RESS_DEV int target_row(const TokenParams &p, int t) {
  if (p.view_tokens == 0) return t;
  const int v = t / p.view_tokens, r = t - v * p.view_tokens;
  const int patch = p.view_tokens - p.specials;
  return r >= p.specials ? v * patch + r - p.specials : p.views * patch + v * p.specials + r;
}

// (amplitude cos, amplitude sin) of pair i of a token, in section order.
RESS_DEV float2 pair_angle(const TokenParams &p, uint64_t phase, int b, int t, int axis) {
  const long long pos =
      p.positions ? (long long)__ldg(p.positions + b * p.pos_b + (long long)t * p.axes + axis) : t;
  const uint64_t turn = (uint64_t)pos * phase;
  const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);
  const long long rest = (long long)(turn - ((uint64_t)quarter << 62));
  float s, c;
  sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);
  if (quarter & 1) {
    const float x = s;
    s = c;
    c = -x;
  }
  if (quarter & 2) {
    s = -s;
    c = -c;
  }
  return make_float2(p.amplitude * c, p.sign * p.amplitude * s);
}

// The angles of a token, by the lanes of a warp.
RESS_DEV void token_angles(const TokenParams &p, const uint64_t *phase, int b, int t, int lane,
                           float2 *cs) {
  const int pairs = p.rot >> 1, per = pairs / p.axes;
  for (int i = lane; i < pairs; i += 32) {
    const int a = i / per;
    cs[i] = pair_angle(p, phase[i - a * per], b, t, a);
  }
}

RESS_DEV float row_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ------------------------------------------------------------------- chunk form
// A lane holds two chunks of V elements of a row, so that a rotated pair never leaves the
// lane: chunks half a section apart in the half layout, neighbours in the interleaved one.
// Chunks are of 16 bytes, or of 8 or 4 where sections, strides or addresses allow no more
// (half a section of 20 elements: 8 bytes of a 16-bit type).  A row takes D / 2V lanes, rounded up to a power of two (the rest idle), and a warp's pass several
// heads of one token.  The passes of all tensors and the CTA's tokens form one list, pass by
// pass, of which each warp takes an equal stretch: a few runs of tokens of one pass, in which
// pointers advance, weights and biases stay in registers and kPieces tokens' loads are in
// flight.
// Both sums of the layer norm are over centred values, in fp32.
constexpr int kAngleFloats = 4096;  // (cos, sin) of the CTA's tokens: 16 KB
// CTAs of an SM: the norm needs 128 registers; the rotation alone lives with 80 and gains from
// more loads in flight (100 views: 110 us with three CTAs, 133 us with two).
constexpr int kCtasRotate = 3, kCtasNorm = 2;
constexpr int kMaxTile = 32;        // tokens of a CTA
constexpr int kPieces = 2;          // pieces worked on, and as many in flight behind them

RESS_DEV uint64_t pk2(float lo, float hi) {
  return ((uint64_t)__float_as_uint(hi) << 32) | __float_as_uint(lo);
}
RESS_DEV float lo2(uint64_t v) { return __uint_as_float((uint32_t)v); }
RESS_DEV float hi2(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
RESS_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
RESS_DEV uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
RESS_DEV uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A chunk of V elements as it lies in memory, as V / 2 pairs of fp32, and back with one
// rounding.
template <typename T, int V>
struct alignas(V * sizeof(T)) Chunk {
  uint32_t w[V * sizeof(T) / 4];
};
template <int V>
RESS_DEV void unpack(const Chunk<float, V> &raw, uint64_t *x) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) x[i] = ((uint64_t)raw.w[2 * i + 1] << 32) | raw.w[2 * i];
}
template <int V>
RESS_DEV void unpack(const Chunk<__nv_bfloat16, V> &raw, uint64_t *x) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) x[i] = ((uint64_t)(raw.w[i] & 0xffff0000u) << 32) | (raw.w[i] << 16);
}
template <int V>
RESS_DEV void unpack(const Chunk<__half, V> &raw, uint64_t *x) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&raw.w[i]));
    x[i] = pk2(v.x, v.y);
  }
}
template <int V>
RESS_DEV void repack(const uint64_t *x, Chunk<float, V> &raw) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    raw.w[2 * i] = (uint32_t)x[i];
    raw.w[2 * i + 1] = (uint32_t)(x[i] >> 32);
  }
}
template <int V>
RESS_DEV void repack(const uint64_t *x, Chunk<__nv_bfloat16, V> &raw) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) raw.w[i] = pack_bf16x2(lo2(x[i]), hi2(x[i]));
}
template <int V>
RESS_DEV void repack(const uint64_t *x, Chunk<__half, V> &raw) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const __half2 h = __floats2half2_rn(lo2(x[i]), hi2(x[i]));
    raw.w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
}

// HALF: the pair layout; NORM: ress_norm, or kAnyNorm (the narrow chunks: fewer kernels).
constexpr int kAnyNorm = -1;
template <typename T, int V, bool HALF, int NORM>
__global__ void __launch_bounds__(kThreads, NORM == RESS_NORM_NONE ? kCtasRotate : kCtasNorm)
    token_chunk_kernel(const __grid_constant__ TokenParams p) {
  using Raw = Chunk<T, V>;
  const int norm = NORM == kAnyNorm ? p.norm : NORM;
  __shared__ __align__(16) float cs[kAngleFloats];
  __shared__ __align__(16) float wb[4][kMaxDim];
  __shared__ int to[kMaxTile];  // rows that the tokens go to
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / p.tiles, t0 = (blockIdx.x - b * p.tiles) * p.tile;
  const int nt = min(p.tile, p.N - t0);
  const int pairs = p.rot >> 1, slots = p.D >> 1;  // cos, then sin, of `slots` pairs a token
  const int used = p.D / (2 * V);  // lanes of a row that hold something
  int lpr = 1;
  while (lpr < used) lpr <<= 1;
  const int rpw = 32 / lpr, sub = lane / lpr, own = lane & (lpr - 1);
  const bool holds = own < used;
  // this lane's chunks: a is element ca of the row, b element cb
  int ca = 2 * own * V, cb = ca + V;
  bool turned = pairs > 0 && own * V < pairs;  // (interleaved: up to pair `pairs`)
  if (HALF && turned) {
    const int hl = p.rot / p.axes / (2 * V);  // chunks of half a section
    const int sec = own / hl;
    ca = (sec * 2 * hl + own - sec * hl) * V;
    cb = ca + hl * V;
  }
  const int it1 = (p.part[0].heads + rpw - 1) / rpw;
  const int it2 = it1 + (p.parts > 1 ? (p.part[1].heads + rpw - 1) / rpw : 0);
  const int its = it2 + (p.parts > 2 ? (p.part[2].heads + rpw - 1) / rpw : 0);
  const float inv_d = 1.0f / p.D;
  const int i0 = its * nt * warp / kWarps, i1 = its * nt * (warp + 1) / kWarps;
  // the run of pieces that is being worked on
  int which = 0, ta = 0, tb = 0;
  bool there = false;
  const T *src = nullptr;
  T *dst = nullptr;
  Raw next[kPieces][2];
  auto load = [&](int t) {
    const long long in_t = p.part[which].in_t;
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      next[u][0] = next[u][1] = Raw{};
      if (there && t + u < tb) {
        next[u][0] = *reinterpret_cast<const Raw *>(src + ca);
        next[u][1] = *reinterpret_cast<const Raw *>(src + cb);
      }
      src += in_t;
    }
  };
  auto open = [&](int i) {
    const int pass = i / nt;
    ta = i - pass * nt;
    tb = min(nt, ta + i1 - i);
    which = pass < it1 ? 0 : (pass < it2 ? 1 : 2);
    const Part &q = p.part[which];
    const int h = (pass - (which == 0 ? 0 : (which == 1 ? it1 : it2))) * rpw + sub;
    there = holds && h < q.heads;
    src = static_cast<const T *>(q.in) + b * q.in_b + h * q.in_h + (t0 + ta) * q.in_t;
    dst = static_cast<T *>(q.out) + b * q.out_b + h * q.out_h;
    load(ta);
  };
  if (i0 < i1) open(i0);  // its loads are under way while the angles are computed
  if (pairs > 0) {
    const int per = pairs / p.axes;
    for (int i = tid; i < nt * pairs; i += kThreads) {
      const int t = i / pairs, k = i - t * pairs, a = k / per;
      const float2 v = pair_angle(p, p.phase[k - a * per], b, t0 + t, a);
      cs[2 * slots * t + k] = v.x;
      cs[2 * slots * t + slots + k] = v.y;
    }
  }
  if (tid < nt) to[tid] = target_row(p, t0 + tid);
  if (norm != RESS_NORM_NONE) {
    for (int i = tid; i < p.D; i += kThreads) {
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        wb[2 * a][i] = p.part[a].weight ? p.part[a].weight[i] : 1.f;
        wb[2 * a + 1][i] = p.part[a].bias ? p.part[a].bias[i] : 0.f;
      }
    }
  }
  __syncthreads();
  for (int i = i0; i < i1;) {
    i += tb - ta;
    const long long out_t = p.part[which].out_t;
    const bool work = p.part[which].work;
    uint64_t w[V], bias[V];  // V / 2 pairs of chunk a, then of chunk b
    if (norm != RESS_NORM_NONE && work) {
      const int ra = holds ? ca : 0, rb = holds ? cb : 0;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        w[e] = *reinterpret_cast<const uint64_t *>(&wb[2 * which][ra + 2 * e]);
        w[V / 2 + e] = *reinterpret_cast<const uint64_t *>(&wb[2 * which][rb + 2 * e]);
        bias[e] = *reinterpret_cast<const uint64_t *>(&wb[2 * which + 1][ra + 2 * e]);
        bias[V / 2 + e] = *reinterpret_cast<const uint64_t *>(&wb[2 * which + 1][rb + 2 * e]);
      }
    }
    for (int t = ta; t < tb; t += kPieces) {
      Raw raw[kPieces][2];
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        raw[u][0] = next[u][0];
        raw[u][1] = next[u][1];
      }
      load(t + kPieces);
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        if (t + u >= tb) break;
        if (work) {
          uint64_t x[V];
          unpack(raw[u][0], x);
          unpack(raw[u][1], x + V / 2);
          if (norm != RESS_NORM_NONE) {
            if (norm == RESS_NORM_LAYER) {
              uint64_t m = x[0];
#pragma unroll
              for (int e = 1; e < V; ++e) m = add2(m, x[e]);
              const float total = row_sum(lo2(m) + hi2(m), lpr);
              const float mean = holds ? total * inv_d : 0.f;  // idle lanes stay 0
              const uint64_t m2 = pk2(-mean, -mean);
#pragma unroll
              for (int e = 0; e < V; ++e) x[e] = add2(x[e], m2);
            }
            uint64_t ss = mul2(x[0], x[0]);
#pragma unroll
            for (int e = 1; e < V; ++e) ss = fma2(x[e], x[e], ss);
            const float r = rsqrtf(fmaf(row_sum(lo2(ss) + hi2(ss), lpr), inv_d, p.eps));
            const uint64_t r2 = pk2(r, r);
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] = fma2(mul2(x[e], r2), w[e], bias[e]);
          }
          if (turned) {
            const float *c = cs + 2 * slots * (t + u) + own * V, *s = c + slots;
#pragma unroll
            for (int e = 0; e < V / 2; e += 2) {
              ulonglong2 ce2, se2;
              if constexpr (V >= 4) {
                ce2 = *reinterpret_cast<const ulonglong2 *>(c + 2 * e);
                se2 = *reinterpret_cast<const ulonglong2 *>(s + 2 * e);
              } else {
                ce2.x = *reinterpret_cast<const uint64_t *>(c);
                se2.x = *reinterpret_cast<const uint64_t *>(s);
              }
#pragma unroll
              for (int f = 0; f < (V >= 4 ? 2 : 1); ++f) {
                const uint64_t ce = f ? ce2.y : ce2.x, se = f ? se2.y : se2.x;
                if (HALF) {  // pairs (x_a, x_b)
                  const uint64_t ns = se ^ 0x8000000080000000ull;
                  const uint64_t a = x[e + f], d = x[V / 2 + e + f];
                  x[e + f] = fma2(d, ns, mul2(a, ce));
                  x[V / 2 + e + f] = fma2(a, se, mul2(d, ce));
                } else {  // pairs inside the packed values
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    if (own * V + 2 * (e + f) + k >= pairs) continue;
                    const float cc = k ? hi2(ce) : lo2(ce), sn = k ? hi2(se) : lo2(se);
                    const float a = lo2(x[2 * (e + f) + k]), d = hi2(x[2 * (e + f) + k]);
                    x[2 * (e + f) + k] = pk2(fmaf(-d, sn, a * cc), fmaf(a, sn, d * cc));
                  }
                }
              }
            }
          }
          repack(x, raw[u][0]);
          repack(x + V / 2, raw[u][1]);
        }
        if (there) {
          T *row = dst + to[t + u] * out_t;
          *reinterpret_cast<Raw *>(row + ca) = raw[u][0];
          *reinterpret_cast<Raw *>(row + cb) = raw[u][1];
        }
      }
    }
    if (i < i1) open(i);
  }
}

// ------------------------------------------------------------------- element form
// What the chunk form leaves: odd head sizes and addresses, and sections of wide heads that
// only single elements halve.  A warp takes the rows of a token one after another, elements
// spread over its lanes.
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

template <typename T, int V, bool HALF>
void launch_chunks(const TokenParams &p, unsigned ctas, cudaStream_t st) {
  if constexpr (V * sizeof(T) < 16)
    token_chunk_kernel<T, V, HALF, kAnyNorm><<<ctas, kThreads, 0, st>>>(p);
  else if (p.norm == RESS_NORM_NONE)
    token_chunk_kernel<T, V, HALF, RESS_NORM_NONE><<<ctas, kThreads, 0, st>>>(p);
  else if (p.norm == RESS_NORM_RMS)
    token_chunk_kernel<T, V, HALF, RESS_NORM_RMS><<<ctas, kThreads, 0, st>>>(p);
  else
    token_chunk_kernel<T, V, HALF, RESS_NORM_LAYER><<<ctas, kThreads, 0, st>>>(p);
}

template <typename T>
cudaError_t launch_typed(TokenParams &p, int sms, cudaStream_t st) {
  // the widest chunks whose pairs make up a row in at most 32 lanes, lie on their boundaries
  // in every tensor, and (half layout) halve a section
  const bool half = p.layout == RESS_ROPE_HALF;
  int V = 16 / (int)sizeof(T);
  for (; V >= 2; V /= 2) {
    bool fits = V * sizeof(T) >= 4 && p.D % (2 * V) == 0 && p.D / (2 * V) <= 32;
    if (p.rot > 0 && half) fits = fits && (p.rot / p.axes) % (2 * V) == 0;
    for (int i = 0; i < p.parts; ++i) {
      const Part &q = p.part[i];
      fits = fits && aligned(q.in, V * sizeof(T)) && aligned(q.out, V * sizeof(T));
      for (long long s : {q.in_b, q.in_h, q.in_t, q.out_b, q.out_h, q.out_t}) fits = fits && s % V == 0;
    }
    if (fits) break;
  }
  const long long tokens = (long long)p.B * p.N;
  if (V >= 2) {
    // full waves of resident CTAs, of as many tokens as their angles have room for
    const long long most = kAngleFloats / p.D < kMaxTile ? kAngleFloats / p.D : kMaxTile;
    const bool lean = p.norm == RESS_NORM_NONE && V * sizeof(T) == 16;
    const long long wave = (long long)sms * (lean ? kCtasRotate : kCtasNorm);
    const long long waves = (tokens + most * wave - 1) / (most * wave);
    const long long tile = (tokens + waves * wave - 1) / (waves * wave);
    p.tile = (int)(tile < p.N ? tile : p.N);
    p.tiles = (p.N + p.tile - 1) / p.tile;
    const unsigned ctas = (unsigned)((long long)p.tiles * p.B);
    constexpr int W = 16 / sizeof(T);
    if (V == W)
      half ? launch_chunks<T, W, true>(p, ctas, st) : launch_chunks<T, W, false>(p, ctas, st);
    else if (V == W / 2)
      half ? launch_chunks<T, W / 2, true>(p, ctas, st) : launch_chunks<T, W / 2, false>(p, ctas, st);
    else if constexpr (W == 8)
      half ? launch_chunks<T, 2, true>(p, ctas, st) : launch_chunks<T, 2, false>(p, ctas, st);
    return cudaGetLastError();
  }
  int rows = 0;
  for (int i = 0; i < p.parts; ++i) rows += p.part[i].heads;
  // few tokens: spread a token's heads over warps until the card has some for every
  // scheduler; each then computes the token's angles again
  const long long want = (long long)sms * 16;
  p.groups = (int)(tokens >= want ? 1 : (want + tokens - 1) / tokens);
  if (p.groups > rows) p.groups = rows;
  p.tasks = tokens * p.groups;
  long long ctas = (p.tasks + kWarps - 1) / kWarps;
  if (ctas > (long long)sms * 8) ctas = (long long)sms * 8;
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
