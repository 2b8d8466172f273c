// What the two forms of attention with changed scores share (k_masked_attn.cu, tensor-core
// tiles; k_masked_step.cu, few rows).
#pragma once

#include "ress_common.cuh"
#include "ress_internal.h"

namespace ress {

constexpr float kNoMax = -3.0e38f;  // running max of a row that has seen no key
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994530942f;

RESS_DEV float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(y) / y as a polynomial in y^2, fitted here for minimax relative error (Lawson's
// iteratively reweighted least squares): up to |y| = 3/8 (degree 3, 5.9e-8), up to 1/2
// (degree 4, 1.3e-8; 1.1e-7 evaluated in fp32) and up to 1 (degree 6, 5e-8; 1.6e-7).
constexpr double kTanhFit3[4] = {9.999999404e-01, -3.333197534e-01, 1.328450292e-01, -4.827226326e-02};
template <int N>
RESS_DEV constexpr float tanh_fit(int k) {
  constexpr float c4[5] = {1.000000000e+00f, -3.333306909e-01f, 1.332477927e-01f, -5.298607424e-02f,
                           1.713500544e-02f};
  constexpr float c6[7] = {9.999999404e-01f, -3.333283961e-01f, 1.332520396e-01f, -5.345702916e-02f,
                           2.028998174e-02f, -6.203379016e-03f, 1.041022479e-03f};
  return N == 4 ? c4[k < 5 ? k : 4] : c6[k];
}

// Any y: 1 - 2 / (1 + e^2y) is off by an fp32 unit absolutely, the polynomial below |y| = 1/2
// relatively.
RESS_DEV float tanh_any(float y) {
  const float t = y * y;
  float a = tanh_fit<4>(4);
#pragma unroll
  for (int k = 3; k >= 0; --k) a = fmaf(a, t, tanh_fit<4>(k));
  const float r = rcp_approx(1.0f + ex2_approx(2.0f * kLog2e * y));
  return fabsf(y) < 0.5f ? a * y : fmaf(-2.0f, r, 1.0f);
}

// Whether the form for few rows takes a call, and that form.
bool masked_step_fits(const Dims &d, int q_len);
cudaError_t launch_masked_step(const Dims &d, const MaskedAttnLaunch &a, cudaStream_t st);

}  // namespace ress
