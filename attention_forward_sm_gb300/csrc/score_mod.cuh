// The score modifications of the attention calls with modified scores, on the
// device: the tanh cap and the distance bias.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace attn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994530942f;

// tanh(x) = x T(x^2) for |x| <= 1, T of degree 5: interpolation of tanh(x) / x
// in the Chebyshev points of x^2 on [0, 1].  Its nearest singularity is at
// x^2 = -pi^2 / 4, so every further coefficient gains a factor of 11.8; this
// one is off by 7e-7 of the value at most, a few roundings of the score.
__device__ __forceinline__ float tanh_poly(float x) {
  const float y = x * x;
  float t = fmaf(y, -0x1.90d924p-9f, 0x1.11f45ap-6f);
  t = fmaf(y, t, -0x1.a697a8p-5f);
  t = fmaf(y, t, 0x1.0ffd3ap-3f);
  t = fmaf(y, t, -0x1.5549d8p-2f);
  t = fmaf(y, t, 0x1.ffffecp-1f);
  return x * t;
}

// tanh for any x.  Beyond 1: 1 - 2 / (1 + e^(2|x|)), which loses nothing there
// (the fraction is below 0.24) and goes to 1 for infinite x.
__device__ __forceinline__ float tanh_any(float x) {
  const float e = ex2_approx(fabsf(x) * (2.f * kLog2e));
  const float far = copysignf(1.f - __fdividef(2.f, 1.f + e), x);
  return fabsf(x) <= 1.f ? tanh_poly(x) : (x == x ? far : x);
}

// The bias is taken relative to the visible key that it favours, at distance
// ref: the nearest one for a slope >= 0, the farthest one otherwise.  Scores
// then keep their fp32 digits however far all visible keys are, and the LSE
// gets the common part -slope * ref back at the end.  For keys [lo, hi):
__device__ __forceinline__ int bias_ref(float slope, int pos, int lo, int hi) {
  const int near = pos < lo ? lo - pos : (pos >= hi ? pos - (hi - 1) : 0);
  const int far = max(abs(pos - lo), abs(pos - (hi - 1)));
  return slope >= 0.f ? near : far;
}

}  // namespace attn
