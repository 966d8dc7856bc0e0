// The soft-cap of a score to fp32 accuracy, for the kernels that take their scores in log2
// units from fp32 sums.
#pragma once

#include "common.cuh"

namespace mattn {

// Soft-cap: cap tanh(s / cap), s and cap in log2 units, inv = 2 / cap (natural).
// Where |s / cap| < 1/4: s (1 - x^2/3 + 2 x^4/15 - 17 x^6/315 + 62 x^8/2835), x = s / cap,
// off by 2^-26 s.
constexpr float kCapNear = 0.25f * 2.0f / 0.69314718f;  // that bound on s inv
__device__ __forceinline__ float soft_cap_near(float s, float inv) {
  constexpr float kX2 = 0.25f * 0.69314718f * 0.69314718f;  // x = s inv ln 2 / 2
  const float y = s * inv, y2 = y * y;
  float p = fmaf(y2, 62.0f / 2835.0f * kX2 * kX2 * kX2 * kX2, -17.0f / 315.0f * kX2 * kX2 * kX2);
  p = fmaf(y2, p, 2.0f / 15.0f * kX2 * kX2);
  p = fmaf(y2, p, -1.0f / 3.0f * kX2);
  return fmaf(s * y2, p, s);
}

// Anywhere: beyond that bound cap - 2 cap / (1 + e^(2 s / cap)), off by at most 2^-22 cap
// (below it that would be many times the score's own rounding: 0.2 for a cap of 10^6).
__device__ __forceinline__ float soft_cap(float s, float cap2, float inv) {
  const float y = s * inv;
  const float far = fmaf(-cap2, __fdividef(2.0f, 1.0f + ex2_approx(y)), cap2);
  return fabsf(y) < kCapNear ? soft_cap_near(s, inv) : far;
}

}  // namespace mattn
