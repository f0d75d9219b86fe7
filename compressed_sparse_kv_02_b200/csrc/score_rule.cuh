// score_rule.cuh -- the rule on attention logits (cap and distance bias) shared by the attention kernels.
#pragma once

#include <stdint.h>

namespace cskv {

// tanh(u) to a relative error of 4e-7, with one reciprocal: an odd rational function u N(u^2) / D(u^2) fitted to
// tanh(u) / u in the relative minimax sense on |u| <= 8 (own fit: weighted least squares on Chebyshev nodes,
// reweighted by the error), clamped there (1 - tanh(8) = 2.3e-7). The relative form keeps small arguments, so a
// large cap leaves the logits as they are; 1 - 2 / (1 + e^2u) would lose cap * 2^-23 and take a second
// special-function operation, which is what bounds the capped softmax (16 per clock and SM).
__host__ __device__ constexpr float tanh_n(int i) {  // coefficients of N and D, constant term first
  return i == 0 ? 0.9999998807907104f : i == 1 ? 0.12925660610198975f : i == 2 ? 0.002951021073386073f
                                                                               : 1.1428394827817101e-05f;
}
__host__ __device__ constexpr float tanh_d(int i) {
  return i == 0 ? 1.f : i == 1 ? 0.46258875727653503f : i == 2 ? 0.023815542459487915f
                      : i == 3 ? 0.00023866878473199904f : 2.4592020508862333e-07f;
}
// u limited to |u| <= 8; a NaN stays one
__device__ __forceinline__ float tanh_clamp(float u) {
  float r;
  asm("min.NaN.xorsign.abs.f32 %0, %1, 0f41000000;\n" : "=f"(r) : "f"(u));
  return r;
}
__device__ __forceinline__ float tanh_rational(float u) {
  u = tanh_clamp(u);
  const float x = u * u;
  const float n = fmaf(fmaf(fmaf(tanh_n(3), x, tanh_n(2)), x, tanh_n(1)), x, tanh_n(0));
  const float d = fmaf(fmaf(fmaf(fmaf(tanh_d(4), x, tanh_d(3)), x, tanh_d(2)), x, tanh_d(1)), x, tanh_d(0));
  return __fdividef(u * n, d);  // d in [1, 2^7.3]
}
// The rule on one logit in log2 units: cap2 * tanh(s * pre) or s * pre, minus slope2 per token of distance, with
// cap2 = score_cap * log2(e), slope2 = slope * log2(e), pre = sm_scale / score_cap (capped) or sm_scale * log2(e).
template <bool CAP>
__device__ __forceinline__ float ruled_score(float s, float pre, float cap2, float slope2, float dist) {
  return fmaf(-slope2, dist, CAP ? cap2 * tanh_rational(s * pre) : s * pre);
}
// distance of entry j (mean position of its own block) from position t, in tokens: a multiple of 1/2, exact below 2^23
__device__ __forceinline__ float entry_distance(int64_t t, int64_t j, int m) {
  return 0.5f * static_cast<float>(2 * (t - j * m) - (m - 1));
}

}  // namespace cskv
