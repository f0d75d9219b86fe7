// score_rule.cuh -- the rule on attention logits (cap and distance bias) shared by the attention kernels.
#pragma once

#include <float.h>
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
// Under a negative slope far keys lead, with a bias whose fp32 step is coarse (1/16 in log2 units at slope -1/2 and 1M
// tokens). Such a row's logits are therefore taken relative to the bias of its farthest key, whose distance this is:
// `first` is the window's first position, j the row's first entry (below 0 or not visible: none). Entry 0 stands at
// the middle of its block, so while the window begins before that its first token is the farther one. Any other key
// would do as well for the answer, at the price of a coarser step.
__device__ __forceinline__ float far_distance(int64_t t, int64_t first, int64_t j, int m, int n_win) {
  const float w = static_cast<float>(t - first);
  return j >= 0 && j * m < t + 1 - n_win ? fmaxf(entry_distance(t, j, m), w) : w;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}
// a max of three, and of the magnitudes of three
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// cap tanh(s pre) as a polynomial in s where |s pre| <= 1, to a relative error of 6e-7: tanh(u) / u in u^2 on [0, 1]
// (fitted like tanh_rational), its coefficients times cap2 pre^(2i + 1). Logits seldom reach the cap, so most tiles
// take this form: 7 fp32 operations a logit instead of 12, and no reciprocal.
constexpr float kTanhP[6] = {0.9999994039535522f, -0.3332904279232025f, 0.13281434774398804f,
                             -0.051605693995952606f, 0.016743136569857597f, -0.0030670680571347475f};
// The rule's numbers, as a kernel argument: packed arithmetic then reads its constants, each a pair of the same number,
// where they are instead of building the pairs in registers.
struct Rule {
  float2 pre, cap2;  // capped: sm_scale / cap and cap log2(e); else sm_scale log2(e) and 0
  float2 c[6];
  float lim;         // |s| up to here takes the polynomial (negative: never)
};
// The coefficients span pre^11, so with a scale far from 1 the last ones leave fp32's range. Above it the rational form
// is taken for every logit. Below it (caps above ~430 at the usual scales) they are left out, and the polynomial is taken
// where the first one left out would add less than 2^-24 of the sum: |u| <= kTanhU[m] with m coefficients, the 2m-th root of
// 2^-24 / |kTanhP[m]|. s^2 has to stay in range as well, which 2^60 keeps it.
constexpr float kTanhU[7] = {0.f, 4.2e-4f, 0.0258f, 0.102f, 0.208f, 0.337f, 1.f};
inline Rule make_rule(float sm_scale, float score_cap) {
  const float log2e = 1.4426950408889634f;
  const bool cap = score_cap > 0.f;
  Rule r;
  const float pre = cap ? sm_scale / score_cap : sm_scale * log2e, cap2 = cap ? score_cap * log2e : 0.f;
  r.pre = make_float2(pre, pre);
  r.cap2 = make_float2(cap2, cap2);
  int kept = 0;
  bool fits = pre < 2048.f;
  float f = cap2 * pre;
  for (int i = 0; i < 6; ++i) {
    if (kept == i && f >= 0x1p-125f) kept = i + 1;
    const float c = kept > i ? f * kTanhP[i] : 0.f;
    r.c[i] = make_float2(c, c);
    fits = fits && f <= FLT_MAX;
    f *= pre * pre;
  }
  const float lim = kTanhU[kept] / pre;
  r.lim = !fits ? -1.f : lim < 0x1p60f ? lim : 0x1p60f;
  return r;
}

// The rule on N logits, two packed pairs in step: with the cap, without, or capped below lim. bias = slope2 * position
// - ref, ref the row's running maximum so far (its subtraction costs nothing here).
enum { kLinear, kRational, kPoly };
template <int FORM, int N>
__device__ __forceinline__ void rule_n(uint32_t (&s)[N], const float4* pos, const Rule& r, float2 slope,
                                       float2 negref) {
#pragma unroll
  for (int b = 0; b < N; b += 4) {
    const float4 pa = pos[b / 4];
    float2 u[2] = {make_float2(__uint_as_float(s[b]), __uint_as_float(s[b + 1])),
                   make_float2(__uint_as_float(s[b + 2]), __uint_as_float(s[b + 3]))};
    const float2 bias[2] = {__ffma2_rn(slope, make_float2(pa.x, pa.y), negref), __ffma2_rn(slope, make_float2(pa.z, pa.w), negref)};
    if constexpr (FORM == kLinear) {
#pragma unroll
      for (int j = 0; j < 2; ++j) u[j] = __ffma2_rn(u[j], r.pre, bias[j]);
    } else if constexpr (FORM == kPoly) {
      float2 x[2], n[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) x[j] = __fmul2_rn(u[j], u[j]);
#pragma unroll
      for (int j = 0; j < 2; ++j) n[j] = __ffma2_rn(r.c[5], x[j], r.c[4]);
#pragma unroll
      for (int i = 3; i >= 0; --i)
#pragma unroll
        for (int j = 0; j < 2; ++j) n[j] = __ffma2_rn(n[j], x[j], r.c[i]);
#pragma unroll
      for (int j = 0; j < 2; ++j) u[j] = __ffma2_rn(u[j], n[j], bias[j]);
    } else {
      float2 x[2], n[2], d[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        u[j] = __fmul2_rn(u[j], r.pre);
        u[j] = make_float2(tanh_clamp(u[j].x), tanh_clamp(u[j].y));
        x[j] = __fmul2_rn(u[j], u[j]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) d[j] = __ffma2_rn(make_float2(tanh_d(4), tanh_d(4)), x[j], make_float2(tanh_d(3), tanh_d(3)));
#pragma unroll
      for (int i = 2; i >= 0; --i)
#pragma unroll
        for (int j = 0; j < 2; ++j) d[j] = __ffma2_rn(d[j], x[j], make_float2(tanh_d(i), tanh_d(i)));
#pragma unroll
      for (int j = 0; j < 2; ++j) n[j] = __ffma2_rn(make_float2(tanh_n(3), tanh_n(3)), x[j], make_float2(tanh_n(2), tanh_n(2)));
#pragma unroll
      for (int i = 1; i >= 0; --i)
#pragma unroll
        for (int j = 0; j < 2; ++j) n[j] = __ffma2_rn(n[j], x[j], make_float2(tanh_n(i), tanh_n(i)));
#pragma unroll
      for (int j = 0; j < 2; ++j) n[j] = __fmul2_rn(n[j], u[j]);
      // two quotients share one reciprocal: 1 / d_a = d_b / (d_a d_b), each d at most 2^7.3
      const float2 dd = __fmul2_rn(d[0], d[1]);
      float2 rc;
      asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(rc.x) : "f"(dd.x));
      asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(rc.y) : "f"(dd.y));
      rc = __fmul2_rn(rc, r.cap2);
      u[0] = __ffma2_rn(__fmul2_rn(n[0], d[1]), rc, bias[0]);
      u[1] = __ffma2_rn(__fmul2_rn(n[1], d[0]), rc, bias[1]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      s[b + 2 * j] = __float_as_uint(u[j].x);
      s[b + 2 * j + 1] = __float_as_uint(u[j].y);
    }
  }
}

// The rule on N logits of a row, in place: pos holds each key's position relative to some reference of the row's, and
// negref what is added to every logit (before the rounding of the bias: slope2 * pos is exact inside the sum).
template <bool CAP, int N>
__device__ __forceinline__ void apply_rule(uint32_t (&s)[N], const float4* pos, const Rule& r, float slope2,
                                           float negref) {
  const float2 sl = make_float2(slope2, slope2), nr = make_float2(negref, negref);
  if constexpr (CAP) {
    float big = 0.f, big1 = 0.f;
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      big = max3_abs(big, __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
      big1 = max3_abs(big1, __uint_as_float(s[j + 2]), __uint_as_float(s[j + 3]));
    }
    if (__all_sync(0xffffffffu, fmaxf(big, big1) <= r.lim))
      rule_n<kPoly>(s, pos, r, sl, nr);
    else
      rule_n<kRational>(s, pos, r, sl, nr);
  } else {
    rule_n<kLinear>(s, pos, r, sl, nr);
  }
}

}  // namespace cskv
