// batch_score.cuh -- the score map of the batched attention kernels: scale,
// cap, base-2 units.
#pragma once

#include "batch.h"
#include "common.cuh"

namespace attn {

// Scores leave the map in base-2 units (times log2 e), so the softmax is 2^(s - m).
struct ScoreMap {
  float scale2;   // without a cap: scale * log2(e)
  float in_mul;   // with one: scale / cap ...
  float out_mul;  // ... and cap * log2(e)
};
inline ScoreMap score_map(const BatchArgs& a) {
  ScoreMap m{};
  m.scale2 = a.scale * kLog2e;
  if (a.softcap > 0.f) {
    m.in_mul = a.scale / a.softcap;
    m.out_mul = a.softcap * kLog2e;
  }
  return m;
}

// Powers of two on fp16 weights (in the sums, too, so they cancel): against a
// reference that lags the maximum by up to 2^8 they reach 2^15, and weights
// down to 2^-21 of the reference keep all their bits; below that each is off by
// at most 2^-32.  Without it 65536 weights of e^-18 beside a large one vanish.
constexpr float kF16Head = 7.f;

// tanh with small relative error everywhere, because the cap multiplies it and
// an exponential follows: for |x| <= 5/8 the odd polynomial x + x u q(u), u =
// x^2, with q interpolating (tanh(x)/x - 1)/u at the five Chebyshev nodes of
// [0, 25/64] (relative error 1.7e-8, 8.4e-8 in fp32); beyond, 1 - 2/(e^2x + 1),
// whose cancellation is harmless there (absolute error about 2^-23 against
// values above 0.55).
constexpr float kTanhPolyMax = 0.625f;
constexpr float kTanhQ0 = -0.333333283662796f, kTanhQ1 = 0.1333276927471161f, kTanhQ2 = -0.05385090783238411f,
                kTanhQ3 = 0.020997179672122f, kTanhQ4 = -0.006096714176237583f;
__device__ __forceinline__ float tanh_poly(float x) {
  const float u = x * x;
  float q = fmaf(kTanhQ4, u, kTanhQ3);
  q = fmaf(q, u, kTanhQ2);
  q = fmaf(q, u, kTanhQ1);
  q = fmaf(q, u, kTanhQ0);
  return fmaf(x, u * q, x);
}
__device__ __forceinline__ float tanh_exp(float x) {
  return 1.f - __fdividef(2.f, ex2(x * (2.f * kLog2e)) + 1.f);
}
// The capped score in base-2 units, rounded as the tcgen05 kernel rounds it on
// pairs of small scores: a tile takes that form or this one by what its largest
// score is, masked ones included, and its results must not tell.
__device__ __forceinline__ float capped_score(float s, const ScoreMap& sc) {
  const float x = s * sc.in_mul;
  if (!(fabsf(x) <= kTanhPolyMax)) return sc.out_mul * tanh_exp(x);
  const float y = s * (sc.in_mul * sc.out_mul), u = x * x;
  float q = fmaf(kTanhQ4, u, kTanhQ3);
  q = fmaf(q, u, kTanhQ2);
  q = fmaf(q, u, kTanhQ1);
  q = fmaf(q, u, kTanhQ0) * u;
  return fmaf(q, y, y);
}
__device__ __forceinline__ float tanh_score(float x) { return fabsf(x) <= kTanhPolyMax ? tanh_poly(x) : tanh_exp(x); }

}  // namespace attn
