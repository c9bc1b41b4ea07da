// The gated linear recurrence's gates, candidates and maps.
#pragma once

#include <hip/hip_runtime.h>

namespace lstm {

// e^x, at most 2^126 (so that 1 + e and its reciprocal are normal numbers; a NaN stays).
// The exponential's relative error is its argument's absolute one.  For bf16 values of x
// the argument is x log2(e), rounded once: off by 1.3 |x| 2^-24, which is 2^-9 of what the
// rounding of x itself means; for fp32 values the product is taken in two parts.
template <bool BF>
__device__ __forceinline__ float exp_of(float x) {
  if constexpr (BF) {
    return __builtin_amdgcn_exp2f(__builtin_elementwise_minimum(x * 1.44269504f, 126.f));
  } else {
    constexpr float kHi = 1.4426950216293335f, kLo = 1.9259629911266175e-08f;  // log2(e)
    x = __builtin_elementwise_minimum(__builtin_elementwise_maximum(x, -104.f), 87.f);
    const float hi = x * kHi;
    const float lo = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -hi));
    const float e = __builtin_amdgcn_exp2f(hi);
    return __builtin_fmaf(e * lo, 0.69314718f, e);  // 2^(hi + lo) = 2^hi (1 + lo ln 2 + ...)
  }
}

// sigmoid(x) and 1 - sigmoid(x), each to fp32's relative accuracy: with e = exp(-x) they
// are 1 / (1 + e) and e / (1 + e).
struct Gate {
  float open, shut;
};
template <bool BF>
__device__ __forceinline__ Gate gate_of(float x) {
  const float e = exp_of<BF>(-x), a = __builtin_amdgcn_rcpf(1.f + e);
  return {a, e * a};
}
template <bool BF>
__device__ __forceinline__ float sigmoid_of(float x) {
  return __builtin_amdgcn_rcpf(1.f + exp_of<BF>(-x));
}

// What a stretch of steps makes of the state before it, c -> G + A c.  (The gradients'
// carry has the same form.)
struct Map {
  float A, G;
};
__device__ __forceinline__ float map_apply(const Map& m, float c) { return __builtin_fmaf(m.A, c, m.G); }
// `later` after `earlier`
__device__ __forceinline__ Map map_join(const Map& later, const Map& earlier) {
  return {later.A * earlier.A, map_apply(later, earlier.G)};
}

// Candidates.  For bf16 values tanh(u) = 1 - 2r with r = 1 / (1 + exp(2|u|)), and its slope 4r (1 - r).  1 - 2r
// cancels near 0, so |u| < 2^-4 takes u - u^3/3, whose next term is 2/15 u^4 of it: either is within 2^-17.5 of
// tanh(u), relative to it, 2^-8.5 of what the rounding of u to bf16 means.  (The fp32 form costs twice as much, 10 to
// 15 % of the passes' time at 32 x 500 x 4096.)
__device__ __forceinline__ float tanh_part(float u) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(2.88539008f * __builtin_fabsf(u)));
}

// For fp32 values tanh(u) = (1 - e) / (1 + e) with e = exp(-2|u|); below 1/4 its series, whose next term
// is 0.009 u^11, since 1 - e cancels there.
template <bool BF>
__device__ __forceinline__ float tanh_of(float u) {
  if constexpr (BF) {
    const float near = __builtin_fmaf(u * u, u * -0.33333333f, u);
    return __builtin_fabsf(u) < 0.0625f ? near : __builtin_copysignf(__builtin_fmaf(-2.f, tanh_part(u), 1.f), u);
  }
  const float e = exp_of<BF>(-2.f * __builtin_fabsf(u));
  const float far = (1.f - e) * __builtin_amdgcn_rcpf(1.f + e);
  const float v = u * u;
  float s = __builtin_fmaf(v, 0.021869488f, -0.053968254f);
  s = __builtin_fmaf(v, s, 0.13333333f);
  s = __builtin_fmaf(v, s, -0.33333333f);
  s = __builtin_fmaf(u * v, s, u);
  return __builtin_fabsf(u) < 0.25f ? s : __builtin_copysignf(far, u);
}

// 1 - tanh(u)^2 = 4 e / (1 + e)^2
template <bool BF>
__device__ __forceinline__ float tanh_slope(float u) {
  if constexpr (BF) {
    const float r = tanh_part(u);
    return __builtin_fmaf(-4.f * r, r, 4.f * r);
  }
  const float e = exp_of<false>(-2.f * __builtin_fabsf(u)), r = __builtin_amdgcn_rcpf(1.f + e);
  return 4.f * e * r * r;
}

}  // namespace lstm
