// GELU as the 8-bit product applies it (gemm8.hip): to bf16 results with the
// same arithmetic as the grouped GEMM's epilogue (gemm.hip), to fp32 results in
// fp32's own accuracy.
#pragma once

#include <hip/hip_runtime.h>

namespace cce {

// Exact (erf) GELU, x * Phi(x) = 0.5 x (1 + erf(x / sqrt 2)).  erf comes from
// the rational approximation of Abramowitz and Stegun, Handbook of
// Mathematical Functions, formula 7.1.26 (absolute error <= 1.5e-7):
//   erfc(a) ~ t (a1 + t (a2 + t (a3 + t (a4 + t a5)))) exp(-a^2),
//   t = 1 / (1 + p a), a >= 0,
// and 1 + erf(u) is formed as 2 - erfc(|u|) for u >= 0 and erfc(|u|) for
// u < 0, so the negative tail has no cancellation.  About a dozen VALU
// operations against several dozen for the library erff; the epilogue runs
// while the matrix cores idle, so its length shows in the kernel time.
__device__ __forceinline__ float gelu_exact(float x) {
  const float u = x * 0.70710678118654752f;
  const float a = fabsf(u);
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.3275911f * a);
  const float poly =
      t * (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f +
                                                                          t * 1.061405429f))));
  const float q = poly * __expf(-(a * a));
  return 0.5f * x * (u >= 0.0f ? 2.0f - q : q);
}

// For fp32 results: the form above is off by up to 1.5e-7 of x, which is 2^-9 of
// the result at x = -4.  Here erfc's error is relative:
//   erfc(|x| / sqrt 2) = exp(-x^2 / 2) t P(t),  t = 1 / (1 + p |x|),
// with P of degree 8 fitted to t P(t) exp(-x^2 / 2) for the least largest
// relative error up to |x| = 14 (beyond, the result is below fp32's range; 8e-8
// with the coefficients in fp32).  In units of u = 2^-24 the result is off by at
// most 1.2 x^2 + 20: x^2 and its factor in the exponent 1.2 x^2, t 3 (times 3,
// erfc's sensitivity), P 5, the exponential 2, the products 3.  (In a 4096 x
// 6144 x 4096 product of 189 us the library's erfcf takes 17 us more, this none
// more than the form above.)
__device__ __forceinline__ float gelu_f32(float x) {
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.265f * fabsf(x));
  float p = 0.0615282245f;
  p = p * t - 0.287920982f;
  p = p * t + 0.434552044f;
  p = p * t - 0.231524169f;
  p = p * t + 0.275096476f;
  p = p * t + 0.120963767f;
  p = p * t + 0.205317155f;
  p = p * t + 0.210505053f;
  p = p * t + 0.21148245f;
  const float q = p * t * __builtin_amdgcn_exp2f(x * x * -0.72134752f);
  return 0.5f * x * (x >= 0.0f ? 2.0f - q : q);
}

template <typename TOut>
__device__ __forceinline__ float gelu_for(float x) {
  if constexpr (sizeof(TOut) == 4) return gelu_f32(x);
  else return gelu_exact(x);
}

}  // namespace cce
