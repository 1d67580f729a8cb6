// GELU as the 8-bit product applies it (gemm8.hip): the same arithmetic as the
// grouped GEMM's epilogue (gemm.hip), so that both give the same bits.
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

}  // namespace cce
