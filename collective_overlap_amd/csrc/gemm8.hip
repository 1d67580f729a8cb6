// Product of two e4m3 matrices whose blocks of 128 carry power-of-two scales:
//
//   C[m, n] = sum_k (A[m, k] 2^(sa[m, k/128] - 127)) (B^T[n, k] 2^(sb[n/128, k/128] - 127))
//
// with fp32 accumulation and an optional GELU on the store.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>

#include "cce_internal.hpp"
#include "elem8.hpp"
#include "gelu.hpp"

namespace cce {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct G8Args {
  const uint8_t* a;
  const uint8_t* b;
  const uint8_t* sa;
  const uint8_t* sb;
  void* c;
  int M, N, K, tiles_n;
  int64_t lda, ldb, ldc, ld_sa, ld_sb;
  bool gelu;
};

// 8 e4m3 values times their block's scale, as bf16.  The instruction takes
// the scale as a float's exponent, which is E8M0's own encoding.  Exact: a
// e4m3 value has 4 significant bits and bf16 float's exponents (results below
// 2^-126 are rounded to bf16's subnormals).
__device__ __forceinline__ bf16x8 scaled(u32x2 v, float scale) {
  bf16x8 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<int>(v[h]), scale, false);
    const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<int>(v[h]), scale, true);
    r[4 * h] = lo[0];
    r[4 * h + 1] = lo[1];
    r[4 * h + 2] = hi[0];
    r[4 * h + 3] = hi[1];
  }
  return r;
}

__device__ __forceinline__ float scale_float(uint8_t s) {
  return __builtin_bit_cast(float, static_cast<uint32_t>(s) << 23);
}

// 64 x 64 tiles, one block of 128 of the contraction at a time: both operands
// through LDS as they are, widened to bf16 on the way to the matrix cores.
template <typename TOut>
__global__ __launch_bounds__(256) void gemm8_wide_kernel(G8Args a) {
  constexpr int BM = 64, BN = 64, ROW = 128 + 16;
  __shared__ __attribute__((aligned(16))) uint8_t sha[BM * ROW];
  __shared__ __attribute__((aligned(16))) uint8_t shb[BN * ROW];
  const int tm = blockIdx.x / a.tiles_n, tn = blockIdx.x - tm * a.tiles_n;
  const int m0 = tm * BM, n0 = tn * BN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  const int r = lane & 31, h = lane >> 5;
  f32x16 acc = {};
  const int m = m0 + wm + r;
  for (int k0 = 0; k0 < a.K; k0 += 128) {
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int row = (tid >> 3) + 32 * p, c = (tid & 7) * 16;
      u32x4 va = {}, vb = {};
      if (m0 + row < a.M && k0 + c < a.K)
        va = *reinterpret_cast<const u32x4*>(a.a + static_cast<int64_t>(m0 + row) * a.lda + k0 + c);
      if (n0 + row < a.N && k0 + c < a.K)
        vb = *reinterpret_cast<const u32x4*>(a.b + static_cast<int64_t>(n0 + row) * a.ldb + k0 + c);
      *reinterpret_cast<u32x4*>(sha + row * ROW + c) = va;
      *reinterpret_cast<u32x4*>(shb + row * ROW + c) = vb;
    }
    __syncthreads();
    const int kb = k0 / 128;
    const float fa = scale_float(m < a.M ? a.sa[static_cast<int64_t>(m) * a.ld_sa + kb] : 127);
    const float fb = scale_float(a.sb[static_cast<int64_t>(n0 / 128) * a.ld_sb + kb]);
#pragma unroll
    for (int kk = 0; kk < 128; kk += 16) {
      const u32x2 xa = *reinterpret_cast<const u32x2*>(sha + (wm + r) * ROW + kk + 8 * h);
      const u32x2 xb = *reinterpret_cast<const u32x2*>(shb + (wn + r) * ROW + kk + 8 * h);
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(scaled(xb, fb), scaled(xa, fa), acc, 0, 0, 0);
    }
  }
  // the result block is C^T: the lane holds row m, columns 8 q + 4 h + e
  if (m >= a.M) return;
  TOut* c = reinterpret_cast<TOut*>(a.c) + static_cast<int64_t>(m) * a.ldc;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int n = n0 + wn + 8 * (i / 4) + 4 * h + i % 4;
    const float v = a.gelu ? gelu_exact(acc[i]) : acc[i];
    if (n < a.N) c[n] = static_cast<TOut>(v);
  }
}

}  // namespace

cce_status launch_gemm8(const Gemm8Launch& L, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  G8Args a{L.a, L.b, L.sa, L.sb, L.c, static_cast<int>(L.M), static_cast<int>(L.N), static_cast<int>(L.K), 0,
           L.lda, L.ldb, L.ldc, L.ld_sa, L.ld_sb, L.gelu};
  a.tiles_n = static_cast<int>((L.N + 63) / 64);
  const int64_t tiles = (L.M + 63) / 64 * a.tiles_n;
  if (tiles > 0x7fffffff) return fail(CCE_EUNSUPPORTED, "block-scaled GEMM: too many output tiles");
  const dim3 grid(static_cast<unsigned>(tiles));
  if (L.out_t == CCE_F32) gemm8_wide_kernel<float><<<grid, 256, 0, s>>>(a);
  else gemm8_wide_kernel<__bf16><<<grid, 256, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(CCE_EHIP, std::string("block-scaled GEMM launch: ") + hipGetErrorString(e));
  return CCE_OK;
}

}  // namespace cce
