// Vectors of 8 consecutive columns, in float, as the row-wise kernels read
// and write them (norm.hip), and the e4m3 / power-of-two scale arithmetic
// that they share with the 8-bit product (gemm8.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace cce {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct e4m3 {          // one byte of OCP E4M3 (finite, NaN 0x7f / 0xff, no infinities)
  uint8_t v;
};

constexpr int kScaleCols = 128;   // columns that share a scale

// Column j of a row of n columns lies before its end.  Unsigned, and so the sums
// and products that give j: the last lanes' columns may lie past 2^31, where n
// is close to it.
__device__ __forceinline__ bool before(uint32_t j, int n) { return j < static_cast<uint32_t>(n); }

// Columns [j, j + 8) of a row at `base` (16-byte aligned with j a multiple of
// 8); columns from n on read as zero.  NT: streamed past the caches.  (bf16 is
// widened inside the check of the row's end, so the compiled code waits there
// for each load: several in a row do not overlap within a wave, as fp32 ones do.)
template <typename T, bool NT = false>
__device__ __forceinline__ void load8(const T* base, uint32_t j, int n, float (&v)[8]) {
  if (before(j + 7, n)) {
    if constexpr (sizeof(T) == 4) {
      const f32x4* p = reinterpret_cast<const f32x4*>(base + j);
      const f32x4 x = NT ? __builtin_nontemporal_load(p) : p[0];
      const f32x4 y = NT ? __builtin_nontemporal_load(p + 1) : p[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = x[e];
        v[e + 4] = y[e];
      }
    } else {
      const u32x4* p = reinterpret_cast<const u32x4*>(base + j);
      const bf16x8 x = __builtin_bit_cast(bf16x8, NT ? __builtin_nontemporal_load(p) : *p);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = static_cast<float>(x[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = before(j + e, n) ? static_cast<float>(base[j + e]) : 0.0f;
  }
}

// One rounding to T (to nearest even), columns from n on left alone.
template <typename T>
__device__ __forceinline__ void store8(T* base, uint32_t j, int n, const float (&v)[8]) {
  if (before(j + 7, n)) {
    if constexpr (sizeof(T) == 4) {
      f32x4* p = reinterpret_cast<f32x4*>(base + j);
      __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, p);
      __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, p + 1);
    } else {
      bf16x8 h;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = static_cast<__bf16>(v[e]);
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4, h), reinterpret_cast<u32x4*>(base + j));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (before(j + e, n)) base[j + e] = static_cast<T>(v[e]);
  }
}

// 8 values to e4m3, each rounded to nearest even.
__device__ __forceinline__ void store8_e4m3(uint8_t* base, uint32_t j, int n, const float (&v)[8]) {
  u32x2 w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], p, true);
    w[h] = static_cast<unsigned>(p);
  }
  if (before(j + 7, n)) {
    __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(base + j));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (before(j + e, n)) base[j + e] = static_cast<uint8_t>(w[e / 4] >> (8 * (e % 4)));
  }
}

// Magnitude of a float as an unsigned integer: ordered like the magnitudes,
// with infinity above every number and NaN above infinity, so that a maximum
// over it keeps both.
__device__ __forceinline__ uint32_t magnitude(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
}

// The E8M0 scale of a block whose largest magnitude has these bits: 2^(s - 127)
// is the smallest power of two, 2^-126 at least, that brings it to 448 (1.75 *
// 2^8) or below.  A block with an infinity or a NaN gets 255, E8M0's NaN.
__device__ __forceinline__ uint32_t scale_of(uint32_t top) {
  const int e = static_cast<int>(top >> 23);
  if (e == 255) return 255u;
  const int s = e - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(s < 1 ? 1 : s);
}

// 1 / 2^(s - 127) for a scale of scale_of: an exact factor (NaN for 255).
__device__ __forceinline__ float inverse_of(uint32_t s) {
  return __builtin_bit_cast(float, s == 255u ? 0x7fc00000u : (254u - s) << 23);
}

}  // namespace cce
