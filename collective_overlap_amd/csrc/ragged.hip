// Products of rows grouped by expert: row r of the row operands belongs to
// the expert e with offsets[e] <= r < offsets[e + 1].
//
//   forward  C[r, n]   = sum_k A[r, k] B_e[n, k]
//   dgrad    A[r, k]   = sum_n C[r, n] B_e[n, k]
//   wgrad    B_e[n, k] = sum over the expert's rows r of C[r, n] A[r, k]
//
// bf16 operands, fp32 accumulation.  The offsets are read on the device, so
// the host needs no count of any expert's rows.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>

#include "cce_internal.hpp"

namespace cce {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// One product per expert, X[i, l] Y[j, l] summed over l, with any strides.
struct RArgs {
  const __bf16* x;
  const __bf16* y;
  void* z;
  const int64_t* offsets;
  int64_t T;
  int experts, I, J, L;       // extents that do not depend on the expert
  int64_t xi, xl, xe;         // strides of X along i, l and from expert to expert
  int64_t yj, yl, ye;
  int64_t zi, ze;             // strides of the result along i and from expert to expert
  int tiles_j;
  bool rows_i;                // the expert's rows are i (forward, dgrad) or l (wgrad)
};

// The next row number of the offsets: kept within [0, T] and not below the one
// before, so that no access leaves the operands and no row has two experts,
// whatever the offsets hold.
__device__ __forceinline__ int64_t next_row(const int64_t* offsets, int e, int64_t T, int64_t before) {
  return min(max(offsets[e], before), T);
}

template <typename TOut>
__global__ __launch_bounds__(256) void ragged_kernel(RArgs a) {
  constexpr int B = 64, BL = 32, ROW = BL + 8;
  __shared__ __attribute__((aligned(16))) __bf16 shx[B * ROW];
  __shared__ __attribute__((aligned(16))) __bf16 shy[B * ROW];
  int t = blockIdx.x / a.tiles_j;
  const int tj = blockIdx.x - t * a.tiles_j;
  int e = 0;
  int64_t lo = 0, hi = 0;
  if (a.rows_i) {
    hi = next_row(a.offsets, 0, a.T, 0);
    for (;; ++e) {
      if (e == a.experts) return;
      lo = hi;
      hi = next_row(a.offsets, e + 1, a.T, lo);
      const int tiles = static_cast<int>((hi - lo + B - 1) / B);
      if (t < tiles) break;
      t -= tiles;
    }
  } else {
    const int tiles_i = (a.I + B - 1) / B;
    e = t / tiles_i;
    t -= e * tiles_i;
    for (int i = 0; i <= e; ++i) lo = next_row(a.offsets, i, a.T, lo);
    hi = next_row(a.offsets, e + 1, a.T, lo);
  }
  const int64_t I = a.rows_i ? hi - lo : a.I;
  const int64_t L = a.rows_i ? a.L : hi - lo;
  const __bf16* x = a.x + e * a.xe + (a.rows_i ? lo * a.xi : lo * a.xl);
  const __bf16* y = a.y + e * a.ye + (a.rows_i ? 0 : lo * a.yl);
  TOut* z = reinterpret_cast<TOut*>(a.z) + e * a.ze + (a.rows_i ? lo * a.zi : 0);
  const int64_t i0 = static_cast<int64_t>(t) * B;
  const int j0 = tj * B;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wi = (wave >> 1) * 32, wj = (wave & 1) * 32;
  const int r = lane & 31, h = lane >> 5;
  f32x16 acc = {};
  for (int64_t l0 = 0; l0 < L; l0 += BL) {
    __syncthreads();
    for (int p = tid; p < B * BL; p += 256) {
      // consecutive threads along the operand's contiguous dimension
      const int ix = a.xl == 1 ? p / BL : p % B, lx = a.xl == 1 ? p % BL : p / B;
      const int iy = a.yl == 1 ? p / BL : p % B, ly = a.yl == 1 ? p % BL : p / B;
      shx[ix * ROW + lx] = i0 + ix < I && l0 + lx < L ? x[(i0 + ix) * a.xi + (l0 + lx) * a.xl] : __bf16(0.0f);
      shy[iy * ROW + ly] = j0 + iy < a.J && l0 + ly < L ? y[(j0 + iy) * a.yj + (l0 + ly) * a.yl] : __bf16(0.0f);
    }
    __syncthreads();
#pragma unroll
    for (int l = 0; l < BL; l += 16) {
      const bf16x8 fx = *reinterpret_cast<const bf16x8*>(shx + (wi + r) * ROW + l + 8 * h);
      const bf16x8 fy = *reinterpret_cast<const bf16x8*>(shy + (wj + r) * ROW + l + 8 * h);
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fy, fx, acc, 0, 0, 0);
    }
  }
  const int64_t i = i0 + wi + r;
  if (i >= I) return;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int j = j0 + wj + 8 * (q / 4) + 4 * h + q % 4;
    if (j < a.J) z[i * a.zi + j] = static_cast<TOut>(acc[q]);
  }
}

}  // namespace

cce_status launch_ragged(const RaggedLaunch& L, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  RArgs r{};
  r.offsets = L.offsets;
  r.T = L.T;
  r.experts = L.experts;
  r.rows_i = L.kind != RAGGED_WGRAD;
  const __bf16* a = static_cast<const __bf16*>(L.a);
  const __bf16* b = static_cast<const __bf16*>(L.b);
  const __bf16* c = static_cast<const __bf16*>(L.c);
  if (L.kind == RAGGED_FORWARD) {
    r.x = a; r.xi = L.lda; r.xl = 1;
    r.y = b; r.yj = L.ldb; r.yl = 1; r.ye = L.stride_b;
    r.z = L.c; r.zi = L.ldc;
    r.J = static_cast<int>(L.N); r.L = static_cast<int>(L.K);
  } else if (L.kind == RAGGED_DGRAD) {
    r.x = c; r.xi = L.ldc; r.xl = 1;
    r.y = b; r.yj = 1; r.yl = L.ldb; r.ye = L.stride_b;
    r.z = L.a; r.zi = L.lda;
    r.J = static_cast<int>(L.K); r.L = static_cast<int>(L.N);
  } else {
    r.x = c; r.xi = 1; r.xl = L.ldc;
    r.y = a; r.yj = 1; r.yl = L.lda;
    r.z = L.b; r.zi = L.ldb; r.ze = L.stride_b;
    r.I = static_cast<int>(L.N); r.J = static_cast<int>(L.K);
  }
  r.tiles_j = (r.J + 63) / 64;
  const int64_t tiles_i = r.rows_i ? L.T / 64 + L.experts : static_cast<int64_t>(L.experts) * ((r.I + 63) / 64);
  if (tiles_i * r.tiles_j > 0x7fffffff) return fail(CCE_EUNSUPPORTED, "ragged GEMM: too many output tiles");
  const dim3 grid(static_cast<unsigned>(tiles_i * r.tiles_j));
  if (L.out_t == CCE_F32) ragged_kernel<float><<<grid, 256, 0, s>>>(r);
  else ragged_kernel<__bf16><<<grid, 256, 0, s>>>(r);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(CCE_EHIP, std::string("ragged GEMM launch: ") + hipGetErrorString(e));
  return CCE_OK;
}

}  // namespace cce
