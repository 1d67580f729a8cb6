// Row-wise operators beside the fused reduce epilogue: the root-mean-square
// norm of the residual stream the epilogue leaves, its backward pass, and the
// quantisation of a matrix into e4m3 blocks.
//
//   r = round(x + residual),  n = r / sqrt(mean(r^2) + eps),  y = n * w
//   dx = (w dy - n mean(w dy n)) / sqrt(mean(r^2) + eps) + d_residual
//   dw = sum over rows of dy n
//
// The norm is that of the rounded r, the tensor the next layer adds to and
// the backward pass reads, so that the gradients are those of the values in
// memory.  Every sum is in fp32 or more; r, y and dx are rounded once, on their
// store.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>
#include <type_traits>

#include "cce_internal.hpp"
#include "elem8.hpp"

namespace cce {
namespace {

constexpr int kThreads = 256;

struct NArgs {
  const void* x;
  const void* res;
  void* res_out;
  const void* w;
  void* out;
  uint8_t* scales;
  int rows, cols;
  int64_t ld_x, ld_res, ld_res_out, ld_out, ld_scales;
  float eps;
  bool w_f32;
  int64_t row0;      // first row of the launch
};

// Sum over the WAVES waves of a row, the same in every thread.  The threads'
// sums, of 8 to 64 terms in fp32, are joined in fp64: the join's roundings
// would be common to the whole row, and each flips the rounding of a few
// e4m3 results.
template <int WAVES>
__device__ __forceinline__ double row_sum(float v, double* sh) {
  double s = v;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m);
  if constexpr (WAVES > 1) {
    __syncthreads();   // the previous sum's reads are done
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = s;
    __syncthreads();
    s = sh[0];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) s += sh[i];
  }
  return s;
}

// 1 / sqrt(mean + eps), from the fp32 instruction's value and one step of
// Newton's method in fp64 (relative error 1.5 times the square of the first
// one's 1e-7); a mean past fp32's range gives 0.
__device__ __forceinline__ float rstd_of(double squares, int cols, float eps) {
  const double x = squares * (1.0 / cols) + eps;
  const double r = __builtin_amdgcn_rsqf(static_cast<float>(x));
  return r > 0.0 ? static_cast<float>(r * (1.5 - 0.5 * x * r * r)) : static_cast<float>(r);
}

__device__ __forceinline__ void load_weight(const NArgs& a, uint32_t j, float (&w)[8]) {
  if (a.w_f32) load8(reinterpret_cast<const float*>(a.w), j, a.cols, w);
  else load8(reinterpret_cast<const __bf16*>(a.w), j, a.cols, w);
}

template <typename T>
__device__ __forceinline__ float rounded(float v) {
  return static_cast<float>(static_cast<T>(v));
}

// Maximum over a group of 16 lanes (128 columns): rotations within the 16.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x128, 0xf, 0xf, true)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x124, 0xf, 0xf, true)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x122, 0xf, 0xf, true)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x121, 0xf, 0xf, true)));
  return v;
}

// 8 columns as they are in memory: 1 (bf16) or 2 (fp32) vectors of 16 bytes.
template <typename T>
struct Raw {
  u32x4 v[sizeof(T) / 2];
};

constexpr int kBufferFlags = 0x00020000;   // raw buffer, 32-bit data format
constexpr int kNontemporal = 2;            // buffer instruction cache policy

// A row of n columns.  Its range ends with the 16-byte vector that holds
// column n - 1 (ld is a multiple of 8, so that lies within the row's ld).
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void* base, int64_t row, int64_t ld, int n) {
  const T* p = reinterpret_cast<const T*>(base) + row * ld;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(p), (short)0,
                                           static_cast<int>((n * static_cast<int>(sizeof(T)) + 15) & ~15), kBufferFlags);
}

// Vector i of a row; zeros past its range.
template <typename T, bool NT>
__device__ __forceinline__ Raw<T> load_raw(__amdgpu_buffer_rsrc_t r, int i) {
  Raw<T> x;
#pragma unroll
  for (unsigned h = 0; h < sizeof(T) / 2; ++h)
    x.v[h] = __builtin_amdgcn_raw_buffer_load_b128(r, i * 8 * static_cast<int>(sizeof(T)) + 16 * h, 0, NT ? kNontemporal : 0);
  return x;
}

// Keeps a vector as it is in memory across a use: without it the compiler
// holds the widened values instead, which take twice the registers (or more)
// and spill.
template <typename T>
__device__ __forceinline__ void keep_raw(Raw<T>& x) {
#pragma unroll
  for (unsigned h = 0; h < sizeof(T) / 2; ++h) asm volatile("" : "+v"(x.v[h]));
}

// In float; columns from n on (of a row whose width is no multiple of 8) are
// zero, whatever lies there.
template <typename T>
__device__ __forceinline__ void widen(const Raw<T>& x, int j, int n, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_bit_cast(f32x4, x.v[e / 4])[e % 4];
  } else {
    const bf16x8 b = __builtin_bit_cast(bf16x8, x.v[0]);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = static_cast<float>(b[e]);
  }
  if (n & 7) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = j + e < n ? v[e] : 0.0f;
  }
}

template <typename TX>
__device__ __forceinline__ void load_sum(const NArgs& a, int64_t row, uint32_t j, float (&v)[8]) {
  load8(reinterpret_cast<const TX*>(a.x) + row * a.ld_x, j, a.cols, v);
  if (a.res) {
    float r[8];
    load8(reinterpret_cast<const TX*>(a.res) + row * a.ld_res, j, a.cols, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = rounded<TX>(v[e] + r[e]);
  }
}

// What follows the norm of vector i (all 16 lanes of its block of 128
// columns): the product with the weight and the store, in TO or in e4m3.
template <typename TO>
__device__ __forceinline__ void finish(const NArgs& a, int64_t row, int i, const float (&v)[8], const float (&w)[8],
                                       float rstd) {
  const uint32_t j = 8u * i;
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = v[e] * rstd * w[e];
  if constexpr (sizeof(TO) == 1) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, before(j + e, a.cols) ? magnitude(y[e]) : 0u);
    const uint32_t s = scale_of(max16(top));
    const float inv = inverse_of(s);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= inv;
    if (before(j, a.cols)) {
      store8_e4m3(reinterpret_cast<uint8_t*>(a.out) + row * a.ld_out, j, a.cols, y);
      if (i % 16 == 0) a.scales[row * a.ld_scales + i / 16] = static_cast<uint8_t>(s);
    }
  } else {
    if (before(j, a.cols)) store8(reinterpret_cast<TO*>(a.out) + row * a.ld_out, j, a.cols, y);
  }
}

// The row in registers: one pass over the data, bound by HBM (8192 x 12288
// bf16 with residual and e4m3 output: 118 us, 6.0 TB/s; two passes took 169).
// A row has 256 / RPW threads with NV vectors each; all its loads (and the
// weight's) are in flight before the first is used.
template <typename TX, typename TW, typename TO, int RPW, int NV>
__global__ __launch_bounds__(kThreads) void rmsnorm_kernel(NArgs a) {
  constexpr int TPR = kThreads / RPW;
  __shared__ double sh[kThreads / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = a.row0 + static_cast<int64_t>(blockIdx.x) * RPW + __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
  if (row >= a.rows) return;      // (rows of a workgroup only share it where each is one wave)
  const __amdgpu_buffer_rsrc_t rx = row_rsrc<TX>(a.x, row, a.ld_x, a.cols);
  const __amdgpu_buffer_rsrc_t rw = row_rsrc<TW>(a.w, 0, 0, a.cols);
  Raw<TX> x[NV], r[NV];
  Raw<TW> w[NV];
  // fp32 rows take two loads to a line, so the line is kept (1537 x 5005: 11.3
  // us against 15.8 with nontemporal loads); bf16 rows take one (8192 x 12288:
  // 118 us against 121 with plain loads).
  constexpr bool kNT = sizeof(TX) == 2;
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = load_raw<TX, kNT>(rx, t + i * TPR);
  if (a.res) {
    const __amdgpu_buffer_rsrc_t rr = row_rsrc<TX>(a.res, row, a.ld_res, a.cols);
#pragma unroll
    for (int i = 0; i < NV; ++i) r[i] = load_raw<TX, kNT>(rr, t + i * TPR);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) w[i] = load_raw<TW, false>(rw, t + i * TPR);
  float v[NV][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = 8 * (t + i * TPR);
    widen(x[i], j, a.cols, v[i]);
    if (a.res) {
      float u[8];
      widen(r[i], j, a.cols, u);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = rounded<TX>(v[i][e] + u[e]);
      if (a.res_out && j < a.cols)
        store8(reinterpret_cast<TX*>(a.res_out) + row * a.ld_res_out, j, a.cols, v[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += v[i][e] * v[i][e];
  }
  const float rstd = rstd_of(row_sum<TPR / 64>(ss, sh), a.cols, a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float u[8];
    widen(w[i], 8 * (t + i * TPR), a.cols, u);
    finish<TO>(a, row, t + i * TPR, v[i], u, rstd);
  }
}

// Narrow rows (per-head norms): TPR threads to a row, one vector each, so that
// a wave takes 64 / TPR rows, and a thread kRowsOfThread of them (400000 x 128
// bf16: 37 us, 5.5 TB/s; a wave per row took 109).  Their loads overlap in fp32;
// in bf16 (load8) other waves' work covers them.
constexpr int kRowsOfThread = 2;

// Sum over groups of TPR lanes, in fp64.
template <int TPR>
__device__ __forceinline__ double lane_sum(float v) {
  double s = v;
#pragma unroll
  for (int m = TPR / 2; m >= 1; m >>= 1) s += __shfl_xor(s, m);
  return s;
}

template <typename TX, typename TW, typename TO, int TPR>
__global__ __launch_bounds__(kThreads) void rmsnorm_narrow_kernel(NArgs a) {
  constexpr int RPW = kThreads / TPR, U = kRowsOfThread;
  const int t = threadIdx.x % TPR, j = 8 * t;
  const int64_t row0 = a.row0 + static_cast<int64_t>(blockIdx.x) * (RPW * U) + threadIdx.x / TPR;
  float v[U][8], r[U][8], w[8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + u * RPW;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[u][e] = r[u][e] = 0.0f;
    if (row < a.rows) {
      load8<TX, true>(reinterpret_cast<const TX*>(a.x) + row * a.ld_x, j, a.cols, v[u]);
      if (a.res) load8<TX, true>(reinterpret_cast<const TX*>(a.res) + row * a.ld_res, j, a.cols, r[u]);
    }
  }
  load8(reinterpret_cast<const TW*>(a.w), j, a.cols, w);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + u * RPW;
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (a.res) v[u][e] = rounded<TX>(v[u][e] + r[u][e]);
      ss += v[u][e] * v[u][e];
    }
    const float rstd = rstd_of(lane_sum<TPR>(ss), a.cols, a.eps);
    if (row < a.rows) {     // (the same for the 16 lanes of a scale)
      if (a.res_out && j < a.cols) store8(reinterpret_cast<TX*>(a.res_out) + row * a.ld_res_out, j, a.cols, v[u]);
      finish<TO>(a, row, t, v[u], w, rstd);
    }
  }
}

// Rows too wide for the registers: one workgroup per row, two passes over it
// (the second mostly from the caches).
template <typename TX, typename TO>
__global__ __launch_bounds__(kThreads) void rmsnorm_wide_kernel(NArgs a) {
  __shared__ double sh[kThreads / 64];
  const int tid = threadIdx.x;
  const int vectors = (a.cols + 7) >> 3;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float ss = 0.0f;
    for (int i = tid; i < vectors; i += kThreads) {
      float v[8];
      load_sum<TX>(a, row, 8 * i, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += v[e] * v[e];
      if (a.res_out) store8(reinterpret_cast<TX*>(a.res_out) + row * a.ld_res_out, 8 * i, a.cols, v);
    }
    const float rstd = rstd_of(row_sum<kThreads / 64>(ss, sh), a.cols, a.eps);
    for (int i0 = 0; i0 < vectors; i0 += kThreads) {   // (every lane: a scale's maximum needs its 16)
      float v[8], w[8];
      load_sum<TX>(a, row, 8u * (i0 + tid), v);
      load_weight(a, 8u * (i0 + tid), w);
      finish<TO>(a, row, i0 + tid, v, w, rstd);
    }
  }
}

// ---- backward ---------------------------------------------------------------
struct BArgs {
  const void* x;
  const void* w;
  const void* dout;
  const void* dres;
  void* dx;
  float* dw;
  float* rstd;      // workspace: [rows]
  float* part;      // workspace: [chunks, ld_part] partial sums of dw
  int rows, cols, chunks, ld_part;
  int64_t ld_x, ld_dout, ld_dres, ld_dx;
  float eps;
  bool w_f32;
};

// One pass over the data: x and dout of a row stay in registers between its
// two sums and its dx, and a thread keeps the sums of its columns of dw over
// the rows its workgroup takes (every gridDim.x-th group of RPW); they go to
// the workspace at the end, a line per group of threads, and column_sum_kernel
// adds the lines in their order.  Where the sum of squares passes fp32's range,
// 1 / root is 0 and so is n, but the sum of w dy x may pass it too: 0 times that
// is no mean, so the sum of w dy n is formed as it stands (0, or NaN where x is
// infinite).  Bound by HBM: 8192 x 12288 bf16 142 us, 5.7
// TB/s (two passes and a third for dw: 267; without the loads ahead: 171).
template <typename TX, typename TW, int THREADS, int RPW, int NV>
__global__ __launch_bounds__(THREADS) void rmsnorm_backward_kernel(BArgs a) {
  constexpr int TPR = THREADS / RPW;
  __shared__ double sh[THREADS / 64], sh2[THREADS / 64];
  const int sub = __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
  const int t = threadIdx.x % TPR;
  const __amdgpu_buffer_rsrc_t rw = row_rsrc<TW>(a.w, 0, 0, a.cols);
  Raw<TW> w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) w[i] = load_raw<TW, false>(rw, t + i * TPR);
  float dw[NV][8] = {};
  struct Row {
    Raw<TX> x[NV], d[NV], r[NV];
  };
  auto load = [&](Row& q, int64_t row) {
    const __amdgpu_buffer_rsrc_t rx = row_rsrc<TX>(a.x, row, a.ld_x, a.cols);
    const __amdgpu_buffer_rsrc_t rd = row_rsrc<TX>(a.dout, row, a.ld_dout, a.cols);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      q.x[i] = load_raw<TX, true>(rx, t + i * TPR);
      q.d[i] = load_raw<TX, true>(rd, t + i * TPR);
    }
    if (a.dres) {
      const __amdgpu_buffer_rsrc_t rr = row_rsrc<TX>(a.dres, row, a.ld_dres, a.cols);
#pragma unroll
      for (int i = 0; i < NV; ++i) q.r[i] = load_raw<TX, true>(rr, t + i * TPR);
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * RPW;
  int64_t row = static_cast<int64_t>(blockIdx.x) * RPW + sub;
  // The next row's loads are in flight during this row's sums, where there are
  // registers for them.
  constexpr bool kAhead = sizeof(TX) == 2 || NV < 3;
  Row next;
  if (kAhead && row < a.rows) load(next, row);
  for (; row < a.rows; row += step) {
    if (!kAhead) load(next, row);
    Row q = next;
    Raw<TX>(&x)[NV] = q.x;
    Raw<TX>(&d)[NV] = q.d;
    Raw<TX>(&r)[NV] = q.r;
    if (kAhead && row + step < a.rows) load(next, row + step);
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = 8 * (t + i * TPR);
      float v[8], g[8], u[8];
      widen(x[i], j, a.cols, v);
      widen(d[i], j, a.cols, g);
      widen(w[i], j, a.cols, u);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss += v[e] * v[e];
        dot += g[e] * u[e] * v[e];
      }
      keep_raw(x[i]);
      keep_raw(d[i]);
      keep_raw(w[i]);
      __builtin_amdgcn_sched_barrier(0);   // (one vector widened at a time)
    }
    const float rstd = rstd_of(row_sum<TPR / 64>(ss, sh), a.cols, a.eps);
    float mean = static_cast<float>(row_sum<TPR / 64>(dot, sh2) * (1.0 / a.cols)) * rstd;   // of w dy n
    if (rstd == 0.0f) {
      dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = 8 * (t + i * TPR);
        float v[8], g[8], u[8];
        widen(x[i], j, a.cols, v);
        widen(d[i], j, a.cols, g);
        widen(w[i], j, a.cols, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot += g[e] * u[e] * (v[e] * rstd);
        keep_raw(x[i]);
        keep_raw(d[i]);
        keep_raw(w[i]);
        __builtin_amdgcn_sched_barrier(0);
      }
      mean = static_cast<float>(row_sum<TPR / 64>(dot, sh2));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = 8 * (t + i * TPR);
      float v[8], g[8], u[8];
      widen(x[i], j, a.cols, v);
      widen(d[i], j, a.cols, g);
      widen(w[i], j, a.cols, u);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = v[e] * rstd;
        dw[i][e] += g[e] * n;
        u[e] = (g[e] * u[e] - n * mean) * rstd;
      }
      if (a.dres) {
        widen(r[i], j, a.cols, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] += g[e];
      }
      if (j < a.cols) store8(reinterpret_cast<TX*>(a.dx) + row * a.ld_dx, j, a.cols, u);
      keep_raw(w[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (!a.dw) return;
  float* p = a.part + (static_cast<int64_t>(blockIdx.x) * RPW + sub) * a.ld_part;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = 8 * (t + i * TPR);
    if (j >= a.cols) continue;      // (ld_part is a multiple of 8)
    *reinterpret_cast<f32x4*>(p + j) = f32x4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
    *reinterpret_cast<f32x4*>(p + j + 4) = f32x4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
  }
}

// Narrow rows: as rmsnorm_narrow_kernel; the workgroup's rows join their sums of
// dw through LDS, in order, to one line (400000 x 128 bf16: 61 us, 5.1 TB/s; a
// wave per row took 252).  The next row is loaded ahead of this one's sums: in
// fp32 the loads are in flight during them, in bf16 they are waited for at once.
template <typename TX, typename TW, int TPR>
__global__ __launch_bounds__(kThreads) void rmsnorm_backward_narrow_kernel(BArgs a) {
  constexpr int RPW = kThreads / TPR;
  __shared__ float sh[RPW][8 * TPR + 4];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR, j = 8 * t;
  struct Row {
    float x[8], d[8], r[8];
  };
  auto load = [&](Row& q, int64_t row) {
#pragma unroll
    for (int e = 0; e < 8; ++e) q.x[e] = q.d[e] = q.r[e] = 0.0f;
    if (row < a.rows) {
      load8<TX, true>(reinterpret_cast<const TX*>(a.x) + row * a.ld_x, j, a.cols, q.x);
      load8<TX, true>(reinterpret_cast<const TX*>(a.dout) + row * a.ld_dout, j, a.cols, q.d);
      if (a.dres) load8<TX, true>(reinterpret_cast<const TX*>(a.dres) + row * a.ld_dres, j, a.cols, q.r);
    }
  };
  float w[8], dw[8] = {};
  load8(reinterpret_cast<const TW*>(a.w), j, a.cols, w);
  const int64_t step = static_cast<int64_t>(gridDim.x) * RPW;
  int64_t row = static_cast<int64_t>(blockIdx.x) * RPW + sub;
  Row next;
  load(next, row);
  for (; row - sub < a.rows; row += step) {      // (the same for the workgroup)
    const Row q = next;
    load(next, row + step);
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ss += q.x[e] * q.x[e];
      dot += q.d[e] * w[e] * q.x[e];
    }
    const float rstd = rstd_of(lane_sum<TPR>(ss), a.cols, a.eps);
    float mean = static_cast<float>(lane_sum<TPR>(dot) * (1.0 / a.cols)) * rstd;   // of w dy n
    if (__any(rstd == 0.0f)) {      // (as above; the wave's other rows keep theirs)
      dot = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) dot += q.d[e] * w[e] * (q.x[e] * rstd);
      const float zero = static_cast<float>(lane_sum<TPR>(dot));
      if (rstd == 0.0f) mean = zero;
    }
    float g[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float n = q.x[e] * rstd;
      dw[e] += q.d[e] * n;
      g[e] = (q.d[e] * w[e] - n * mean) * rstd + q.r[e];
    }
    if (row < a.rows && j < a.cols) store8(reinterpret_cast<TX*>(a.dx) + row * a.ld_dx, j, a.cols, g);
  }
  if (!a.dw) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sh[sub][j + e] = dw[e];
  __syncthreads();
  const int c = threadIdx.x;
  if (c >= a.cols || c >= 8 * TPR) return;
  float s = sh[0][c];
  for (int i = 1; i < RPW; ++i) s += sh[i][c];
  a.part[static_cast<int64_t>(blockIdx.x) * a.ld_part + c] = s;
}

// Rows too wide for the registers: dx by two passes over each row, which also
// leave 1 / root in the workspace, and dw by a pass of its own (below).
template <typename TX>
__global__ __launch_bounds__(kThreads) void rmsnorm_backward_wide_kernel(BArgs a) {
  __shared__ double sh[kThreads / 64], sh2[kThreads / 64];
  const int tid = threadIdx.x;
  const int vectors = (a.cols + 7) >> 3;
  NArgs wa{};
  wa.w = a.w;
  wa.cols = a.cols;
  wa.w_f32 = a.w_f32;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const TX* x = reinterpret_cast<const TX*>(a.x) + row * a.ld_x;
    const TX* dy = reinterpret_cast<const TX*>(a.dout) + row * a.ld_dout;
    float ss = 0.0f, dot = 0.0f;
    for (int i = tid; i < vectors; i += kThreads) {
      float v[8], d[8], w[8];
      load8(x, 8 * i, a.cols, v);
      load8(dy, 8 * i, a.cols, d);
      load_weight(wa, 8 * i, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss += v[e] * v[e];
        dot += d[e] * w[e] * v[e];
      }
    }
    const float rstd = rstd_of(row_sum<kThreads / 64>(ss, sh), a.cols, a.eps);
    float mean = static_cast<float>(row_sum<kThreads / 64>(dot, sh2) * (1.0 / a.cols)) * rstd;
    if (rstd == 0.0f) {      // (as above)
      dot = 0.0f;
      for (int i = tid; i < vectors; i += kThreads) {
        float v[8], d[8], w[8];
        load8(x, 8 * i, a.cols, v);
        load8(dy, 8 * i, a.cols, d);
        load_weight(wa, 8 * i, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot += d[e] * w[e] * (v[e] * rstd);
      }
      mean = static_cast<float>(row_sum<kThreads / 64>(dot, sh2));
    }
    if (a.dw && tid == 0) a.rstd[row] = rstd;
    for (int i = tid; i < vectors; i += kThreads) {
      float v[8], d[8], w[8], g[8];
      load8(x, 8 * i, a.cols, v);
      load8(dy, 8 * i, a.cols, d);
      load_weight(wa, 8 * i, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = (d[e] * w[e] - v[e] * rstd * mean) * rstd;
      if (a.dres) {
        float r[8];
        load8(reinterpret_cast<const TX*>(a.dres) + row * a.ld_dres, 8 * i, a.cols, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] += r[e];
      }
      store8(reinterpret_cast<TX*>(a.dx) + row * a.ld_dx, 8 * i, a.cols, g);
    }
  }
}

// Partial sums of dw over a contiguous chunk of rows: 64 vectors of columns
// per workgroup, its 4 waves on every fourth row.
template <typename TX>
__global__ __launch_bounds__(kThreads) void rmsnorm_dweight_kernel(BArgs a) {
  __shared__ float sh[4][64 * 8 + 4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t j = (blockIdx.x * 64 + lane) * 8;
  const int64_t per = (a.rows + a.chunks - 1) / a.chunks;
  const int64_t r0 = blockIdx.y * per, r1 = min(r0 + per, static_cast<int64_t>(a.rows));
  float s[8] = {};
  if (before(j, a.cols)) {
    for (int64_t row = r0 + wave; row < r1; row += 4) {
      float v[8], d[8];
      load8(reinterpret_cast<const TX*>(a.x) + row * a.ld_x, j, a.cols, v);
      load8(reinterpret_cast<const TX*>(a.dout) + row * a.ld_dout, j, a.cols, d);
      const float rstd = a.rstd[row];
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += d[e] * (v[e] * rstd);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sh[wave][lane * 8 + e] = s[e];
  __syncthreads();
  if (wave == 0 && before(j, a.cols)) {
    float* p = a.part + static_cast<int64_t>(blockIdx.y) * a.ld_part + j;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (before(j + e, a.cols))
        p[e] = sh[0][lane * 8 + e] + sh[1][lane * 8 + e] + sh[2][lane * 8 + e] + sh[3][lane * 8 + e];
  }
}

// dw = the sum of the partial sums: 16 columns per workgroup of 16 x 16
// threads, each thread every 16th line, then the 16 of a column in order.
__global__ __launch_bounds__(kThreads) void column_sum_kernel(const float* part, int chunks, int ld_part,
                                                              float* dw, int cols) {
  __shared__ float sh[16][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int j = blockIdx.x * 16 + c;
  float s = 0.0f;
  if (j < cols) {
#pragma unroll 8
    for (int i = r; i < chunks; i += 16) s += part[static_cast<int64_t>(i) * ld_part + j];
  }
  sh[r][c] = s;
  __syncthreads();
  if (r != 0 || j >= cols) return;
  for (int i = 1; i < 16; ++i) s += sh[i][c];
  dw[j] = s;
}

// ---- quantisation -------------------------------------------------------------
struct QArgs {
  const void* x;
  uint8_t* q;
  uint8_t* scales;
  int rows, cols;
  int64_t ld_x, ld_q, ld_scales;
  int64_t block0;      // first block of the launch (128 x 128)
};

// Blocks of 1 x 128: 16 lanes per block.  TPR threads side by side take 8 TPR
// columns of kRowsEach rows in one pass, bound by HBM (8192 x 6144 bf16: 26 us,
// 5.8 TB/s).  A thread's loads overlap in fp32 only (load8).
constexpr int kRowsEach = 2;
template <typename TX, int TPR>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(QArgs a) {
  constexpr int RPW = kThreads / TPR;
  const int chunks = (a.cols + 8u * TPR - 1) / (8 * TPR);
  const int64_t total = (a.rows + int64_t{RPW} * kRowsEach - 1) / (RPW * kRowsEach) * chunks;
  for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {   // (more than once only in a grid of the most workgroups)
    const int group = static_cast<int>(b / chunks), chunk = static_cast<int>(b - static_cast<int64_t>(group) * chunks);
    const uint32_t j = chunk * 8u * TPR + 8 * (threadIdx.x % TPR);
    const int64_t row0 = static_cast<int64_t>(group) * RPW * kRowsEach + threadIdx.x / TPR;
    float v[kRowsEach][8];
#pragma unroll
    for (int u = 0; u < kRowsEach; ++u) {
      const int64_t row = row0 + u * RPW;
      if (row < a.rows) {
        load8<TX, true>(reinterpret_cast<const TX*>(a.x) + row * a.ld_x, j, a.cols, v[u]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] = 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsEach; ++u) {
      const int64_t row = row0 + u * RPW;
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, magnitude(v[u][e]));
      const uint32_t s = scale_of(max16(top));
      const float inv = inverse_of(s);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[u][e] *= inv;
      if (row < a.rows && before(j, a.cols)) {
        store8_e4m3(a.q + row * a.ld_q, j, a.cols, v[u]);
        if ((j & (kScaleCols - 1)) == 0) a.scales[row * a.ld_scales + j / kScaleCols] = static_cast<uint8_t>(s);
      }
    }
  }
}

// Blocks of 128 x 128: one workgroup per block, which it holds in registers
// (16 threads side by side, 8 rows each).  Plain loads: a weight that was just
// written is read from the last-level cache (4001 x 2056 fp32: 12 us against
// 15 with nontemporal ones).
template <typename TX>
__global__ __launch_bounds__(kThreads) void quantize_tiles_kernel(QArgs a) {
  __shared__ uint32_t sh[kThreads / 64];
  const int blocks = (a.cols + kScaleCols - 1u) / kScaleCols;
  const int64_t b = a.block0 + blockIdx.x, br = b / blocks;          // block row and column
  const int bc = static_cast<int>(b - br * blocks);
  const uint32_t j = bc * static_cast<uint32_t>(kScaleCols) + 8 * (threadIdx.x & 15);
  const int64_t row0 = br * 128 + (threadIdx.x >> 4);
  float v[8][8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int64_t row = row0 + 16 * u;
    if (row < a.rows) {
      load8(reinterpret_cast<const TX*>(a.x) + row * a.ld_x, j, a.cols, v[u]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[u][e] = 0.0f;
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, magnitude(v[u][e]));
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(top, m)));
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = top;
  __syncthreads();
  const uint32_t s = scale_of(max(max(sh[0], sh[1]), max(sh[2], sh[3])));
  const float inv = inverse_of(s);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int64_t row = row0 + 16 * u;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[u][e] *= inv;
    if (row < a.rows && before(j, a.cols)) store8_e4m3(a.q + row * a.ld_q, j, a.cols, v[u]);
  }
  if (threadIdx.x == 0) a.scales[br * a.ld_scales + bc] = static_cast<uint8_t>(s);
}

cce_status launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(CCE_EHIP, std::string(what) + " launch: " + hipGetErrorString(e));
  return CCE_OK;
}

// A launch has fewer than 2^32 threads: more rows than that take turns.
constexpr int64_t kMaxGrid = 1 << 22;
dim3 grid_for(int64_t workgroups) { return dim3(static_cast<unsigned>(std::min(workgroups, kMaxGrid))); }

// Widest row that the kernels keep in registers (two tensors of it in the
// backward pass; a fourth vector per thread spills there).
constexpr int64_t kMaxForwardCols = 16384, kMaxBackwardCols = 12288;

// Lines of partial sums of dw.  In registers: a line per row of a workgroup,
// two workgroups per compute unit, one for wide rows, whose registers leave
// room for no more (8192 x 12288: 149 us against 156 with two).  Wider: chunks
// of rows, enough for the GPU and few enough that the lines stay a small part
// of the traffic.
// Narrow: a line per workgroup of 16 or 8 rows, four per compute unit.
constexpr int64_t kMaxNarrowCols = 256;
int narrow_rows_per_group(int64_t cols) { return cols <= 128 ? 16 : 8; }
int64_t backward_groups(int64_t cols) { return cols > 4096 ? 256 : cols > kMaxNarrowCols ? 512 : 1024; }
int backward_rows_per_group(int64_t cols) { return cols <= 1024 ? 4 : 1; }
int dweight_lines(int64_t rows, int64_t cols) {
  if (cols <= kMaxNarrowCols) {
    const int rpw = narrow_rows_per_group(cols);
    return static_cast<int>(std::min(backward_groups(cols), (rows + rpw - 1) / rpw));
  }
  if (cols <= kMaxBackwardCols) {
    const int rpw = backward_rows_per_group(cols);
    return static_cast<int>(std::min(backward_groups(cols), (rows + rpw - 1) / rpw) * rpw);
  }
  return static_cast<int>(std::max<int64_t>(1, std::min({rows / 16, int64_t{64}})));
}

template <typename TX, typename TW, typename TO>
void launch_norm(NArgs a, hipStream_t s) {
  auto go = [&](auto rpw, auto nv) {
    constexpr int RPW = decltype(rpw)::value, NV = decltype(nv)::value;
    // (more than one launch from 2^22 workgroups on: a loop in the kernel made
    // all calls 6% slower)
    for (a.row0 = 0; a.row0 < a.rows; a.row0 += kMaxGrid * RPW)
      rmsnorm_kernel<TX, TW, TO, RPW, NV><<<grid_for((a.rows - a.row0 + RPW - 1) / RPW), kThreads, 0, s>>>(a);
  };
  auto narrow = [&](auto tpr) {
    constexpr int64_t TPR = decltype(tpr)::value, each = kThreads / TPR * kRowsOfThread;
    for (a.row0 = 0; a.row0 < a.rows; a.row0 += kMaxGrid * each)
      rmsnorm_narrow_kernel<TX, TW, TO, TPR><<<grid_for((a.rows - a.row0 + each - 1) / each), kThreads, 0, s>>>(a);
  };
  if (a.cols <= 128) return narrow(std::integral_constant<int, 16>{});
  if (a.cols <= kMaxNarrowCols) return narrow(std::integral_constant<int, 32>{});
  // A wave per row up to 1024 columns, a workgroup of four per row above.
  if (a.cols <= 512) go(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
  else if (a.cols <= 1024) go(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
  else if (a.cols <= 2048) go(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
  else if (a.cols <= 4096) go(std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{});
  else if (a.cols <= 6144) go(std::integral_constant<int, 1>{}, std::integral_constant<int, 3>{});
  else if (a.cols <= 8192) go(std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
  else if (a.cols <= 12288) go(std::integral_constant<int, 1>{}, std::integral_constant<int, 6>{});
  else if (a.cols <= kMaxForwardCols) go(std::integral_constant<int, 1>{}, std::integral_constant<int, 8>{});
  else rmsnorm_wide_kernel<TX, TO><<<grid_for(a.rows), kThreads, 0, s>>>(a);
}

template <typename TX, typename TO>
void launch_norm_w(const NArgs& a, hipStream_t s) {
  if (a.w_f32) launch_norm<TX, float, TO>(a, s);
  else launch_norm<TX, __bf16, TO>(a, s);
}

template <typename TX, typename TW>
void launch_backward(const BArgs& a, hipStream_t s) {
  auto go = [&](auto threads, auto rpw, auto nv) {
    constexpr int T = decltype(threads)::value, RPW = decltype(rpw)::value, NV = decltype(nv)::value;
    const int64_t groups = std::min<int64_t>(backward_groups(a.cols), (a.rows + RPW - 1) / RPW);
    rmsnorm_backward_kernel<TX, TW, T, RPW, NV><<<dim3(static_cast<unsigned>(groups)), T, 0, s>>>(a);
  };
  auto narrow = [&](auto tpr) {
    constexpr int TPR = decltype(tpr)::value;
    rmsnorm_backward_narrow_kernel<TX, TW, TPR>
        <<<dim3(static_cast<unsigned>(dweight_lines(a.rows, a.cols))), kThreads, 0, s>>>(a);
  };
  if (a.cols <= 128) return narrow(std::integral_constant<int, 16>{});
  if (a.cols <= kMaxNarrowCols) return narrow(std::integral_constant<int, 32>{});
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  using I4 = std::integral_constant<int, 4>;
  using T256 = std::integral_constant<int, 256>;
  using T512 = std::integral_constant<int, 512>;
  if (a.cols <= 512) go(T256{}, I4{}, I1{});
  else if (a.cols <= 1024) go(T256{}, I4{}, I2{});
  else if (a.cols <= 2048) go(T256{}, I1{}, I1{});
  else if (a.cols <= 4096) go(T512{}, I1{}, I1{});
  else if (a.cols <= 8192) go(T512{}, I1{}, I2{});
  else go(T512{}, I1{}, I3{});
}

}  // namespace

cce_status launch_rmsnorm(const NormLaunch& L, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  NArgs a{L.x, L.res, L.res_out, L.w, L.out, L.scales, static_cast<int>(L.rows), static_cast<int>(L.cols),
          L.ld_x, L.ld_res, L.ld_res_out, L.ld_out, L.ld_scales, L.eps, L.w_t == CCE_F32, 0};
  if (L.x_t == CCE_F32) {
    if (L.out_t == CCE_E4M3) launch_norm_w<float, e4m3>(a, s);
    else if (L.out_t == CCE_F32) launch_norm_w<float, float>(a, s);
    else launch_norm_w<float, __bf16>(a, s);
  } else {
    if (L.out_t == CCE_E4M3) launch_norm_w<__bf16, e4m3>(a, s);
    else if (L.out_t == CCE_F32) launch_norm_w<__bf16, float>(a, s);
    else launch_norm_w<__bf16, __bf16>(a, s);
  }
  return launched("rmsnorm");
}

// Workspace: [rows] floats (wide rows), then the lines of partial sums.
static int64_t rstd_bytes(int64_t rows, int64_t cols) {
  return cols <= kMaxBackwardCols ? 0 : (rows * 4 + 255) & ~int64_t{255};
}

size_t rmsnorm_backward_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  const int64_t ld = (cols + 7) & ~int64_t{7};
  return static_cast<size_t>(rstd_bytes(rows, cols) + dweight_lines(rows, cols) * ld * 4);
}

cce_status launch_rmsnorm_backward(const NormBackwardLaunch& L, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  BArgs a{};
  a.x = L.x; a.w = L.w; a.dout = L.dout; a.dres = L.dres; a.dx = L.dx; a.dw = L.dw;
  a.rows = static_cast<int>(L.rows);
  a.cols = static_cast<int>(L.cols);
  a.chunks = L.rows > 0 ? dweight_lines(L.rows, L.cols) : 0;
  a.ld_part = static_cast<int>((L.cols + 7) & ~int64_t{7});
  a.rstd = reinterpret_cast<float*>(L.workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(L.workspace) + rstd_bytes(L.rows, L.cols));
  a.ld_x = L.ld_x; a.ld_dout = L.ld_dout; a.ld_dres = L.ld_dres; a.ld_dx = L.ld_dx;
  a.eps = L.eps;
  a.w_f32 = L.w_t == CCE_F32;
  const bool xf = L.x_t == CCE_F32, wide = L.cols > kMaxBackwardCols;
  if (L.rows > 0) {
    if (wide) {
      if (xf) rmsnorm_backward_wide_kernel<float><<<grid_for(a.rows), kThreads, 0, s>>>(a);
      else rmsnorm_backward_wide_kernel<__bf16><<<grid_for(a.rows), kThreads, 0, s>>>(a);
    } else if (xf) {
      if (a.w_f32) launch_backward<float, float>(a, s);
      else launch_backward<float, __bf16>(a, s);
    } else {
      if (a.w_f32) launch_backward<__bf16, float>(a, s);
      else launch_backward<__bf16, __bf16>(a, s);
    }
    if (const cce_status st = launched("rmsnorm backward"); st != CCE_OK) return st;
    if (wide && L.dw) {
      const dim3 grid(static_cast<unsigned>((L.cols + 511) / 512), static_cast<unsigned>(a.chunks));
      if (xf) rmsnorm_dweight_kernel<float><<<grid, kThreads, 0, s>>>(a);
      else rmsnorm_dweight_kernel<__bf16><<<grid, kThreads, 0, s>>>(a);
      if (const cce_status st = launched("rmsnorm weight gradient"); st != CCE_OK) return st;
    }
  }
  if (!L.dw) return CCE_OK;
  for (int64_t c = 0; c < L.cols; c += 16 * kMaxGrid)
    column_sum_kernel<<<grid_for((L.cols - c + 15) / 16), kThreads, 0, s>>>(a.part + c, a.chunks, a.ld_part, a.dw + c,
                                                                           static_cast<int>(L.cols - c));
  return launched("rmsnorm weight gradient sum");
}

template <typename TX>
void launch_quantize(QArgs a, int block_rows, hipStream_t s) {
  if (block_rows == 128) {
    const int64_t blocks = ((a.cols + int64_t{127}) / 128) * ((a.rows + int64_t{127}) / 128);
    for (; a.block0 < blocks; a.block0 += kMaxGrid)
      quantize_tiles_kernel<TX><<<grid_for(blocks - a.block0), kThreads, 0, s>>>(a);
    return;
  }
  auto go = [&](auto tpr) {
    constexpr int64_t TPR = decltype(tpr)::value, rows = kThreads / TPR * kRowsEach;
    const int64_t groups = ((a.rows + rows - 1) / rows) * ((a.cols + 8 * TPR - 1) / (8 * TPR));
    quantize_rows_kernel<TX, TPR><<<grid_for(groups), kThreads, 0, s>>>(a);
  };
  // Threads side by side: no more than a row fills.
  if (a.cols <= 256) go(std::integral_constant<int, 16>{});
  else if (a.cols <= 1024) go(std::integral_constant<int, 64>{});
  else go(std::integral_constant<int, 256>{});
}

cce_status launch_quantize_blocks(const QuantizeLaunch& L, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  QArgs a{L.x, L.q, L.scales, static_cast<int>(L.rows), static_cast<int>(L.cols), L.ld_x, L.ld_q, L.ld_scales, 0};
  if (L.x_t == CCE_F32) launch_quantize<float>(a, L.block_rows, s);
  else launch_quantize<__bf16>(a, L.block_rows, s);
  return launched("quantize");
}

}  // namespace cce
