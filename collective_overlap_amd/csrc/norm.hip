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
// memory.  Every sum is in fp32; r, y and dx are rounded once, on their store.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

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
};

// Sum over the workgroup, the same in every thread.
__device__ __forceinline__ float block_sum(float v, float* sh) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  const int waves = blockDim.x >> 6;
  __syncthreads();   // the previous sum's reads are done
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = sh[0];
  for (int i = 1; i < waves; ++i) s += sh[i];
  return s;
}

__device__ __forceinline__ void load_weight(const NArgs& a, int j, float (&w)[8]) {
  if (a.w_f32) load8(reinterpret_cast<const float*>(a.w), j, a.cols, w);
  else load8(reinterpret_cast<const __bf16*>(a.w), j, a.cols, w);
}

template <typename T>
__device__ __forceinline__ float rounded(float v) {
  return static_cast<float>(static_cast<T>(v));
}

// Maximum over a group of 16 lanes (128 columns).
__device__ __forceinline__ uint32_t max16(uint32_t v) {
#pragma unroll
  for (int m = 8; m >= 1; m >>= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(v, m)));
  return v;
}

template <typename TX>
__device__ __forceinline__ void load_sum(const NArgs& a, int64_t row, int j, float (&v)[8]) {
  load8(reinterpret_cast<const TX*>(a.x) + row * a.ld_x, j, a.cols, v);
  if (a.res) {
    float r[8];
    load8(reinterpret_cast<const TX*>(a.res) + row * a.ld_res, j, a.cols, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = rounded<TX>(v[e] + r[e]);
  }
}

// One workgroup per row, two passes over it.
template <typename TX, typename TO>
__global__ __launch_bounds__(kThreads) void rmsnorm_kernel(NArgs a) {
  __shared__ float sh[kThreads / 64];
  const int tid = threadIdx.x;
  const int vectors = (a.cols + 7) >> 3;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float ss = 0.0f;
    for (int i = tid; i < vectors; i += kThreads) {
      float v[8];
      load_sum<TX>(a, row, 8 * i, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += v[e] * v[e];
      if (a.res_out)
        store8(reinterpret_cast<TX*>(a.res_out) + row * a.ld_res_out, 8 * i, a.cols, v);
    }
    ss = block_sum(ss, sh);
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.cols) + a.eps);
    for (int i0 = 0; i0 < vectors; i0 += kThreads) {   // (every lane: the scale's maximum needs them)
      const int i = i0 + tid;
      float v[8], w[8];
      if (i < vectors) {
        load_sum<TX>(a, row, 8 * i, v);
        load_weight(a, 8 * i, w);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = w[e] = 0.0f;
      }
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = v[e] * rstd * w[e];
      if constexpr (sizeof(TO) == 1) {
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, 8 * i + e < a.cols ? magnitude(y[e]) : 0u);
        const uint32_t s = scale_of(max16(top));
        const float inv = inverse_of(s);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= inv;
        if (i < vectors) {
          store8_e4m3(reinterpret_cast<uint8_t*>(a.out) + row * a.ld_out, 8 * i, a.cols, y);
          if (i % 16 == 0) a.scales[row * a.ld_scales + i / 16] = static_cast<uint8_t>(s);
        }
      } else {
        if (i < vectors) store8(reinterpret_cast<TO*>(a.out) + row * a.ld_out, 8 * i, a.cols, y);
      }
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

template <typename TX>
__global__ __launch_bounds__(kThreads) void rmsnorm_backward_rows_kernel(BArgs a) {
  __shared__ float sh[kThreads / 64];
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
    ss = block_sum(ss, sh);
    dot = block_sum(dot, sh);
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.cols) + a.eps);
    const float mean = dot * rstd / static_cast<float>(a.cols);   // mean of w dy n
    if (tid == 0) a.rstd[row] = rstd;
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
  const int j = (blockIdx.x * 64 + lane) * 8;
  const int64_t per = (a.rows + a.chunks - 1) / a.chunks;
  const int64_t r0 = blockIdx.y * per, r1 = min(r0 + per, static_cast<int64_t>(a.rows));
  float s[8] = {};
  if (j < a.cols) {
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
  if (wave == 0 && j < a.cols) {
    float* p = a.part + static_cast<int64_t>(blockIdx.y) * a.ld_part + j;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j + e < a.cols)
        p[e] = sh[0][lane * 8 + e] + sh[1][lane * 8 + e] + sh[2][lane * 8 + e] + sh[3][lane * 8 + e];
  }
}

// dw = the sum of the partial sums, in the order of the chunks.
__global__ __launch_bounds__(kThreads) void column_sum_kernel(const float* part, int chunks, int ld_part,
                                                              float* dw, int cols) {
  const int j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= cols) return;
  float s = 0.0f;
  for (int c = 0; c < chunks; ++c) s += part[static_cast<int64_t>(c) * ld_part + j];
  dw[j] = s;
}

// ---- quantisation -------------------------------------------------------------
struct QArgs {
  const void* x;
  uint8_t* q;
  uint8_t* scales;
  int rows, cols;
  int64_t ld_x, ld_q, ld_scales;
};

// Blocks of 1 x 128: 16 lanes per block.
template <typename TX>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(QArgs a) {
  const int blocks = (a.cols + kScaleCols - 1) / kScaleCols;
  const int64_t total = static_cast<int64_t>(a.rows) * blocks;
  const int lane16 = threadIdx.x & 15;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kThreads / 16);
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * (kThreads / 16) + (threadIdx.x >> 4); b < total;
       b += stride) {
    const int64_t row = b / blocks;
    const int c = static_cast<int>(b - row * blocks);
    const int j = c * kScaleCols + 8 * lane16;
    float v[8];
    load8(reinterpret_cast<const TX*>(a.x) + row * a.ld_x, j, a.cols, v);
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, magnitude(v[e]));
    const uint32_t s = scale_of(max16(top));
    const float inv = inverse_of(s);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= inv;
    store8_e4m3(a.q + row * a.ld_q, j, a.cols, v);
    if (lane16 == 0) a.scales[row * a.ld_scales + c] = static_cast<uint8_t>(s);
  }
}

// Blocks of 128 x 128: one workgroup per block, two passes over it.
template <typename TX>
__global__ __launch_bounds__(kThreads) void quantize_tiles_kernel(QArgs a) {
  __shared__ uint32_t sh[kThreads / 64];
  const int lane16 = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int blocks = (a.cols + kScaleCols - 1) / kScaleCols;
  const int64_t br = blockIdx.x / blocks;          // block row and column
  const int bc = static_cast<int>(blockIdx.x - br * blocks);
  const int j = bc * kScaleCols + 8 * lane16;
  const int64_t row0 = br * 128;
  uint32_t top = 0;
  for (int i = r; i < 128; i += 16) {
    if (row0 + i >= a.rows) break;
    float v[8];
    load8(reinterpret_cast<const TX*>(a.x) + (row0 + i) * a.ld_x, j, a.cols, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, magnitude(v[e]));
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(top, m)));
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = top;
  __syncthreads();
  const uint32_t s = scale_of(max(max(sh[0], sh[1]), max(sh[2], sh[3])));
  const float inv = inverse_of(s);
  for (int i = r; i < 128; i += 16) {
    if (row0 + i >= a.rows) break;
    float v[8];
    load8(reinterpret_cast<const TX*>(a.x) + (row0 + i) * a.ld_x, j, a.cols, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= inv;
    store8_e4m3(a.q + (row0 + i) * a.ld_q, j, a.cols, v);
  }
  if (threadIdx.x == 0) a.scales[br * a.ld_scales + bc] = static_cast<uint8_t>(s);
}

cce_status launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(CCE_EHIP, std::string(what) + " launch: " + hipGetErrorString(e));
  return CCE_OK;
}

constexpr int64_t kMaxRowGrid = 1 << 20;

// Chunks of rows whose sums of dw are kept apart: enough workgroups for the
// GPU, and few enough that the partial sums stay a small part of the traffic.
int dweight_chunks(int64_t rows, int64_t cols) {
  const int64_t wide = (cols + 511) / 512;
  return static_cast<int>(std::max<int64_t>(1, std::min({rows / 16, int64_t{2048} / wide, int64_t{256}})));
}

}  // namespace

cce_status launch_rmsnorm(const NormLaunch& L, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  NArgs a{L.x, L.res, L.res_out, L.w, L.out, L.scales, static_cast<int>(L.rows), static_cast<int>(L.cols),
          L.ld_x, L.ld_res, L.ld_res_out, L.ld_out, L.ld_scales, L.eps, L.w_t == CCE_F32};
  const dim3 grid(static_cast<unsigned>(std::min(L.rows, kMaxRowGrid)));
  if (L.x_t == CCE_F32) {
    if (L.out_t == CCE_E4M3) rmsnorm_kernel<float, e4m3><<<grid, kThreads, 0, s>>>(a);
    else if (L.out_t == CCE_F32) rmsnorm_kernel<float, float><<<grid, kThreads, 0, s>>>(a);
    else rmsnorm_kernel<float, __bf16><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (L.out_t == CCE_E4M3) rmsnorm_kernel<__bf16, e4m3><<<grid, kThreads, 0, s>>>(a);
    else if (L.out_t == CCE_F32) rmsnorm_kernel<__bf16, float><<<grid, kThreads, 0, s>>>(a);
    else rmsnorm_kernel<__bf16, __bf16><<<grid, kThreads, 0, s>>>(a);
  }
  return launched("rmsnorm");
}

size_t rmsnorm_backward_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  const int64_t ld = (cols + 7) & ~int64_t{7};
  return static_cast<size_t>(((rows * 4 + 255) & ~int64_t{255}) + dweight_chunks(rows, cols) * ld * 4);
}

cce_status launch_rmsnorm_backward(const NormBackwardLaunch& L, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  BArgs a{};
  a.x = L.x; a.w = L.w; a.dout = L.dout; a.dres = L.dres; a.dx = L.dx; a.dw = L.dw;
  a.rows = static_cast<int>(L.rows);
  a.cols = static_cast<int>(L.cols);
  a.chunks = dweight_chunks(L.rows, L.cols);
  a.ld_part = static_cast<int>((L.cols + 7) & ~int64_t{7});
  a.rstd = reinterpret_cast<float*>(L.workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(L.workspace) + ((L.rows * 4 + 255) & ~int64_t{255}));
  a.ld_x = L.ld_x; a.ld_dout = L.ld_dout; a.ld_dres = L.ld_dres; a.ld_dx = L.ld_dx;
  a.eps = L.eps;
  a.w_f32 = L.w_t == CCE_F32;
  const unsigned cols_grid = static_cast<unsigned>((L.cols + kThreads - 1) / kThreads);
  if (L.rows > 0) {
    const dim3 grid(static_cast<unsigned>(std::min(L.rows, kMaxRowGrid)));
    if (L.x_t == CCE_F32) rmsnorm_backward_rows_kernel<float><<<grid, kThreads, 0, s>>>(a);
    else rmsnorm_backward_rows_kernel<__bf16><<<grid, kThreads, 0, s>>>(a);
    if (const cce_status st = launched("rmsnorm backward"); st != CCE_OK) return st;
    if (!L.dw) return CCE_OK;
    const dim3 wgrid(static_cast<unsigned>((L.cols + 511) / 512), static_cast<unsigned>(a.chunks));
    if (L.x_t == CCE_F32) rmsnorm_dweight_kernel<float><<<wgrid, kThreads, 0, s>>>(a);
    else rmsnorm_dweight_kernel<__bf16><<<wgrid, kThreads, 0, s>>>(a);
    if (const cce_status st = launched("rmsnorm weight gradient"); st != CCE_OK) return st;
  } else {
    a.chunks = 0;
  }
  if (!L.dw) return CCE_OK;
  column_sum_kernel<<<dim3(cols_grid), kThreads, 0, s>>>(a.part, a.chunks, a.ld_part, a.dw, a.cols);
  return launched("rmsnorm weight gradient sum");
}

cce_status launch_quantize_blocks(const QuantizeLaunch& L, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  QArgs a{L.x, L.q, L.scales, static_cast<int>(L.rows), static_cast<int>(L.cols), L.ld_x, L.ld_q, L.ld_scales};
  const int64_t blocks = (L.cols + kScaleCols - 1) / kScaleCols;
  if (L.block_rows == 1) {
    const int64_t wgs = (L.rows * blocks + kThreads / 16 - 1) / (kThreads / 16);
    const dim3 grid(static_cast<unsigned>(std::min(wgs, kMaxRowGrid)));
    if (L.x_t == CCE_F32) quantize_rows_kernel<float><<<grid, kThreads, 0, s>>>(a);
    else quantize_rows_kernel<__bf16><<<grid, kThreads, 0, s>>>(a);
  } else {
    const dim3 grid(static_cast<unsigned>(blocks * ((L.rows + 127) / 128)));
    if (L.x_t == CCE_F32) quantize_tiles_kernel<float><<<grid, kThreads, 0, s>>>(a);
    else quantize_tiles_kernel<__bf16><<<grid, kThreads, 0, s>>>(a);
  }
  return launched("quantize");
}

}  // namespace cce
