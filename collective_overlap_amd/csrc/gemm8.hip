// Product of two e4m3 matrices whose blocks of 128 carry power-of-two scales:
//
//   C[m, n] = sum_k (A[m, k] 2^(sa[m, k/128] - 127)) (B^T[n, k] 2^(sb[n/128, k/128] - 127))
//
// with fp32 accumulation and an optional GELU on the store.  Three kernels:
//
//   gemm8_kernel       bf16 results, many rows: the matrix cores' 8-bit
//                      instruction, which takes the scales as operands.
//   gemm8_wide_kernel  fp32 results: e4m3 widened to bf16 on the way to the
//                      matrix cores, because the 8-bit instruction's own sums
//                      of 64 products keep about 16 bits (measured: 1.5e-5
//                      of the result's norm against 1e-7).
//   gemm8_rows_kernel  few rows, and small products: bound by reading B once, or
//                      by one trip to memory; widened too.

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
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef const __attribute__((address_space(3))) uint8_t* lds_bytes;

constexpr int kBufferFlags = 0x00020000;   // raw buffer, 32-bit data format
constexpr uint32_t kOob = 0x40000000;      // past every buffer below
constexpr int kBK = 128;                   // bytes of the contraction per tile: one scale block

struct G8Args {
  const uint8_t* a;
  const uint8_t* b;
  const uint8_t* sa;
  const uint8_t* sb;
  void* c;
  int M, N, K, tiles_m, tiles_n;
  int lda, ldb, ldc, ld_sa, ld_sb;
  bool gelu;
  bool scale_words;     // both scale matrices' rows start on 4-byte words
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  const int n = static_cast<int>(min(bytes, static_cast<int64_t>(kOob) - 256));
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, n, kBufferFlags);
}
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t voffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)lds, 16, voffset, 0, 0, 0);
}
// s_waitcnt vmcnt(0), the other counters left alone.
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }

__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// A byte of LDS.  (The restrict pointer gives the read alias information, which
// a byte's type does not; without any the compiler takes it to depend on every
// load to LDS in flight and waits for them.)
__device__ __forceinline__ int read_byte(const __attribute__((address_space(3))) uint8_t* __restrict__ p) { return *p; }

// 8 e4m3 values times a power of two (a float's exponent, which is E8M0's own
// encoding; 255 gives NaN), as bf16.  Exact where the products are normal bf16
// numbers: a e4m3 value has 4 significant bits.
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

// The factors of a block of A's rows (FM of the lane's) and of a block of B,
// for `scaled`.  The two scales act as one, 2^e with e = sa + sb - 254, which
// goes to A, so that a scale that bf16 cannot hold does no harm where the other
// one brings the product back.  448 2^e fits bf16 up to e = 119.  Where one of
// the wave's rows has more, B takes 2^9: what A's values then overflow bf16
// with is past fp32 with the least of B's, 2^-9, too; and from e = 137 on, where
// A's factor would pass 2^127, 2^18 (A's least value is 2^-9 as well).
// The products are exact from e = -117 on, where A's values are normal (-108 or
// -99 beside such a row); below they lose bits to bf16's subnormals, and A's
// factor is 2^-127 at least.  A scale of 255 stands for NaN.
template <int FM>
__device__ __forceinline__ void block_factors(const int (&sa)[FM], int sb, float (&fa)[FM], float& fb) {
  bool nan[FM];
  int top = 0;
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    nan[j] = max(sa[j], sb) == 255;
    top = max(top, nan[j] ? 0 : sa[j] + sb);
  }
  int over = 0;
  if (__any(top > 254 + 119)) over = __any(top > 254 + 136) ? 18 : 9;
#pragma unroll
  for (int j = 0; j < FM; ++j)
    fa[j] = __builtin_bit_cast(float, (nan[j] ? 255 : min(max(sa[j] + sb - 127 - over, 0), 254)) << 23);
  fb = __builtin_bit_cast(float, (127 + over) << 23);
}

// Tile of a workgroup: each of the 8 XCDs (dealt workgroups in turn) gets a
// contiguous range of tiles, walked in bands of 4 tile rows, so that the
// tiles in flight share A and B rows in its L2.
__device__ __forceinline__ void find_tile(const G8Args& a, int& tm, int& tn) {
  const int w = blockIdx.x, per = gridDim.x / 8;
  const int t = w < per * 8 ? (w & 7) * per + (w >> 3) : w;
  constexpr int kBand = 4;
  const int band = t / (kBand * a.tiles_n);
  const int in_band = t - band * kBand * a.tiles_n;
  const int height = min(a.tiles_m - band * kBand, kBand);
  tm = band * kBand + in_band % height;
  tn = in_band / height;
}

// ---------------------------------------------------------------------------
// bf16 results on v_mfma_scale_f32_32x32x64_f8f6f4.
//
// The grouped GEMM's design (gemm.hip) at one byte per element: BM x BN x 128
// tiles, LDS rows of 128 bytes in XOR-swizzled 16-byte chunks, two stages
// filled by direct global-to-LDS loads, 4 waves of (BM/2) x (BN/2).  A tile
// of the contraction is exactly one block of scales: the instruction takes
// each lane's row scale as an operand, so the scales cost no arithmetic.  They
// are copied to LDS ahead, kPanel blocks at a time, and read from there a tile
// ahead: read from memory tile by tile, a byte of each of 256 rows, they took
// as many L2 requests as the operands and 19% of the time (8192 x 6144 x
// 12288: 575 us, 483 from LDS, 479 with none).  Per tile two steps of 64:
//   step 0: MFMA | fragment reads of step 1
//   wait for the next tile's loads, barrier
//   step 1: MFMA | fragment reads of the next tile | loads of the tile after
//           next into this tile's buffer
// ---------------------------------------------------------------------------
constexpr int kPanel = 124;   // (row stride of 31 words: 32 rows on 32 banks)

// Copies n blocks' scales from block kb0 on to the panel: BM rows of A's from
// row m0, then B_BLOCKS block rows of B's from column n0; a thread per row, in
// vectors where the rows are aligned to words.
template <int BM, int B_BLOCKS>
__device__ __forceinline__ void copy_scales(const G8Args& a, uint8_t* panel, int m0, int n0, int kb0, int n) {
  for (int row = threadIdx.x; row < BM + B_BLOCKS; row += 256) {
    const uint8_t* src =
        (row < BM ? a.sa + static_cast<int64_t>(min(m0 + row, a.M - 1)) * a.ld_sa
                  : a.sb + static_cast<int64_t>(min(n0 + 128 * (row - BM), a.N - 1) / 128) * a.ld_sb) + kb0;
    uint32_t* dst = reinterpret_cast<uint32_t*>(panel + row * kPanel);
    constexpr int kVec = kPanel / 16;
    int done = 0;
    if (a.scale_words) {
      u32x4 v[kVec];
#pragma unroll
      for (int c = 0; c < kVec; ++c)
        if (16 * c + 16 <= n) v[c] = *reinterpret_cast<const u32x4_a4*>(src + 16 * c);
#pragma unroll
      for (int c = 0; c < kVec; ++c)
        if (16 * c + 16 <= n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[4 * c + e] = v[c][e];
        }
      done = min(n, 16 * kVec) & ~15;
    }
#pragma unroll 8
    for (int k = done; k < n; ++k) reinterpret_cast<uint8_t*>(dst)[k] = src[k];
  }
  wait_loads();   // (here: the compiler would wait in the main loop instead)
}

template <int BM, int BN, bool GELU>
__global__ __launch_bounds__(256, 1) void gemm8_kernel(G8Args a) {
  constexpr int NW = 4, WTM = BM / 2, WTN = BN / 2, FM = WTM / 32, FN = WTN / 32;
  constexpr int A_BYTES = BM * kBK, STAGE = (BM + BN) * kBK;
  constexpr int A_DMA = BM / 32, B_DMA = BN / 32, N_DMA = A_DMA + B_DMA;   // 8 rows per instruction
  constexpr int B_BLOCKS = BN / 128;
  static_assert(WTN <= 128 && 128 % WTN == 0, "one scale of B per wave");
  __shared__ __attribute__((aligned(16))) char smem[2 * STAGE + (BM + B_BLOCKS) * kPanel];
  uint8_t* panel = reinterpret_cast<uint8_t*>(smem + 2 * STAGE);

  int tm, tn;
  find_tile(a, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const __amdgpu_buffer_rsrc_t ra =
      make_rsrc(a.a + static_cast<int64_t>(m0) * a.lda, static_cast<int64_t>(min(a.M - m0, BM) - 1) * a.lda + a.K);
  const __amdgpu_buffer_rsrc_t rb =
      make_rsrc(a.b + static_cast<int64_t>(n0) * a.ldb, static_cast<int64_t>(min(a.N - n0, BN) - 1) * a.ldb + a.K);

  // Loads: instruction p of wave w fills rows 8 (4 p + w) + lane / 8; rows
  // past the end are out of the buffer's range, chunks past K steered there.
  const int dl_row = 8 * wave + (lane >> 3);
  const int dl_chunk = (lane & 7) ^ swz(dl_row);
  const uint32_t off_a = static_cast<uint32_t>(dl_row) * a.lda + 16u * dl_chunk;
  const uint32_t off_b = static_cast<uint32_t>(dl_row) * a.ldb + 16u * dl_chunk;
  auto add_of = [&](int k0) { return k0 + (k0 + 16 * dl_chunk < a.K ? 0u : kOob); };
  auto load = [&](int buf, uint32_t add, int d) {
    char* s = smem + buf * STAGE + wave * 1024;
    if (d < A_DMA) dma16(ra, s + d * NW * 1024, off_a + add + 32u * d * a.lda);
    else dma16(rb, s + A_BYTES + (d - A_DMA) * NW * 1024, off_b + add + 32u * (d - A_DMA) * a.ldb);
  };

  // Fragments: row lane & 31 of a block, 32 bytes of the step's 64.
  const int r = lane & 31, h = lane >> 5;
  const int fa0 = (wm * WTM + r) * kBK, fb0 = A_BYTES + (wn * WTN + r) * kBK;
  int fsw[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) fsw[q] = ((4 * (q >> 1) + 2 * h + (q & 1)) ^ swz(r)) << 4;
  i32x8 fa[2][FM], fb[2][FN];
  // half f & 1 of fragment f / 2 of step kk: B blocks first
  auto fread = [&](int buf, int kk, int slot, int f) {
    const int q = f >> 1, e = f & 1;
    const char* s = smem + buf * STAGE + (q < FN ? fb0 + q * 32 * kBK : fa0 + (q - FN) * 32 * kBK);
    const u32x4 v = *reinterpret_cast<const u32x4*>(s + fsw[2 * kk + e]);
    i32x8& d = q < FN ? fb[slot][q] : fa[slot][q - FN];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[4 * e + i] = static_cast<int>(v[i]);
  };

  const int KT = (a.K + kBK - 1) / kBK;
  auto fill_panel = [&](int kb0) { copy_scales<BM, B_BLOCKS>(a, panel, m0, n0, kb0, min(KT - kb0, kPanel)); };
  const int pa0 = (wm * WTM + r) * kPanel, pb0 = (BM + wn * WTN / 128) * kPanel;
  int va[FM], vb = 0, na[FM], nb = 0;     // of this tile, of the next
  auto read_scales = [&](int k) {
#pragma unroll
    for (int j = 0; j < FM; ++j) na[j] = read_byte((lds_bytes)(panel + pa0 + 32 * j * kPanel + k));
    nb = read_byte((lds_bytes)(panel + pb0 + k));
  };
  auto next_scales = [&] {
#pragma unroll
    for (int j = 0; j < FM; ++j) va[j] = na[j];
    vb = nb;
  };

  f32x16 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = f32x16{};
  auto mfma = [&](int slot, int q) {
    const int i = q / FM, j = (i & 1) ? FM - 1 - q % FM : q % FM;
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[slot][i], fa[slot][j], acc[i][j], 0, 0, 0, vb, 0, va[j]);
  };

  constexpr int NMF = FM * FN, NRD = 2 * (FM + FN);
  if (KT > 0) {
#pragma unroll
    for (int d = 0; d < N_DMA; ++d) load(0, add_of(0), d);
    fill_panel(0);
    wait_loads();
    __syncthreads();
    read_scales(0);
    next_scales();
#pragma unroll
    for (int f = 0; f < NRD; ++f) fread(0, 0, 0, f);
#pragma unroll
    for (int d = 0; d < N_DMA; ++d) load(1, add_of(kBK), d);
  }
  int kp = 0;                   // block of the next tile in the panel
  for (int kt = 0; kt < KT; ++kt) {
    const int cur = kt & 1, nxt = cur ^ 1;
    if (++kp == kPanel) {       // (uniform)
      kp = 0;
      __syncthreads();          // every wave has read this tile's scales
      fill_panel(min(kt + 1, KT - 1));
      __syncthreads();
    }
    read_scales(kp);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < NMF; ++q) {
      mfma(0, q);
#pragma unroll
      for (int f = 0; f < NRD; ++f)
        if (f * NMF / NRD == q) fread(cur, 1, 1, f);
      __builtin_amdgcn_sched_barrier(0);
    }
    wait_loads();
    __syncthreads();
    const uint32_t add = add_of((kt + 2) * kBK);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < NMF; ++q) {
      mfma(1, q);
#pragma unroll
      for (int f = 0; f < NRD; ++f)
        if (f * NMF / NRD == q) fread(nxt, 0, 0, f);
#pragma unroll
      for (int d = 0; d < N_DMA; ++d)
        if (d * NMF / N_DMA == q) load(cur, add, d);
      __builtin_amdgcn_sched_barrier(0);
    }
    next_scales();
  }
  wait_loads();       // (loads past K, which land as zeros)
  __syncthreads();    // every wave's fragment reads are done

  // The result passes through LDS, so that whole rows are stored: a block of
  // the accumulators holds C^T, 4 consecutive columns of one row per lane and
  // register quad.
  constexpr int ERB = BN * 2, ECR = ERB / 16, ERI = 64 * NW / ECR, EIT = BM / ERI;
  constexpr int ESW = ECR < 32 ? ECR - 1 : 31;
  static_assert(BM * ERB <= 2 * STAGE && 32 % ERI == 0, "staged store");
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int lr = wm * WTM + 32 * j + r;
#pragma unroll
    for (int i = 0; i < FN; ++i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        bf16x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = acc[i][j][4 * q + e];
          if (GELU) x = gelu_exact(x);
          v[e] = static_cast<__bf16>(x);
        }
        const int byte = (wn * WTN + 32 * i + 8 * q + 4 * h) * 2;
        *reinterpret_cast<bf16x4*>(smem + lr * ERB + (((byte >> 4) ^ (lr & ESW)) << 4) + (byte & 15)) = v;
        __builtin_amdgcn_sched_barrier(0);   // (one quad at a time: all at once spill)
      }
    }
  }
  __syncthreads();
  const int e_r = tid / ECR, e_c = tid % ECR;
  const int n = n0 + 8 * e_c;
#pragma unroll
  for (int it = 0; it < EIT; ++it) {
    const int lr = ERI * it + e_r, m = m0 + lr;
    const u32x4 raw = *reinterpret_cast<const u32x4*>(smem + lr * ERB + ((e_c ^ (lr & ESW)) << 4));
    __bf16* dst = reinterpret_cast<__bf16*>(a.c) + static_cast<int64_t>(m) * a.ldc + n;
    if (m < a.M && n + 8 <= a.N) {
      __builtin_nontemporal_store(raw, reinterpret_cast<u32x4*>(dst));
    } else if (m < a.M) {
      const bf16x8 v = __builtin_bit_cast(bf16x8, raw);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < a.N) dst[e] = v[e];
    }
  }
}

// ---------------------------------------------------------------------------
// fp32 results, and products too small for the tiles above: e4m3 widened to
// bf16 between LDS and the matrix cores (v_mfma_f32_32x32x16_bf16), the scale
// with it.  BM x BN x 128 tiles in the LDS layout of gemm8_kernel, NS stages:
// the loads of tile kt + NS - 1 go out behind the barrier of tile kt, into the
// buffer that every wave has left.  (The barrier as compiled waits for all loads
// in flight, not for those of the tile alone: they have one tile's time.)  A
// lane's 16-byte chunk feeds two instructions (the order of the k among them is
// the same for both operands).
// ---------------------------------------------------------------------------
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

template <int BM, int BN, int NS, typename TOut>
__global__ __launch_bounds__(256) void gemm8_wide_kernel(G8Args a) {
  constexpr int NW = 4, WTM = BM / 2, WTN = BN / 2, FM = WTM / 32, FN = WTN / 32;
  constexpr int A_BYTES = BM * kBK, STAGE = (BM + BN) * kBK;
  constexpr int A_DMA = BM / 32, B_DMA = BN / 32, N_DMA = A_DMA + B_DMA;
  static_assert(BN <= 128, "one scale of B per workgroup");
  __shared__ __attribute__((aligned(16))) char smem[NS * STAGE + (BM + 1) * kPanel];
  uint8_t* panel = reinterpret_cast<uint8_t*>(smem + NS * STAGE);

  int tm, tn;
  find_tile(a, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const __amdgpu_buffer_rsrc_t ra =
      make_rsrc(a.a + static_cast<int64_t>(m0) * a.lda, static_cast<int64_t>(min(a.M - m0, BM) - 1) * a.lda + a.K);
  const __amdgpu_buffer_rsrc_t rb =
      make_rsrc(a.b + static_cast<int64_t>(n0) * a.ldb, static_cast<int64_t>(min(a.N - n0, BN) - 1) * a.ldb + a.K);
  const int dl_row = 8 * wave + (lane >> 3);
  const int dl_chunk = (lane & 7) ^ swz(dl_row);
  const uint32_t off_a = static_cast<uint32_t>(dl_row) * a.lda + 16u * dl_chunk;
  const uint32_t off_b = static_cast<uint32_t>(dl_row) * a.ldb + 16u * dl_chunk;
  auto load = [&](int buf, int k0) {
    const uint32_t add = k0 + (k0 + 16 * dl_chunk < a.K ? 0u : kOob);
    char* s = smem + buf * STAGE + wave * 1024;
#pragma unroll
    for (int d = 0; d < A_DMA; ++d) dma16(ra, s + d * NW * 1024, off_a + add + 32u * d * a.lda);
#pragma unroll
    for (int d = 0; d < B_DMA; ++d) dma16(rb, s + A_BYTES + d * NW * 1024, off_b + add + 32u * d * a.ldb);
  };
  const int KT = (a.K + kBK - 1) / kBK;
  auto fill_panel = [&](int kb0) { copy_scales<BM, 1>(a, panel, m0, n0, kb0, min(KT - kb0, kPanel)); };

  const int r = lane & 31, h = lane >> 5;
  const int fa0 = (wm * WTM + r) * kBK, fb0 = A_BYTES + (wn * WTN + r) * kBK;
  const int pa0 = (wm * WTM + r) * kPanel, pb0 = BM * kPanel;
  f32x16 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = f32x16{};

  if (KT > 0) {
    fill_panel(0);
#pragma unroll
    for (int d = 0; d < NS - 1; ++d) load(d, d * kBK);
  }
  int sa[FM], sb;
  auto read_scales = [&](int k) {
#pragma unroll
    for (int j = 0; j < FM; ++j) sa[j] = read_byte((lds_bytes)(panel + pa0 + 32 * j * kPanel + k));
    sb = read_byte((lds_bytes)(panel + pb0 + k));
  };
  float fa[FM], fb;             // of tile kt
  int cur = 0, kp = 0;          // buffer of tile kt, its block in the panel
  for (int kt = 0; kt < KT; ++kt) {
    wait_vmcnt<(NS - 2) * N_DMA>();
    if (kp == kPanel) {         // (uniform)
      kp = 0;
      __syncthreads();          // every wave has read its last scales
      fill_panel(kt);
    }
    __syncthreads();
    const int prv = cur == 0 ? NS - 1 : cur - 1;
    load(prv, (kt + NS - 1) * kBK);
    if (kp == 0) {              // (the others' factors were formed in the tile before)
      read_scales(0);
      block_factors(sa, sb, fa, fb);
    }
    read_scales(min(kp + 1, kPanel - 1));
    const char* s = smem + cur * STAGE;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = ((2 * q + h) ^ swz(r)) << 4;
      u32x4 xa[FM], xb[FN];
#pragma unroll
      for (int i = 0; i < FN; ++i) xb[i] = *reinterpret_cast<const u32x4*>(s + fb0 + 32 * i * kBK + c);
#pragma unroll
      for (int j = 0; j < FM; ++j) xa[j] = *reinterpret_cast<const u32x4*>(s + fa0 + 32 * j * kBK + c);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        bf16x8 vb[FN];
#pragma unroll
        for (int i = 0; i < FN; ++i) vb[i] = scaled(u32x2{xb[i][2 * e], xb[i][2 * e + 1]}, fb);
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          const bf16x8 va = scaled(u32x2{xa[j][2 * e], xa[j][2 * e + 1]}, fa[j]);
#pragma unroll
          for (int i = 0; i < FN; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vb[i], va, acc[i][j], 0, 0, 0);
        }
      }
    }
    block_factors(sa, sb, fa, fb);
    ++kp;
    cur = cur + 1 == NS ? 0 : cur + 1;
  }
  wait_loads();       // (loads past K, which land as zeros)
  // the result block is C^T: the lane holds row m, columns 8 q + 4 h + e
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int m = m0 + wm * WTM + 32 * j + r;
    if (m >= a.M) continue;
    TOut* c = reinterpret_cast<TOut*>(a.c) + static_cast<int64_t>(m) * a.ldc;
#pragma unroll
    for (int i = 0; i < FN; ++i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + wn * WTN + 32 * i + 8 * q + 4 * h;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = a.gelu ? gelu_for<TOut>(acc[i][j][4 * q + e]) : acc[i][j][4 * q + e];
        if (n + 4 <= a.N) {       // (16 or 8 bytes, aligned: ldc is a multiple of 8)
          if constexpr (sizeof(TOut) == 4) {
            *reinterpret_cast<f32x4*>(c + n) = f32x4{v[0], v[1], v[2], v[3]};
          } else {
            bf16x4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = static_cast<__bf16>(v[e]);
            *reinterpret_cast<bf16x4*>(c + n) = x;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < a.N) c[n + e] = static_cast<TOut>(v[e]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows, and small products: the time is that of reading B once, or of one
// trip to memory.  A workgroup takes 16 FM rows and 16 FN columns; its WAVES
// waves take every WAVES-th block of 128 of the contraction, straight from
// memory to registers, DEPTH blocks ahead, and join their sums through LDS in
// the order of the waves.  v_mfma_f32_16x16x32_bf16: lane l holds row l & 15
// and the 16-byte chunks l / 16 and l / 16 + 4 of a block, so a load
// instruction reads 64 consecutive bytes of 16 rows; each chunk feeds two
// instructions of 32 (which k go together is the same for both operands, so
// their order does not matter).
// ---------------------------------------------------------------------------
template <int FM, int FN, int WAVES, typename TOut>
__global__ __launch_bounds__(64 * WAVES) void gemm8_rows_kernel(G8Args a) {
  __shared__ f32x4 part[WAVES > 1 ? WAVES - 1 : 1][FM][FN][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int tm = blockIdx.x / a.tiles_n, tn = blockIdx.x - tm * a.tiles_n;
  const int m0 = tm * 16 * FM, n0 = tn * 16 * FN;
  const int KB = (a.K + 127) / 128;
  // Rows past the end and chunks past K are out of the buffers' range: zeros.
  const __amdgpu_buffer_rsrc_t rb =
      make_rsrc(a.b + static_cast<int64_t>(n0) * a.ldb, static_cast<int64_t>(min(a.N - n0, 16 * FN) - 1) * a.ldb + a.K);
  const __amdgpu_buffer_rsrc_t ra =
      make_rsrc(a.a + static_cast<int64_t>(m0) * a.lda, static_cast<int64_t>(min(a.M - m0, 16 * FM) - 1) * a.lda + a.K);
  const uint8_t* sb = a.sb + static_cast<int64_t>(n0 / 128) * a.ld_sb;
  const uint8_t* sa[FM];
  uint32_t off_a[FM], off_b[FN];
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int m = m0 + 16 * j + r;
    off_a[j] = m < a.M ? static_cast<uint32_t>(16 * j + r) * a.lda : kOob;
    sa[j] = a.sa + static_cast<int64_t>(min(m, a.M - 1)) * a.ld_sa;
  }
#pragma unroll
  for (int i = 0; i < FN; ++i) off_b[i] = n0 + 16 * i + r < a.N ? static_cast<uint32_t>(16 * i + r) * a.ldb : kOob;
  struct Block {
    u32x4 b[FN][2], a[FM][2];
    int sb, sa[FM];
  };
  auto load = [&](Block& x, int kb) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int k = kb * 128 + 64 * c + 16 * g;
      const uint32_t add = k + (k < a.K ? 0u : kOob);
#pragma unroll
      for (int i = 0; i < FN; ++i) x.b[i][c] = __builtin_amdgcn_raw_buffer_load_b128(rb, off_b[i] + add, 0, 0);
#pragma unroll
      for (int j = 0; j < FM; ++j) x.a[j][c] = __builtin_amdgcn_raw_buffer_load_b128(ra, off_a[j] + add, 0, 0);
    }
    // (a block past the end is zeros times the last scale: a scale of NaN
    // there has made the result NaN already)
    const int s = min(kb, KB - 1);
    x.sb = sb[s];
#pragma unroll
    for (int j = 0; j < FM; ++j) x.sa[j] = sa[j][s];
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int j = 0; j < FM; ++j)
#pragma unroll
    for (int i = 0; i < FN; ++i) acc[j][i] = f32x4{};
  auto use = [&](const Block& x) {
    float fa[FM], fb;
    block_factors(x.sa, x.sb, fa, fb);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        bf16x8 vb[FN];
#pragma unroll
        for (int i = 0; i < FN; ++i) vb[i] = scaled(u32x2{x.b[i][c][2 * e], x.b[i][c][2 * e + 1]}, fb);
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          const bf16x8 va = scaled(u32x2{x.a[j][c][2 * e], x.a[j][c][2 * e + 1]}, fa[j]);
#pragma unroll
          for (int i = 0; i < FN; ++i) acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb[i], va, acc[j][i], 0, 0, 0);
        }
      }
    }
  };
  if (wave < KB) {
    constexpr int DEPTH = FM + FN > 2 ? 2 : 4;      // blocks in flight per wave
    Block x[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      load(x[d], wave + d * WAVES);
      __builtin_amdgcn_sched_barrier(0);   // (in the loop's order, which its waits count on)
    }
    for (int kb = wave; kb < KB; kb += DEPTH * WAVES) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        use(x[d]);
        load(x[d], kb + (d + DEPTH) * WAVES);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int i = 0; i < FN; ++i) part[wave - 1][j][i][lane] = acc[j][i];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int m = m0 + 16 * j + r;
#pragma unroll
    for (int i = 0; i < FN; ++i) {
#pragma unroll
      for (int w = 0; w < WAVES - 1; ++w) acc[j][i] = acc[j][i] + part[w][j][i][lane];
      if (m >= a.M) continue;
      // the result block is C^T: the lane holds row r, columns 4 g + e
      TOut* c = reinterpret_cast<TOut*>(a.c) + static_cast<int64_t>(m) * a.ldc;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = n0 + 16 * i + 4 * g + e;
        const float v = a.gelu ? gelu_for<TOut>(acc[j][i][e]) : acc[j][i][e];
        if (n < a.N) c[n] = static_cast<TOut>(v);
      }
    }
  }
}

template <int FM, int FN, int WAVES>
void launch_rows(G8Args a, bool f32, hipStream_t s) {
  a.tiles_n = (a.N + 16 * FN - 1) / (16 * FN);
  const dim3 grid(static_cast<unsigned>((a.M + 16 * FM - 1) / (16 * FM)) * a.tiles_n);
  if (f32) gemm8_rows_kernel<FM, FN, WAVES, float><<<grid, 64 * WAVES, 0, s>>>(a);
  else gemm8_rows_kernel<FM, FN, WAVES, __bf16><<<grid, 64 * WAVES, 0, s>>>(a);
}

template <int BM, int BN>
void launch_tiles(G8Args a, hipStream_t s) {
  a.tiles_m = (a.M + BM - 1) / BM;
  a.tiles_n = (a.N + BN - 1) / BN;
  const dim3 grid(static_cast<unsigned>(a.tiles_m) * a.tiles_n);
  if (a.gelu) gemm8_kernel<BM, BN, true><<<grid, 256, 0, s>>>(a);
  else gemm8_kernel<BM, BN, false><<<grid, 256, 0, s>>>(a);
}

template <int BM, int BN, int NS>
void launch_wide(G8Args a, bool f32, hipStream_t s) {
  a.tiles_m = (a.M + BM - 1) / BM;
  a.tiles_n = (a.N + BN - 1) / BN;
  const dim3 grid(static_cast<unsigned>(a.tiles_m) * a.tiles_n);
  if (f32) gemm8_wide_kernel<BM, BN, NS, float><<<grid, 256, 0, s>>>(a);
  else gemm8_wide_kernel<BM, BN, NS, __bf16><<<grid, 256, 0, s>>>(a);
}

}  // namespace

cce_status launch_gemm8(const Gemm8Launch& L, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  G8Args a{L.a, L.b, L.sa, L.sb, L.c, static_cast<int>(L.M), static_cast<int>(L.N), static_cast<int>(L.K), 0, 0,
           static_cast<int>(L.lda), static_cast<int>(L.ldb), static_cast<int>(L.ldc), static_cast<int>(L.ld_sa),
           static_cast<int>(L.ld_sb), L.gelu,
           ((reinterpret_cast<uintptr_t>(L.sa) | reinterpret_cast<uintptr_t>(L.sb) | L.ld_sa | L.ld_sb) & 3) == 0};
  auto tiles = [&](int64_t b) { return ((L.M + b - 1) / b) * ((L.N + b - 1) / b); };
  // (128 x 128 are the smallest where there are many; a launch has fewer than 2^32 threads)
  if (tiles(128) > 0xffffff) return fail(CCE_EUNSUPPORTED, "block-scaled GEMM: too many output tiles");
  const bool f32 = L.out_t == CCE_F32;
  // Few rows, or so few 64 x 64 tiles that a tile's length in K is the time
  // (64 x 64 x 8192: 11 us against 27; 130 x 520 x 4096: 13 against 15).  Up to
  // 8 rows in 16 columns per workgroup, of two waves where the columns alone
  // fill the GPU (4 x 12288 x 6144: 15.5 us against 16.2 with four); more rows,
  // which A's own reading begins to cost, in 32 columns, or in 64 where there
  // are enough (16 x 12288 x 6144: 21.1 us in 16, 20.8 in 32, 17.2 in 64; 16 x
  // 5000 x 4096: 11.9, 9.3, 12.8; 16 x 4096 x 4096: 7.3, 9.2; 32 x 12288 x 6144:
  // 21.6 in 64, 24.5 in 64 x 64 tiles; 32 x 4096 x 4096: 12.7 in 32, 16.5).
  // Then the largest tiles that come close to one per compute unit; with fewer
  // than 96 of the 128 x 128 ones the deeper 64 x 64 ones are faster (1000 x
  // 1000 x 4096: 18 us against 22; 128 x 12288 x 4096, 96 tiles: 23 against 22).
  if (L.M <= 32 || tiles(64) <= 32) {
    const bool more = L.M > 8 && L.M <= 32;
    if (more && L.N > 8192 && L.M <= 16) launch_rows<1, 4, 2>(a, f32, s);
    else if (more && L.N > 8192) launch_rows<2, 4, 2>(a, f32, s);
    else if (more && L.N > 4096 && L.M <= 16) launch_rows<1, 2, 4>(a, f32, s);
    else if (more && L.N > 2048 && L.M > 16) launch_rows<2, 2, 4>(a, f32, s);
    else if (L.N > 4096) launch_rows<1, 1, 2>(a, f32, s);
    else launch_rows<1, 1, 4>(a, f32, s);
  } else if (!f32 && tiles(256) >= 256) {
    launch_tiles<256, 256>(a, s);
  } else if (!f32 && L.M > 64 && tiles(128) >= 96) {
    launch_tiles<128, 128>(a, s);
  } else if (tiles(128) >= 256) {
    launch_wide<128, 128, 2>(a, f32, s);
  } else {
    launch_wide<64, 64, 4>(a, f32, s);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(CCE_EHIP, std::string("block-scaled GEMM launch: ") + hipGetErrorString(e));
  return CCE_OK;
}

}  // namespace cce
