// Products of rows grouped by expert: row r of the row operands belongs to
// the expert e with offsets[e] <= r < offsets[e + 1].
//
//   forward  C[r, n]   = sum_k A[r, k] B_e[n, k]
//   dgrad    A[r, k]   = sum_n C[r, n] B_e[n, k]
//   wgrad    B_e[n, k] = sum over the expert's rows r of C[r, n] A[r, k]
//
// One kernel computes all three as Z[i, j] = sum_l X[i, l] Y[j, l] per expert,
// in bf16 with fp32 accumulation (v_mfma_f32_32x32x16_bf16).  An operand is
// stored either with l contiguous ("row" form: A, and B in the forward
// product) or with i or j contiguous ("column" form: B in dgrad, both
// operands in wgrad); nothing is transposed in memory.
//
// Staging.  Tiles of 64 l go from global memory to LDS directly (16 bytes per
// lane), two stages, as the grouped GEMM does it (gemm.hip): the loads of a
// stage are spread over the matrix instructions of the one before.
//   row form: LDS rows of 64 l (128 bytes), 16-byte chunks XOR-swizzled by the
//     row so that 32 rows read at one chunk spread over the banks; a lane's
//     fragment (8 consecutive l of one row) is one 16-byte read.
//   column form: LDS rows of one l (BM or BN elements).  A fragment is two
//     transposing reads (ds_read_b64_tr_b16): 16 lanes read 4 l x 16 columns
//     and each gets 4 l of its own column.  Chunk c of row l is kept at
//     c ^ swz_col(l), so that the 4 rows that 32 lanes read at 64 bytes each
//     fall on all 64 banks.
// Where l ends: chunks and rows past the end are out of the buffer's range
// and land as zeros; a last chunk that is partly past the end (row form, l
// not a multiple of 8) is zeroed in LDS, since what lies behind a row may be
// anything, NaN included.
//
// The offsets are read on the device: every workgroup finds its tile from
// them (a scan over the experts), so the host needs no count of any expert's
// rows and launches the most tiles there can be.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>
#include <type_traits>

#include "cce_internal.hpp"

namespace cce {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

constexpr int kBufferFlags = 0x00020000;   // raw buffer, 32-bit data format
constexpr uint32_t kOob = 0x40000000;      // past every buffer below
constexpr int kBL = 64;                    // l per tile
constexpr int kNW = 4;                     // waves (of a group)
constexpr int kRowWaves = 2;               // waves of a workgroup of ragged_rows_kernel,
constexpr int64_t kRowGroups = 2048;       // and the most workgroups (4 waves, 1024: 3% slower)
constexpr int kGroups = 4;                 // groups of waves where tiles are few

struct RArgs {
  const __bf16* x;
  const __bf16* y;
  void* z;
  const int64_t* offsets;
  int T;
  int experts, I, J, L;       // extents that do not depend on the expert
  int ldx, ldy, ldz;
  int64_t xe, ye, ze;         // strides from expert to expert
  int tiles_j;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  const int n = bytes <= 0 ? 0 : static_cast<int>(min((bytes + 15) & ~int64_t{15}, static_cast<int64_t>(kOob) - 256));
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, n, kBufferFlags);
}

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t voffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)lds, 16, voffset, 0, 0, 0);
}

// s_waitcnt vmcnt(0), the other counters left alone.
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }

__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// Row number i of the offsets, within [0, T].  (Callers take the running
// maximum, so that no row has two experts, whatever the offsets hold.)
__device__ __forceinline__ int row_number(const RArgs& a, int i) {
  const int64_t v = a.offsets[i];
  return v < 0 ? 0 : v > a.T ? a.T : static_cast<int>(v);
}

__device__ __forceinline__ int wave_max(int v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = max(v, __shfl_xor(v, m));
  return v;
}

struct Tile {
  int e, lo, hi;    // expert and its rows
  int ti, tj;
};

// Tile rows of a tile height, from the experts' rows: calls f(first tile row,
// tile rows, expert, lo, hi) for the lane's expert of every group of 64.
// Returns the number of all tile rows.
template <int BM, typename F>
__device__ __forceinline__ int scan_experts(const RArgs& a, F&& f) {
  const int lane = threadIdx.x & 63;
  int before = row_number(a, 0), rows = 0;     // end of the rows, tile rows so far
  for (int e0 = 0; e0 < a.experts; e0 += 64) {
    const int e = e0 + lane;
    int hi = max(row_number(a, min(e, a.experts - 1) + 1), before);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(hi, d);
      if (lane >= d) hi = max(hi, o);
    }
    const int prev = __shfl_up(hi, 1);
    const int lo = lane == 0 ? before : prev;
    const int mine = e < a.experts ? (hi - lo + BM - 1) / BM : 0;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(sum, d);
      if (lane >= d) sum += o;
    }
    f(rows + sum - mine, mine, e, lo, hi);
    rows += __shfl(sum, 63);
    before = __shfl(hi, 63);
  }
  return rows;
}

// Tiles of the expert's rows (forward, dgrad).  Workgroups are dealt to the 8
// XCDs in turn: each XCD gets a contiguous range of the tiles there are, and
// walks an expert's tiles in bands of 4 tile rows, so that the tiles in
// flight share X and Y in the XCD's L2.  false: no tile for this workgroup.
template <int BM>
__device__ __forceinline__ bool find_row_tile(const RArgs& a, int64_t w, Tile& t) {
  // Of up to 64 experts the lanes keep what the scan saw; of more, a second
  // scan finds the tile's.
  int f = 0, n = 0, lo = 0, hi = 0;
  const int rows = __builtin_amdgcn_readfirstlane(scan_experts<BM>(a, [&](int f_, int n_, int, int l_, int h_) {
    f = f_;
    n = n_;
    lo = l_;
    hi = h_;
  }));
  const int64_t tiles = static_cast<int64_t>(rows) * a.tiles_j;
  const int64_t per = (tiles + 7) / 8;
  const int64_t id = (w & 7) * per + (w >> 3);
  if ((w >> 3) >= per || id >= tiles) return false;
  const int row = __builtin_amdgcn_readfirstlane(static_cast<int>(id / a.tiles_j));    // tile row
  int first = 0, mine = 0, e = 0, l = 0, h = 0;
  auto take = [&](int f_, int n_, int e_, int l_, int h_) {
    const uint64_t found = __ballot(f_ <= row && row < f_ + n_);
    if (found) {
      const int src = __ffsll(static_cast<unsigned long long>(found)) - 1;
      first = __shfl(f_, src);
      mine = __shfl(n_, src);
      e = __shfl(e_, src);
      l = __shfl(l_, src);
      h = __shfl(h_, src);
    }
  };
  if (a.experts <= 64) take(f, n, threadIdx.x & 63, lo, hi);
  else scan_experts<BM>(a, take);
  t.e = __builtin_amdgcn_readfirstlane(e);
  t.lo = __builtin_amdgcn_readfirstlane(l);
  t.hi = __builtin_amdgcn_readfirstlane(h);
  const int rem = static_cast<int>(id - static_cast<int64_t>(first) * a.tiles_j);
  constexpr int kBand = 4;
  const int band = rem / (kBand * a.tiles_j);
  const int in_band = rem - band * kBand * a.tiles_j;
  const int height = min(mine - band * kBand, kBand);
  t.ti = __builtin_amdgcn_readfirstlane(band * kBand + in_band % height);
  t.tj = __builtin_amdgcn_readfirstlane(in_band / height);
  return true;
}

// Tiles of the experts' matrices (wgrad), expert by expert: a tile's time goes
// by its expert's rows, so each XCD gets a contiguous eighth of every expert's
// tiles (an XCD with all of the largest expert's took twice the others' time).
// false: no tile for this workgroup.
template <int BM>
__device__ __forceinline__ bool find_matrix_tile(const RArgs& a, Tile& t) {
  const int tiles_i = (a.I + BM - 1) / BM, tiles = tiles_i * a.tiles_j, per = (tiles + 7) / 8;
  const int w = blockIdx.x;
  t.e = (w >> 3) / per;
  const int rem = (w & 7) * per + (w >> 3) - t.e * per;
  if (rem >= tiles) return false;
  constexpr int kBand = 4;
  const int band = rem / (kBand * a.tiles_j);
  const int in_band = rem - band * kBand * a.tiles_j;
  const int height = min(tiles_i - band * kBand, kBand);
  t.ti = band * kBand + in_band % height;
  t.tj = in_band / height;
  int lo = 0;
  for (int i = threadIdx.x & 63; i <= t.e; i += 64) lo = max(lo, row_number(a, i));
  lo = wave_max(lo);
  t.lo = __builtin_amdgcn_readfirstlane(lo);
  t.hi = __builtin_amdgcn_readfirstlane(max(lo, row_number(a, t.e + 1)));
  return true;
}

// A transposing read.  (The restrict pointer gives it alias information, as an
// ordinary load has by its type; without any the compiler takes it to depend
// on every load to LDS in flight and waits for them, 8 times a tile.)
__device__ __forceinline__ s16x4 tr_read(const __attribute__((address_space(3))) s16x4* __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(const_cast<lds_s16x4>(p));
}

// One operand's share of a tile: its loads and its fragments.  BT: rows of
// the tile (i or j); WT: rows of a wave; COL: the column form.
template <int BT, int WT, bool COL>
struct Operand {
  static constexpr int kChunks = COL ? BT / 8 : kBL / 8;      // 16-byte chunks per LDS row
  static constexpr int kRowBytes = kChunks * 16;
  static constexpr int kBytes = BT * kBL * 2;
  static constexpr int kRPI = 64 / kChunks;                   // LDS rows per load instruction
  static constexpr int kLoads = kBytes / (1024 * kNW);        // load instructions per wave
  static constexpr int kFrags = WT / 32;
  static_assert(!COL || kChunks >= 8, "the swizzle needs 8 chunks");

  // Column form: rows of 256 bytes or more start on the same bank, rows of
  // 128 on two by turns.
  __device__ static __forceinline__ int swz_col(int l) { return kChunks >= 16 ? (l & 3) << 2 : ((l >> 1) & 1) << 2; }

  const __bf16* base;      // (tile's first row, l = 0)
  int ld, rows, L;
  uint32_t off[kLoads];
  int chunk;               // of the lane's loads, row form
  int f0, fsw[4], ftr[4];  // fragment addresses

  __device__ __forceinline__ void init(const __bf16* b, int ld_, int rows_, int L_, int lane, int wave, int wt) {
    base = b;
    ld = ld_;
    rows = rows_;
    L = L_;
    const int r0 = lane / kChunks, c = lane % kChunks;
    chunk = COL ? 0 : c ^ swz(kRPI * wave + r0);    // (the swizzle of rows kRPI * kNW * p further is the same)
#pragma unroll
    for (int p = 0; p < kLoads; ++p) {
      const int r = kRPI * (kNW * p + wave) + r0;   // LDS row: i, or l
      off[p] = static_cast<uint32_t>(r) * ld * 2u + 16u * (COL ? c ^ swz_col(r) : chunk);
    }
    const int h = lane >> 5;
    if constexpr (COL) {
      // lane q of a group of 16 reads row q / 4, columns 4 (q % 4) .. + 3
      const int q = lane & 15, m = q >> 2;
      const int byte = 2 * (16 * ((lane >> 4) & 1) + 4 * (q & 3));       // in the wave's 32 columns
#pragma unroll
      for (int f = 0; f < kFrags; ++f) {
        const int cc = (wt * WT + 32 * f) / 8 + (byte >> 4);
        ftr[f] = (8 * h + m) * kRowBytes + ((cc ^ swz_col(m)) << 4) + (byte & 15);
      }
    } else {
      const int r = lane & 31;
      f0 = (wt * WT + r) * kRowBytes;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) fsw[kk] = ((2 * kk + h) ^ swz(r)) << 4;
    }
  }

  // Buffer of the tile at l0: rows past the end are out of its range.
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(int l0) const {
    if constexpr (COL) {
      const int n = min(L - l0, kBL);
      return make_rsrc(base + static_cast<int64_t>(l0) * ld,
                       n <= 0 ? 0 : (static_cast<int64_t>(n - 1) * ld + rows) * 2);
    } else {
      return make_rsrc(base, (static_cast<int64_t>(min(rows, BT) - 1) * ld + L) * 2);
    }
  }
  // What the tile at l0 adds to the lane's offsets.
  __device__ __forceinline__ uint32_t add(int l0) const {
    return COL ? 0u : l0 * 2u + (l0 + chunk * 8 < L ? 0u : kOob);
  }
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t add, int p, int wave) const {
    dma16(r, lds + (p * kNW + wave) * 1024, off[p] + add);
  }
  // Fragment f of l step kk (16 l): 8 l of the lane's row.
  __device__ __forceinline__ bf16x8 frag(const char* lds, int kk, int f) const {
    if constexpr (COL) {
      const char* p = lds + ftr[f] + kk * 16 * kRowBytes;
      const s16x4 lo = tr_read((lds_s16x4)(p));
      const s16x4 hi = tr_read((lds_s16x4)(p + 4 * kRowBytes));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(lds + f0 + fsw[kk] + f * 32 * kRowBytes));
    }
  }
  // Zeroes what a last chunk holds past the end of l (row form).
  __device__ __forceinline__ void zero_tail(char* lds, int l0) const {
    if constexpr (!COL) {
      const int l = L - l0;                      // in the tile: 0 < l < 64, l % 8 != 0
      for (int r = threadIdx.x & (64 * kNW - 1); r < BT; r += 64 * kNW) {
        __bf16* c = reinterpret_cast<__bf16*>(lds + r * kRowBytes + (((l >> 3) ^ swz(r)) << 4));
        for (int e = l & 7; e < 8; ++e) c[e] = static_cast<__bf16>(0.0f);
      }
    }
  }
};

// A tile's operands and result.
template <bool XC, bool YC, typename TOut>
struct TileArgs {
  int I, L;                  // rows (columns, wgrad) of the result, length of the sum
  const __bf16* x;
  const __bf16* y;
  TOut* z;                   // of the expert's first result row
  __device__ __forceinline__ TileArgs(const RArgs& a, const Tile& t, int i0, int j0) {
    I = XC ? a.I : t.hi - t.lo;
    L = XC ? t.hi - t.lo : a.L;
    x = a.x + t.e * a.xe + (XC ? static_cast<int64_t>(t.lo) * a.ldx + i0 : (static_cast<int64_t>(t.lo) + i0) * a.ldx);
    y = a.y + t.e * a.ye + (YC ? static_cast<int64_t>(XC ? t.lo : 0) * a.ldy + j0 : static_cast<int64_t>(j0) * a.ldy);
    z = reinterpret_cast<TOut*>(a.z) + t.e * a.ze + (XC ? 0 : static_cast<int64_t>(t.lo) * a.ldz);
  }
};

template <int BM, int BN, bool XC, bool YC, typename TOut>
__global__ __launch_bounds__(64 * kNW, 1) void ragged_kernel(RArgs a) {
  constexpr int WTM = BM / 2, WTN = BN / 2, FM = WTM / 32, FN = WTN / 32;
  using OX = Operand<BM, WTM, XC>;
  using OY = Operand<BN, WTN, YC>;
  constexpr int STAGE = OX::kBytes + OY::kBytes;
  constexpr int N_DMA = OX::kLoads + OY::kLoads;
  __shared__ __attribute__((aligned(16))) char smem[2 * STAGE];

  Tile t;
  if (!(XC ? find_matrix_tile<BM>(a, t) : find_row_tile<BM>(a, blockIdx.x, t))) return;
  const int i0 = t.ti * BM, j0 = t.tj * BN;
  const TileArgs<XC, YC, TOut> p(a, t, i0, j0);
  const int I = p.I, L = p.L;
  TOut* z = p.z;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  OX ox;
  OY oy;
  ox.init(p.x, a.ldx, I - i0, L, lane, wave, wm);
  oy.init(p.y, a.ldy, a.J - j0, L, lane, wave, wn);

  bf16x8 fx[2][FM], fy[2][FN];
  auto fread = [&](int buf, int kk, int slot, int q) {
    const char* s = smem + buf * STAGE;
    if (q < FN) fy[slot][q] = oy.frag(s + OX::kBytes, kk, q);
    else fx[slot][q - FN] = ox.frag(s, kk, q - FN);
  };
  f32x16 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = f32x16{};
  // Blocks in a snake order: consecutive instructions share an operand.
  auto mfma = [&](int slot, int q) {
    const int i = q / FM, j = (i & 1) ? FM - 1 - q % FM : q % FM;
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fy[slot][i], fx[slot][j], acc[i][j], 0, 0, 0);
  };

  const int KT = (L + kBL - 1) / kBL;
  const bool tail = (!XC || !YC) && (L & 7) != 0;
  auto load_all = [&](int buf, int l0) {
    const __amdgpu_buffer_rsrc_t rx = ox.rsrc(l0), ry = oy.rsrc(l0);
    const uint32_t ax = ox.add(l0), ay = oy.add(l0);
    char* s = smem + buf * STAGE;
#pragma unroll
    for (int p = 0; p < OX::kLoads; ++p) ox.load(rx, s, ax, p, wave);
#pragma unroll
    for (int p = 0; p < OY::kLoads; ++p) oy.load(ry, s + OX::kBytes, ay, p, wave);
  };
  auto mend_tail = [&](int buf, int kt) {
    if (tail && kt == KT - 1) {
      char* s = smem + buf * STAGE;
      ox.zero_tail(s, kt * kBL);
      oy.zero_tail(s + OX::kBytes, kt * kBL);
      __syncthreads();
    }
  };
  if (KT > 0) {
    load_all(0, 0);
    wait_loads();
    __syncthreads();
    mend_tail(0, 0);
#pragma unroll
    for (int q = 0; q < FM + FN; ++q) fread(0, 0, 0, q);
    load_all(1, kBL);
  }
  // Per tile: steps 0..2 read the next step's fragments between their matrix
  // instructions; then the next tile's loads are waited for, and the last
  // step reads its first fragments while the loads of the tile after it go
  // into this tile's buffer.
  constexpr int NMF = FM * FN;
  constexpr int RS = NMF >= 2 * (FM + FN) ? 2 : 1;
  for (int kt = 0; kt < KT; ++kt) {
    const int cur = kt & 1, nxt = cur ^ 1;
#pragma unroll
    for (int kk = 0; kk < 3; ++kk) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int q = 0; q < NMF; ++q) {
        mfma(kk & 1, q);
        if (q % RS == 0 && q / RS < FM + FN) fread(cur, kk + 1, (kk + 1) & 1, q / RS);
        if (NMF < FM + FN && q == NMF - 1) {
#pragma unroll
          for (int r = NMF; r < FM + FN; ++r) fread(cur, kk + 1, (kk + 1) & 1, r);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    wait_loads();
    __syncthreads();
    mend_tail(nxt, kt + 1);
    {
      const int l0 = (kt + 2) * kBL;
      const __amdgpu_buffer_rsrc_t rx = ox.rsrc(l0), ry = oy.rsrc(l0);
      const uint32_t ax = ox.add(l0), ay = oy.add(l0);
      char* s = smem + cur * STAGE;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int q = 0; q < NMF; ++q) {
        mfma(1, q);
        if (q % RS == 0 && q / RS < FM + FN) fread(nxt, 0, 0, q / RS);
        if (NMF < FM + FN && q == NMF - 1) {
#pragma unroll
          for (int r = NMF; r < FM + FN; ++r) fread(nxt, 0, 0, r);
        }
#pragma unroll
        for (int d = 0; d < N_DMA; ++d)
          if (d * NMF / N_DMA == q) {
            if (d < OX::kLoads) ox.load(rx, s, ax, d, wave);
            else oy.load(ry, s + OX::kBytes, ay, d - OX::kLoads, wave);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  wait_loads();       // (loads past the end, which land as zeros)
  __syncthreads();    // every wave's fragment reads are done

  // The result passes through LDS, so that whole rows are stored: a block of
  // the accumulators holds Z^T, 4 consecutive columns of one row per lane and
  // register quad.  A tile that does not fit goes in EP passes of EJP blocks
  // per wave.
  constexpr int ESZ = static_cast<int>(sizeof(TOut));
  constexpr int ERB = BN * ESZ, ECR = ERB / 16, EPC = 16 / ESZ;
  constexpr int EP = (BM * ERB + 2 * STAGE - 1) / (2 * STAGE);
  constexpr int EJP = FM / EP, EPR = BM / EP, ERI = 64 * kNW / ECR, EIT = EPR / ERI;
  constexpr int ESW = ECR < 32 ? ECR - 1 : 31;
  static_assert(FM % EP == 0 && EPR * ERB <= 2 * STAGE && 32 % ERI == 0, "staged store shape");
  const int e_r = tid / ECR, e_c = tid % ECR;
  const bool whole = i0 + BM <= I && j0 + BN <= a.J;
#pragma unroll
  for (int pass = 0; pass < EP; ++pass) {
    if (pass > 0) __syncthreads();
#pragma unroll
    for (int jj = 0; jj < EJP; ++jj) {
      const int j = pass * EJP + jj;
      const int lr = wm * 32 * EJP + jj * 32 + (lane & 31);
      char* srow = smem + lr * ERB;
#pragma unroll
      for (int i = 0; i < FN; ++i) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4 v = {acc[i][j][4 * q + 0], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          const int byte = (wn * WTN + 32 * i + 8 * q + 4 * (lane >> 5)) * ESZ;
          char* d = srow + (((byte >> 4) ^ (lr & ESW)) << 4) + (byte & 15);
          if constexpr (ESZ == 4) {
            *reinterpret_cast<f32x4*>(d) = v;
          } else {
            bf16x4 hv;
#pragma unroll
            for (int e = 0; e < 4; ++e) hv[e] = static_cast<__bf16>(v[e]);
            *reinterpret_cast<bf16x4*>(d) = hv;
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < EIT; ++it) {
      const int lr = ERI * it + e_r;
      const u32x4 raw = *reinterpret_cast<const u32x4*>(smem + lr * ERB + ((e_c ^ (lr & ESW)) << 4));
      const int i = i0 + ((ERI * it) / (32 * EJP)) * WTM + 32 * (pass * EJP + ((ERI * it) / 32) % EJP) + (ERI * it) % 32 + e_r;
      const int j = j0 + EPC * e_c;
      TOut* dst = z + static_cast<int64_t>(i) * a.ldz + j;
      if (whole || (i < I && j + EPC <= a.J)) {
        __builtin_nontemporal_store(raw, reinterpret_cast<u32x4*>(dst));
      } else if (i < I) {
        const TOut* src = reinterpret_cast<const TOut*>(&raw);
#pragma unroll
        for (int e = 0; e < EPC; ++e)
          if (j + e < a.J) dst[e] = src[e];
      }
    }
  }
}

// Small products: BM x BN tiles with NS stages, more workgroups per compute
// unit: the loads of the tile NS - 1 further go out behind a tile's barrier, into
// the buffer that every wave has left.  (The barrier as compiled waits for all
// loads in flight, so they have one tile's time.)  With few tiles and a long l, G groups of 4 waves each take every G-th
// tile of l with stages of their own, and join their sums through LDS in the
// order of the groups.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// 4 consecutive columns from j on of a row of J.
template <typename TOut>
__device__ __forceinline__ void store4(TOut* row, int j, int J, f32x4 v) {
  if (j + 4 <= J) {       // (aligned: ld is a multiple of 8)
    if constexpr (sizeof(TOut) == 4) {
      *reinterpret_cast<f32x4*>(row + j) = v;
    } else {
      bf16x4 h;
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = static_cast<__bf16>(v[e]);
      *reinterpret_cast<bf16x4*>(row + j) = h;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < J) row[j + e] = static_cast<TOut>(v[e]);
  }
}

template <int BM, int BN, int NS, int G, bool XC, bool YC, typename TOut>
__global__ __launch_bounds__(64 * kNW * G) void ragged_small_kernel(RArgs a) {
  constexpr int WTM = BM / 2, WTN = BN / 2, FM = WTM / 32, FN = WTN / 32;
  using OX = Operand<BM, WTM, XC>;
  using OY = Operand<BN, WTN, YC>;
  constexpr int STAGE = OX::kBytes + OY::kBytes, N_DMA = OX::kLoads + OY::kLoads;
  __shared__ __attribute__((aligned(16))) char smem[G * NS * STAGE];
  Tile t;
  if (!(XC ? find_matrix_tile<BM>(a, t) : find_row_tile<BM>(a, blockIdx.x, t))) return;
  const int i0 = t.ti * BM, j0 = t.tj * BN;
  const TileArgs<XC, YC, TOut> p(a, t, i0, j0);
  const int tid = threadIdx.x & (64 * kNW - 1), lane = tid & 63;
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * kNW));
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  OX ox;
  OY oy;
  ox.init(p.x, a.ldx, p.I - i0, p.L, lane, wave, wm);
  oy.init(p.y, a.ldy, a.J - j0, p.L, lane, wave, wn);
  const int KT = (p.L + kBL - 1) / kBL;
  const bool tail = (!XC || !YC) && (p.L & 7) != 0;
  char* stages = smem + group * NS * STAGE;
  auto load = [&](int buf, int l0) {
    const __amdgpu_buffer_rsrc_t rx = ox.rsrc(l0), ry = oy.rsrc(l0);
    const uint32_t ax = ox.add(l0), ay = oy.add(l0);
    char* s = stages + buf * STAGE;
#pragma unroll
    for (int d = 0; d < OX::kLoads; ++d) ox.load(rx, s, ax, d, wave);
#pragma unroll
    for (int d = 0; d < OY::kLoads; ++d) oy.load(ry, s + OX::kBytes, ay, d, wave);
  };
  f32x16 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = f32x16{};
  // (every group goes as many rounds: a tile past the end is zeros)
  if (KT > 0) {
#pragma unroll
    for (int d = 0; d < NS - 1; ++d) load(d, (group + d * G) * kBL);
  }
  int cur = 0;
  for (int k0 = 0; k0 < KT; k0 += G) {
    const int kt = k0 + group;
    wait_vmcnt<(NS - 2) * N_DMA>();
    __syncthreads();
    char* s = stages + cur * STAGE;
    if (tail && k0 + G >= KT) {
      if (kt == KT - 1) {
        ox.zero_tail(s, kt * kBL);
        oy.zero_tail(s + OX::kBytes, kt * kBL);
      }
      __syncthreads();
    }
    load(cur == 0 ? NS - 1 : cur - 1, (kt + (NS - 1) * G) * kBL);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      bf16x8 fx[FM], fy[FN];
#pragma unroll
      for (int i = 0; i < FN; ++i) fy[i] = oy.frag(s + OX::kBytes, kk, i);
#pragma unroll
      for (int j = 0; j < FM; ++j) fx[j] = ox.frag(s, kk, j);
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fy[i], fx[j], acc[i][j], 0, 0, 0);
    }
    cur = cur + 1 == NS ? 0 : cur + 1;
  }
  wait_vmcnt<0>();    // (loads past the end, which land as zeros)
  if constexpr (G > 1) {
    static_assert(FM == 1 && FN == 1 && (G - 1) * 16 * 256 * 4 <= G * NS * STAGE, "join");
    f32x4* part = reinterpret_cast<f32x4*>(smem);
    __syncthreads();  // every wave has left the stages
    if (group > 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        part[((group - 1) * 4 + q) * 256 + tid] =
            f32x4{acc[0][0][4 * q], acc[0][0][4 * q + 1], acc[0][0][4 * q + 2], acc[0][0][4 * q + 3]};
    }
    __syncthreads();
    if (group > 0) return;
    for (int g = 1; g < G; ++g) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 v = part[((g - 1) * 4 + q) * 256 + tid];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][0][4 * q + e] += v[e];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int i = i0 + wm * WTM + 32 * j + (lane & 31);
    if (i >= p.I) continue;
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        store4(p.z + static_cast<int64_t>(i) * a.ldz, j0 + wn * WTN + 32 * n + 8 * q + 4 * (lane >> 5), a.J,
               f32x4{acc[n][j][4 * q], acc[n][j][4 * q + 1], acc[n][j][4 * q + 2], acc[n][j][4 * q + 3]});
  }
}

// A few rows per expert (forward): the time is that of reading the weights of
// the experts that have rows.  A workgroup takes 16 FM rows of an expert and
// 16 columns; its WAVES waves take every WAVES-th 64 of l, straight from
// memory to registers, DEPTH of them ahead, and join their sums through LDS in
// the order of the waves.  v_mfma_f32_16x16x32_bf16: lane l holds row l & 15
// and 8 l from 8 (l / 16) on.
template <int FM, int WAVES, typename TOut>
__global__ __launch_bounds__(64 * WAVES) void ragged_rows_kernel(RArgs a) {
  __shared__ f32x4 part[WAVES - 1][FM][64];
  // (a workgroup takes several tiles, and most tiles that there could be are not
  // there: a workgroup for each of those took 2 to 3 us of 17)
  Tile t;
  for (int64_t w = blockIdx.x; find_row_tile<16 * FM>(a, w, t); w += gridDim.x) {
    if (w != blockIdx.x) __syncthreads();   // the last tile's sums are read
    const int i0 = t.ti * 16 * FM, j0 = t.tj * 16;
    const TileArgs<false, false, TOut> p(a, t, i0, j0);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int KB = (p.L + 63) / 64;
    const int rows = min(p.I - i0, 16 * FM), cols = min(a.J - j0, 16);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x, (static_cast<int64_t>(rows - 1) * a.ldx + p.L) * 2);
    const __amdgpu_buffer_rsrc_t ry = make_rsrc(p.y, (static_cast<int64_t>(cols - 1) * a.ldy + p.L) * 2);
    uint32_t off_x[FM];
#pragma unroll
    for (int j = 0; j < FM; ++j) off_x[j] = 16 * j + r < rows ? static_cast<uint32_t>(16 * j + r) * a.ldx * 2u : kOob;
    const uint32_t off_y = r < cols ? static_cast<uint32_t>(r) * a.ldy * 2u : kOob;
    struct Block {
      u32x4 y[2], x[FM][2];
    };
    auto load = [&](Block& b, int kb) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int l = kb * 64 + 32 * c + 8 * g;
        const uint32_t add = l * 2u + (l < p.L ? 0u : kOob);
        b.y[c] = __builtin_amdgcn_raw_buffer_load_b128(ry, off_y + add, 0, 0);
#pragma unroll
        for (int j = 0; j < FM; ++j) b.x[j][c] = __builtin_amdgcn_raw_buffer_load_b128(rx, off_x[j] + add, 0, 0);
      }
    };
    f32x4 acc[FM];
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[j] = f32x4{};
    const bool tail = (p.L & 7) != 0;
    // (what the last vector of l holds past the end may be anything)
    auto clip = [&](u32x4 v, int l) {
      bf16x8 b = __builtin_bit_cast(bf16x8, v);
      if (tail) {
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = l + e < p.L ? b[e] : static_cast<__bf16>(0.0f);
      }
      return b;
    };
    auto use = [&](const Block& b, int kb) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int l = kb * 64 + 32 * c + 8 * g;
        const bf16x8 vy = clip(b.y[c], l);
#pragma unroll
        for (int j = 0; j < FM; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vy, clip(b.x[j][c], l), acc[j], 0, 0, 0);
      }
    };
    if (wave < KB) {
      constexpr int DEPTH = 4;
      Block b[DEPTH];
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        load(b[d], wave + d * WAVES);
        __builtin_amdgcn_sched_barrier(0);   // (in the loop's order, which its waits count on)
      }
      for (int kb = wave; kb < KB; kb += DEPTH * WAVES) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
          use(b[d], kb + d * WAVES);
          load(b[d], kb + (d + DEPTH) * WAVES);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    if (wave > 0) {
#pragma unroll
      for (int j = 0; j < FM; ++j) part[wave - 1][j][lane] = acc[j];
    }
    __syncthreads();
    if (wave > 0) continue;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
#pragma unroll
      for (int q = 0; q < WAVES - 1; ++q) acc[j] = acc[j] + part[q][j][lane];
      // the result block is C^T: the lane holds row r, columns 4 g .. + 3
      const int i = i0 + 16 * j + r;
      if (i < p.I) store4(p.z + static_cast<int64_t>(i) * a.ldz, j0 + 4 * g, a.J, acc[j]);
    }
  }
}

int64_t most_row_tiles(const RArgs& r, int64_t bm) { return r.T / bm + std::min<int64_t>(r.experts, r.T); }

// (a launch has fewer than 2^32 threads, of at most 256 each but for small grids)
constexpr int64_t kMaxGrid = 0xffffff;

// Workgroups for `groups` times `tiles_i` rows of tiles, eight per eight tiles.
hipError_t grid_of(RArgs& r, int64_t groups, int64_t tiles_i, int bn, dim3& grid) {
  r.tiles_j = (r.J + bn - 1) / bn;
  const int64_t tiles = (tiles_i * r.tiles_j + 7) / 8 * 8;
  if (tiles > kMaxGrid || groups * tiles > kMaxGrid) return hipErrorInvalidValue;
  grid = dim3(static_cast<unsigned>(groups * tiles));
  return hipSuccess;
}

template <int BM, int BN, bool XC, bool YC>
hipError_t launch_tiles(RArgs& r, bool f32, hipStream_t s) {
  dim3 grid;
  const int64_t tiles_i = XC ? (r.I + int64_t{BM} - 1) / BM : most_row_tiles(r, BM);
  if (const hipError_t e = grid_of(r, XC ? r.experts : 1, tiles_i, BN, grid); e != hipSuccess) return e;
  if constexpr (BM == 64) {
    // a tile or less per compute unit: four groups of waves each (gradients of
    // 4000 rows, 128 x 256: 33 -> 23 us; two groups with four stages 26)
    if (static_cast<int64_t>(grid.x) <= 256) {
      if (f32) ragged_small_kernel<BM, BN, 2, kGroups, XC, YC, float><<<grid, 64 * kNW * kGroups, 0, s>>>(r);
      else ragged_small_kernel<BM, BN, 2, kGroups, XC, YC, __bf16><<<grid, 64 * kNW * kGroups, 0, s>>>(r);
    } else {
      if (f32) ragged_small_kernel<BM, BN, 4, 1, XC, YC, float><<<grid, 64 * kNW, 0, s>>>(r);
      else ragged_small_kernel<BM, BN, 4, 1, XC, YC, __bf16><<<grid, 64 * kNW, 0, s>>>(r);
    }
  } else {
    if (f32) ragged_kernel<BM, BN, XC, YC, float><<<grid, 64 * kNW, 0, s>>>(r);
    else ragged_kernel<BM, BN, XC, YC, __bf16><<<grid, 64 * kNW, 0, s>>>(r);
  }
  return hipGetLastError();
}

template <int FM>
hipError_t launch_rows(RArgs& r, bool f32, hipStream_t s) {
  r.tiles_j = (r.J + 15) / 16;
  const int64_t tiles = (most_row_tiles(r, 16 * FM) * r.tiles_j + 7) / 8 * 8;
  const dim3 grid(static_cast<unsigned>(std::min(tiles, kRowGroups)));    // (each takes its tiles in turn)
  if (f32) ragged_rows_kernel<FM, kRowWaves, float><<<grid, 64 * kRowWaves, 0, s>>>(r);
  else ragged_rows_kernel<FM, kRowWaves, __bf16><<<grid, 64 * kRowWaves, 0, s>>>(r);
  return hipGetLastError();
}

// The largest tiles that there are enough of for the 256 compute units, and
// that the experts' rows fill.  The host does not know the offsets: it counts
// as if the experts were even, with half a tile row more for each (forward,
// dgrad).  256 x 256 tiles run at 1280 TFLOP/s (8192 rows, 8 even experts of
// 4096 x 4096), 128 x 128 at 890; of little over 256 of the large ones the
// second round is mostly idle (4096 rows, 4 experts: 179 us, 155 with the
// small ones), and of rows that do not fill them much is wasted (8000 rows, 64
// experts: 542 us against 492).
template <bool XC, bool YC>
hipError_t launch_form(RArgs& r, bool f32, hipStream_t s) {
  const int64_t rows = r.T / r.experts;      // of an expert
  auto tiles = [&](int64_t b) {
    return r.experts * (((XC ? r.I : rows) + b - 1) / b) * ((r.J + b - 1) / b);
  };
  if constexpr (!XC && !YC) {
    if (rows <= 4) return launch_rows<1>(r, f32, s);
  }
  const int64_t large = tiles(256) + (XC ? 0 : r.experts * ((r.J + int64_t{255}) / 256) / 2);
  if (large >= (XC ? 256 : 384) && (XC || rows >= 200)) return launch_tiles<256, 256, XC, YC>(r, f32, s);
  if (tiles(128) >= 128 && (XC || rows >= 48)) return launch_tiles<128, 128, XC, YC>(r, f32, s);
  return launch_tiles<64, 64, XC, YC>(r, f32, s);
}

}  // namespace

cce_status launch_ragged(const RaggedLaunch& L, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  RArgs r{};
  r.offsets = L.offsets;
  r.T = static_cast<int>(L.T);
  r.experts = L.experts;
  const __bf16* a = static_cast<const __bf16*>(L.a);
  const __bf16* b = static_cast<const __bf16*>(L.b);
  const __bf16* c = static_cast<const __bf16*>(L.c);
  const int N = static_cast<int>(L.N), K = static_cast<int>(L.K);
  const int lda = static_cast<int>(L.lda), ldb = static_cast<int>(L.ldb), ldc = static_cast<int>(L.ldc);
  const bool f32 = L.out_t == CCE_F32;
  hipError_t e;
  if (L.kind == RAGGED_FORWARD) {
    r.x = a; r.ldx = lda;
    r.y = b; r.ldy = ldb; r.ye = L.stride_b;
    r.z = L.c; r.ldz = ldc;
    r.J = N; r.L = K;
    e = launch_form<false, false>(r, f32, s);
  } else if (L.kind == RAGGED_DGRAD) {
    r.x = c; r.ldx = ldc;
    r.y = b; r.ldy = ldb; r.ye = L.stride_b;
    r.z = L.a; r.ldz = lda;
    r.J = K; r.L = N;
    e = launch_form<false, true>(r, f32, s);
  } else {
    r.x = c; r.ldx = ldc;
    r.y = a; r.ldy = lda;
    r.z = L.b; r.ldz = ldb; r.ze = L.stride_b;
    r.I = N; r.J = K;
    e = launch_form<true, true>(r, f32, s);
  }
  if (e == hipErrorInvalidValue) return fail(CCE_EUNSUPPORTED, "ragged GEMM: too many output tiles");
  if (e != hipSuccess) return fail(CCE_EHIP, std::string("ragged GEMM launch: ") + hipGetErrorString(e));
  return CCE_OK;
}

}  // namespace cce
