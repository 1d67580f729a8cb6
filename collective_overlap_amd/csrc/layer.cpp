// C entry points of the operators around the einsums: the norm, the 8-bit
// quantisation and product, the products grouped by expert.  Arguments are
// validated here; nothing is enqueued unless all of them pass.

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <exception>
#include <initializer_list>
#include <string>

#include "abi_util.hpp"
#include "cce_internal.hpp"

namespace cce {
namespace {

// An operand's bytes, for the overlap check (no allocation unless it fails:
// these calls take a few microseconds on small inputs).
struct Span {
  const char* name;
  const void* p;
  int64_t bytes;
  bool writes;
};

cce_status check_spans(std::initializer_list<Span> spans) {
  for (const Span* i = spans.begin(); i != spans.end(); ++i) {
    if (i->bytes <= 0) continue;
    for (const Span* j = i + 1; j != spans.end(); ++j) {
      if (j->bytes <= 0 || (!i->writes && !j->writes)) continue;
      const uintptr_t a = reinterpret_cast<uintptr_t>(i->p), b = reinterpret_cast<uintptr_t>(j->p);
      if (a < b + static_cast<uintptr_t>(j->bytes) && b < a + static_cast<uintptr_t>(i->bytes))
        return fail(CCE_EINVAL, std::string(i->name) + " overlaps " + j->name);
    }
  }
  return CCE_OK;
}

// A matrix whose rows are 16-byte vectors: as check_mat, with a base pointer.
cce_status check_operand(const char* name, const void* p, const cce_mat& m, int64_t bytes) {
  CCE_TRY(check_mat(name, m));
  return check_ptr(name, p, bytes);
}

// A matrix of one-byte scales: any alignment and any ld that holds the row.
cce_status check_scales(const char* name, const void* p, const cce_mat& m) {
  if (m.ld < m.cols) return fail(CCE_EINVAL, std::string(name) + ": bad extents " + mat_str(m));
  if (m.ld > 0x7fffffff) return fail(CCE_EUNSUPPORTED, std::string(name) + ": extent exceeds 2^31");
  if (!p && m.rows > 0 && m.cols > 0) return fail(CCE_EINVAL, std::string(name) + ": NULL pointer");
  return CCE_OK;
}

cce_status check_eps(double eps) {
  if (!(eps >= FLT_MIN) || !(eps <= FLT_MAX))
    return fail(CCE_EINVAL, "eps must be a positive, normal fp32 number");
  return CCE_OK;
}

int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

// Tiles of a product are addressed by 32-bit offsets from their first row.
constexpr int64_t kMaxLd = int64_t{1} << 20;

constexpr int64_t kMaxRows = int64_t{1} << 30;
cce_status check_rows(const cce_mat& m) {
  if (m.rows > kMaxRows) return fail(CCE_EUNSUPPORTED, "more than 2^30 rows");
  return CCE_OK;
}

cce_status check_ld(const char* name, int64_t ld) {
  if (ld > kMaxLd) return fail(CCE_EUNSUPPORTED, std::string(name) + ": ld exceeds 2^20 elements");
  return CCE_OK;
}

// No C++ exception leaves a C entry point (a failed host allocation, as of an
// error text, is the only one that these can meet).
template <typename F>
cce_status guarded(F&& f) noexcept {
  try {
    clear_error();
    return f();
  } catch (const std::exception&) {
    return CCE_EHIP;
  }
}

struct RaggedArgs {
  cce_ctx* ctx;
  cce_dtype out_t;
  int n_experts;
  const int64_t* offsets;
  void* a;
  cce_mat a_shape;
  void* b;
  cce_mat b_shape;
  int64_t b_stride;
  void* c;
  cce_mat c_shape;
  uint32_t flags;
  cce_stream stream;
};

cce_status ragged(int kind, const RaggedArgs& g) {
  if (!g.ctx) return fail(CCE_EINVAL, "ctx is NULL");
  if (g.flags != 0) return fail(CCE_EINVAL, "flags must be 0");
  if (!dtype_ok(g.out_t)) return fail(CCE_EINVAL, "bad dtype");
  if (g.n_experts < 1) return fail(CCE_EINVAL, "n_experts < 1");
  if (g.n_experts > 65536) return fail(CCE_EUNSUPPORTED, "n_experts > 65536");
  const bool fwd = kind == RAGGED_FORWARD, dgrad = kind == RAGGED_DGRAD, wgrad = kind == RAGGED_WGRAD;
  const int64_t eo = esize(g.out_t);
  const int64_t as = span_bytes(g.a_shape, dgrad ? eo : 2), cs = span_bytes(g.c_shape, fwd ? eo : 2);
  const int64_t b1 = span_bytes(g.b_shape, wgrad ? eo : 2);
  CCE_TRY(check_operand("a", g.a, g.a_shape, as));
  CCE_TRY(check_operand("b", g.b, g.b_shape, b1));
  CCE_TRY(check_operand("c", g.c, g.c_shape, cs));
  CCE_TRY(check_rows(g.a_shape));
  CCE_TRY(check_ld("a", g.a_shape.ld));
  CCE_TRY(check_ld("b", g.b_shape.ld));
  CCE_TRY(check_ld("c", g.c_shape.ld));
  if (g.a_shape.rows != g.c_shape.rows) return fail(CCE_EINVAL, "a and c must have the same rows");
  if (g.b_shape.rows != g.c_shape.cols || g.b_shape.cols != g.a_shape.cols)
    return fail(CCE_EINVAL, "each expert's b must be [c cols, a cols]");
  if (g.b_stride % 8 != 0) return fail(CCE_EUNSUPPORTED, "b_stride must be a multiple of 8");
  if (g.b_stride < 0 || g.b_stride > (int64_t{1} << 40)) return fail(CCE_EINVAL, "b_stride out of range");
  const int64_t be = wgrad ? eo : 2;
  if (wgrad && g.n_experts > 1 && g.b_stride * be < b1)
    return fail(CCE_EINVAL, "b_stride is smaller than one expert's matrix");
  if (!g.offsets) return fail(CCE_EINVAL, "offsets: NULL pointer");
  if (reinterpret_cast<uintptr_t>(g.offsets) % 8 != 0)
    return fail(CCE_EUNSUPPORTED, "offsets: pointer not 8-byte aligned");
  const int64_t bs = b1 == 0 ? 0 : (g.n_experts - 1) * g.b_stride * be + b1;
  CCE_TRY(check_spans({{"a", g.a, as, dgrad},
                       {"b", g.b, bs, wgrad},
                       {"c", g.c, cs, fwd},
                       {"offsets", g.offsets, 8 * (static_cast<int64_t>(g.n_experts) + 1), false}}));
  RaggedLaunch L;
  L.kind = kind;
  L.experts = g.n_experts;
  L.offsets = g.offsets;
  L.a = g.a;
  L.b = g.b;
  L.c = g.c;
  L.out_t = g.out_t;
  L.T = g.a_shape.rows;
  L.N = g.c_shape.cols;
  L.K = g.a_shape.cols;
  L.lda = g.a_shape.ld;
  L.ldb = g.b_shape.ld;
  L.ldc = g.c_shape.ld;
  L.stride_b = g.b_stride;
  // nothing to write (an empty contraction still writes zeros)
  if ((fwd && (L.T == 0 || L.N == 0)) || (dgrad && (L.T == 0 || L.K == 0)) || (wgrad && (L.N == 0 || L.K == 0)))
    return CCE_OK;
  DeviceGuard guard(g.ctx->device);
  hipStream_t hs = static_cast<hipStream_t>(g.stream);
  int slot;
  CCE_TRY(prof_begin(g.ctx, hs, 0, -1, 2.0 * L.T * L.N * L.K, 0.0, &slot));
  CCE_TRY(launch_ragged(L, g.stream));
  return prof_end(g.ctx, hs, slot);
}

}  // namespace
}  // namespace cce

using namespace cce;

extern "C" {

cce_status cce_rmsnorm(cce_ctx* ctx, cce_dtype x_t, const void* x, cce_mat x_shape, const void* residual,
                       int64_t ld_residual, void* residual_out, int64_t ld_residual_out,
                       const void* weight, cce_dtype weight_t, double eps, void* out, cce_dtype out_t,
                       int64_t ld_out, uint8_t* scales, int64_t ld_scales, uint32_t flags,
                       cce_stream stream) {
  return guarded([&]() -> cce_status {
    if (!ctx) return fail(CCE_EINVAL, "ctx is NULL");
    if (flags != 0) return fail(CCE_EINVAL, "flags must be 0");
    if (!dtype_ok(x_t) || !dtype_ok(weight_t) || !(dtype_ok(out_t) || out_t == CCE_E4M3))
      return fail(CCE_EINVAL, "bad dtype");
    CCE_TRY(check_eps(eps));
    if (residual_out && !residual) return fail(CCE_EINVAL, "residual_out needs a residual");
    const bool q = out_t == CCE_E4M3;
    if (!q && scales) return fail(CCE_EINVAL, "scales need an e4m3 output");
    const int64_t rows = x_shape.rows, cols = x_shape.cols;
    const cce_mat rm{rows, cols, ld_residual}, rom{rows, cols, ld_residual_out}, om{rows, cols, ld_out};
    const cce_mat sm{rows, blocks_of(cols), ld_scales};
    const size_t ex = esize(x_t);
    const int64_t xs = span_bytes(x_shape, ex), rs = residual ? span_bytes(rm, ex) : 0,
                  ros = residual_out ? span_bytes(rom, ex) : 0,
                  os = span_bytes(om, q ? 1 : esize(out_t)), ss = q ? span_bytes(sm, 1) : 0,
                  ws = cols * static_cast<int64_t>(esize(weight_t));
    CCE_TRY(check_operand("x", x, x_shape, xs));
    CCE_TRY(check_rows(x_shape));
    if (residual) CCE_TRY(check_operand("residual", residual, rm, rs));
    if (residual_out) CCE_TRY(check_operand("residual_out", residual_out, rom, ros));
    CCE_TRY(check_operand("out", out, om, os));
    CCE_TRY(check_ptr("weight", weight, ws));
    if (q) CCE_TRY(check_scales("scales", scales, sm));
    CCE_TRY(check_spans({{"x", x, xs, false},
                         {"residual", residual, rs, false},
                         {"weight", weight, ws, false},
                         {"residual_out", residual_out, ros, true},
                         {"out", out, os, true},
                         {"scales", scales, ss, true}}));
    if (rows == 0 || cols == 0) return CCE_OK;
    NormLaunch L;
    L.x_t = x_t;
    L.w_t = weight_t;
    L.out_t = out_t;
    L.x = x;
    L.res = residual;
    L.res_out = residual_out;
    L.w = weight;
    L.out = out;
    L.scales = scales;
    L.rows = rows;
    L.cols = cols;
    L.ld_x = x_shape.ld;
    L.ld_res = ld_residual;
    L.ld_res_out = ld_residual_out;
    L.ld_out = ld_out;
    L.ld_scales = ld_scales;
    L.eps = static_cast<float>(eps);
    DeviceGuard guard(ctx->device);
    hipStream_t hs = static_cast<hipStream_t>(stream);
    int slot;
    CCE_TRY(prof_begin(ctx, hs, 4, -1, 0.0,
                       static_cast<double>(rows) * cols * (ex * (1 + !!residual + !!residual_out) + (q ? 1 : esize(out_t))),
                       &slot));
    CCE_TRY(launch_rmsnorm(L, stream));
    return prof_end(ctx, hs, slot);
  });
}

cce_status cce_rmsnorm_backward_workspace(cce_mat x_shape, size_t* bytes) {
  return guarded([&]() -> cce_status {
    if (!bytes) return fail(CCE_EINVAL, "bytes is NULL");
    CCE_TRY(check_mat("x", x_shape));
    *bytes = rmsnorm_backward_bytes(x_shape.rows, x_shape.cols);
    return CCE_OK;
  });
}

cce_status cce_rmsnorm_backward(cce_ctx* ctx, cce_dtype x_t, const void* x, cce_mat x_shape,
                                const void* weight, cce_dtype weight_t, const void* dout, int64_t ld_dout,
                                const void* d_residual, int64_t ld_d_residual, double eps, void* dx,
                                int64_t ld_dx, float* dweight, void* workspace, size_t workspace_bytes,
                                uint32_t flags, cce_stream stream) {
  return guarded([&]() -> cce_status {
    if (!ctx) return fail(CCE_EINVAL, "ctx is NULL");
    if (flags != 0) return fail(CCE_EINVAL, "flags must be 0");
    if (!dtype_ok(x_t) || !dtype_ok(weight_t)) return fail(CCE_EINVAL, "bad dtype");
    CCE_TRY(check_eps(eps));
    const int64_t rows = x_shape.rows, cols = x_shape.cols;
    const cce_mat dm{rows, cols, ld_dout}, rm{rows, cols, ld_d_residual}, om{rows, cols, ld_dx};
    const size_t ex = esize(x_t);
    const int64_t xs = span_bytes(x_shape, ex), ds = span_bytes(dm, ex),
                  rs = d_residual ? span_bytes(rm, ex) : 0, os = span_bytes(om, ex),
                  ws = cols * static_cast<int64_t>(esize(weight_t)), dws = dweight ? cols * 4 : 0;
    CCE_TRY(check_operand("x", x, x_shape, xs));
    CCE_TRY(check_rows(x_shape));
    CCE_TRY(check_ptr("weight", weight, ws));
    CCE_TRY(check_operand("dout", dout, dm, ds));
    if (d_residual) CCE_TRY(check_operand("d_residual", d_residual, rm, rs));
    CCE_TRY(check_operand("dx", dx, om, os));
    CCE_TRY(check_ptr("dweight", dweight, dws));
    const size_t need = dweight ? rmsnorm_backward_bytes(rows, cols) : 0;   // (all of it is for dweight)
    if (need > 0 && (!workspace || workspace_bytes < need))
      return fail(CCE_EWORKSPACE, "workspace: " + std::to_string(need) + " bytes needed");
    if (need > 0) CCE_TRY(check_ptr("workspace", workspace, static_cast<int64_t>(need)));
    CCE_TRY(check_spans({{"x", x, xs, false},
                         {"weight", weight, ws, false},
                         {"dout", dout, ds, false},
                         {"d_residual", d_residual, rs, false},
                         {"dx", dx, os, true},
                         {"dweight", dweight, dws, true},
                         {"workspace", workspace, static_cast<int64_t>(need), true}}));
    if (cols == 0 || (rows == 0 && !dweight)) return CCE_OK;
    NormBackwardLaunch L;
    L.x_t = x_t;
    L.w_t = weight_t;
    L.x = x;
    L.w = weight;
    L.dout = dout;
    L.dres = d_residual;
    L.dx = dx;
    L.dw = dweight;
    L.workspace = workspace;
    L.rows = rows;
    L.cols = cols;
    L.ld_x = x_shape.ld;
    L.ld_dout = ld_dout;
    L.ld_dres = ld_d_residual;
    L.ld_dx = ld_dx;
    L.eps = static_cast<float>(eps);
    DeviceGuard guard(ctx->device);
    hipStream_t hs = static_cast<hipStream_t>(stream);
    int slot;
    CCE_TRY(prof_begin(ctx, hs, 4, -1, 0.0, static_cast<double>(rows) * cols * ex * (3 + !!d_residual), &slot));
    CCE_TRY(launch_rmsnorm_backward(L, stream));
    return prof_end(ctx, hs, slot);
  });
}

cce_status cce_quantize_blocks(cce_ctx* ctx, cce_dtype x_t, const void* x, cce_mat x_shape, int block_rows,
                               uint8_t* q, int64_t ld_q, uint8_t* scales, int64_t ld_scales,
                               uint32_t flags, cce_stream stream) {
  return guarded([&]() -> cce_status {
    if (!ctx) return fail(CCE_EINVAL, "ctx is NULL");
    if (flags != 0) return fail(CCE_EINVAL, "flags must be 0");
    if (!dtype_ok(x_t)) return fail(CCE_EINVAL, "bad dtype");
    if (block_rows != 1 && block_rows != 128) return fail(CCE_EINVAL, "block_rows must be 1 or 128");
    const int64_t rows = x_shape.rows, cols = x_shape.cols;
    const cce_mat qm{rows, cols, ld_q}, sm{(rows + block_rows - 1) / block_rows, blocks_of(cols), ld_scales};
    const int64_t xs = span_bytes(x_shape, esize(x_t)), qs = span_bytes(qm, 1), ss = span_bytes(sm, 1);
    CCE_TRY(check_operand("x", x, x_shape, xs));
    CCE_TRY(check_rows(x_shape));
    CCE_TRY(check_operand("q", q, qm, qs));
    CCE_TRY(check_scales("scales", scales, sm));
    CCE_TRY(check_spans({{"x", x, xs, false}, {"q", q, qs, true}, {"scales", scales, ss, true}}));
    if (rows == 0 || cols == 0) return CCE_OK;
    QuantizeLaunch L;
    L.x_t = x_t;
    L.x = x;
    L.q = q;
    L.scales = scales;
    L.block_rows = block_rows;
    L.rows = rows;
    L.cols = cols;
    L.ld_x = x_shape.ld;
    L.ld_q = ld_q;
    L.ld_scales = ld_scales;
    DeviceGuard guard(ctx->device);
    hipStream_t hs = static_cast<hipStream_t>(stream);
    int slot;
    CCE_TRY(prof_begin(ctx, hs, 5, -1, 0.0, static_cast<double>(rows) * cols * (esize(x_t) + 1), &slot));
    CCE_TRY(launch_quantize_blocks(L, stream));
    return prof_end(ctx, hs, slot);
  });
}

cce_status cce_block_scaled_gemm(cce_ctx* ctx, cce_dtype out_t, const uint8_t* a, cce_mat a_shape,
                                 const uint8_t* a_scales, int64_t ld_a_scales, const uint8_t* b,
                                 cce_mat b_shape, const uint8_t* b_scales, int64_t ld_b_scales, void* c,
                                 cce_mat c_shape, uint32_t flags, cce_stream stream) {
  return guarded([&]() -> cce_status {
    if (!ctx) return fail(CCE_EINVAL, "ctx is NULL");
    if (flags & ~CCE_FLAG_GELU) return fail(CCE_EINVAL, "unsupported flags for the block-scaled GEMM");
    if (!dtype_ok(out_t)) return fail(CCE_EINVAL, "bad dtype");
    const int64_t M = a_shape.rows, N = b_shape.rows, K = a_shape.cols, kb = blocks_of(K);
    const cce_mat sam{M, kb, ld_a_scales}, sbm{blocks_of(N), kb, ld_b_scales};
    const int64_t as = span_bytes(a_shape, 1), bs = span_bytes(b_shape, 1), cs = span_bytes(c_shape, esize(out_t)),
                  sas = span_bytes(sam, 1), sbs = span_bytes(sbm, 1);
    CCE_TRY(check_operand("a", a, a_shape, as));
    CCE_TRY(check_operand("b", b, b_shape, bs));
    CCE_TRY(check_operand("c", c, c_shape, cs));
    if (b_shape.cols != K) return fail(CCE_EINVAL, "a and b must share the contraction length");
    if (c_shape.rows != M || c_shape.cols != N) return fail(CCE_EINVAL, "c must be [a rows, b rows]");
    if (K % 16 != 0 || a_shape.ld % 16 != 0 || b_shape.ld % 16 != 0)
      return fail(CCE_EUNSUPPORTED, "the contraction length and both ld must be multiples of 16");
    CCE_TRY(check_rows(a_shape));
    CCE_TRY(check_rows(b_shape));
    CCE_TRY(check_ld("a", a_shape.ld));
    CCE_TRY(check_ld("b", b_shape.ld));
    CCE_TRY(check_ld("c", c_shape.ld));
    CCE_TRY(check_ld("a_scales", ld_a_scales));
    CCE_TRY(check_ld("b_scales", ld_b_scales));
    CCE_TRY(check_scales("a_scales", a_scales, sam));
    CCE_TRY(check_scales("b_scales", b_scales, sbm));
    CCE_TRY(check_spans({{"a", a, as, false},
                         {"a_scales", a_scales, sas, false},
                         {"b", b, bs, false},
                         {"b_scales", b_scales, sbs, false},
                         {"c", c, cs, true}}));
    if (M == 0 || N == 0) return CCE_OK;
    Gemm8Launch L;
    L.a = a;
    L.b = b;
    L.sa = a_scales;
    L.sb = b_scales;
    L.c = c;
    L.out_t = out_t;
    L.gelu = (flags & CCE_FLAG_GELU) != 0;
    L.M = M;
    L.N = N;
    L.K = K;
    L.lda = a_shape.ld;
    L.ldb = b_shape.ld;
    L.ldc = c_shape.ld;
    L.ld_sa = ld_a_scales;
    L.ld_sb = ld_b_scales;
    DeviceGuard guard(ctx->device);
    hipStream_t hs = static_cast<hipStream_t>(stream);
    int slot;
    CCE_TRY(prof_begin(ctx, hs, 0, -1, 2.0 * M * N * K, 0.0, &slot));
    CCE_TRY(launch_gemm8(L, stream));
    return prof_end(ctx, hs, slot);
  });
}

cce_status cce_ragged_gemm(cce_ctx* ctx, cce_dtype out_t, int n_experts, const int64_t* offsets, const void* a,
                           cce_mat a_shape, const void* b, cce_mat b_shape, int64_t b_stride, void* c,
                           cce_mat c_shape, uint32_t flags, cce_stream stream) {
  return guarded([&] {
    return ragged(RAGGED_FORWARD, {ctx, out_t, n_experts, offsets, const_cast<void*>(a), a_shape,
                                   const_cast<void*>(b), b_shape, b_stride, c, c_shape, flags, stream});
  });
}

cce_status cce_ragged_gemm_dgrad(cce_ctx* ctx, cce_dtype out_t, int n_experts, const int64_t* offsets,
                                 const void* dc, cce_mat c_shape, const void* b, cce_mat b_shape,
                                 int64_t b_stride, void* da, cce_mat a_shape, uint32_t flags,
                                 cce_stream stream) {
  return guarded([&] {
    return ragged(RAGGED_DGRAD, {ctx, out_t, n_experts, offsets, da, a_shape, const_cast<void*>(b), b_shape,
                                 b_stride, const_cast<void*>(dc), c_shape, flags, stream});
  });
}

cce_status cce_ragged_gemm_wgrad(cce_ctx* ctx, cce_dtype out_t, int n_experts, const int64_t* offsets,
                                 const void* dc, cce_mat c_shape, const void* a, cce_mat a_shape, void* db,
                                 cce_mat b_shape, int64_t b_stride, uint32_t flags, cce_stream stream) {
  return guarded([&] {
    return ragged(RAGGED_WGRAD, {ctx, out_t, n_experts, offsets, const_cast<void*>(a), a_shape, db, b_shape,
                                 b_stride, const_cast<void*>(dc), c_shape, flags, stream});
  });
}

}  // extern "C"
