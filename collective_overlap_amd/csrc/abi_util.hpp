// What the C entry points share (abi.cpp: the looped calls and the epilogues;
// layer.cpp: the operators around them): the context, argument checks, the
// device of a call and the timing brackets.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>
#include <vector>

#include "cce_internal.hpp"

struct cce_prof_slot {
  int kind = 0;
  int iter = -1;
  double flops = 0, bytes = 0;
  hipEvent_t start = nullptr, stop = nullptr;
};

struct cce_ctx {
  int device = 0;
  hipStream_t copy = nullptr;            // the stream the permute copies run on
  hipStream_t own_copy = nullptr;        // the context's own copy stream
  unsigned* err = nullptr;               // device word: chunk consumers that gave up (fine-grained overlap)
  std::vector<hipEvent_t> events;        // ordering events (no timing)
  bool profiling = false;
  std::vector<hipEvent_t> timing_pool;   // timing events, reused
  size_t timing_used = 0;
  std::vector<cce_prof_slot> prof;
};

namespace cce {

// GEMM operands are addressed through 32-bit buffer offsets (see gemm.hip).
constexpr int64_t kMaxOperandBytes = (int64_t{1} << 30) - 256;

inline size_t esize(cce_dtype t) { return t == CCE_F32 ? 4 : 2; }
inline bool dtype_ok(int t) { return t == CCE_F32 || t == CCE_BF16; }
inline int64_t align256(int64_t b) { return (b + 255) & ~int64_t{255}; }
inline int64_t round8(int64_t v) { return (v + 7) & ~int64_t{7}; }

inline int64_t span_bytes(const cce_mat& m, size_t es) {
  if (m.rows <= 0 || m.cols <= 0) return 0;
  return ((m.rows - 1) * m.ld + m.cols) * static_cast<int64_t>(es);
}

inline std::string mat_str(const cce_mat& m) {
  return "[" + std::to_string(m.rows) + "," + std::to_string(m.cols) + "] ld " + std::to_string(m.ld);
}

inline cce_status check_mat(const char* name, const cce_mat& m) {
  if (m.rows < 0 || m.cols < 0 || m.ld < m.cols || m.ld < 0)
    return fail(CCE_EINVAL, std::string(name) + ": bad extents " + mat_str(m));
  if (m.ld % 8 != 0)
    return fail(CCE_EUNSUPPORTED, std::string(name) + ": ld must be a multiple of 8, got " + mat_str(m));
  if (m.rows > 0x7fffffff || m.cols > 0x7fffffff || m.ld > 0x7fffffff)
    return fail(CCE_EUNSUPPORTED, std::string(name) + ": extent exceeds 2^31");
  return CCE_OK;
}

inline cce_status check_ptr(const char* name, const void* p, int64_t span) {
  if (span == 0) return CCE_OK;
  if (!p) return fail(CCE_EINVAL, std::string(name) + ": NULL pointer");
  if (reinterpret_cast<uintptr_t>(p) % 16 != 0)
    return fail(CCE_EUNSUPPORTED, std::string(name) + ": pointer not 16-byte aligned");
  return CCE_OK;
}

struct Range {
  uintptr_t lo, hi;
  std::string name;
  bool writes;
};

// Outputs may overlap nothing; inputs may overlap each other.
inline cce_status check_overlaps(const std::vector<Range>& rs) {
  for (size_t i = 0; i < rs.size(); ++i) {
    if (rs[i].hi <= rs[i].lo) continue;
    for (size_t j = i + 1; j < rs.size(); ++j) {
      if (rs[j].hi <= rs[j].lo) continue;
      if (!rs[i].writes && !rs[j].writes) continue;
      if (rs[i].lo < rs[j].hi && rs[j].lo < rs[i].hi)
        return fail(CCE_EINVAL, rs[i].name + " overlaps " + rs[j].name);
    }
  }
  return CCE_OK;
}

inline Range range_of(const void* p, int64_t span, const std::string& name, bool writes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + static_cast<uintptr_t>(span), name, writes};
}

#define CCE_TRY(expr)                       \
  do {                                      \
    cce_status _s = (expr);                 \
    if (_s != CCE_OK) return _s;            \
  } while (0)

#define HIP_TRY(expr)                                                              \
  do {                                                                             \
    hipError_t _e = (expr);                                                        \
    if (_e != hipSuccess)                                                          \
      return fail(CCE_EHIP, std::string(#expr) + ": " + hipGetErrorString(_e));    \
  } while (0)

// Makes ctx->device current for the duration of a call.
class DeviceGuard {
 public:
  explicit DeviceGuard(int dev) {
    if (hipGetDevice(&prev_) != hipSuccess) prev_ = -1;
    if (prev_ != dev) hipSetDevice(dev);
    dev_ = dev;
  }
  ~DeviceGuard() {
    if (prev_ >= 0 && prev_ != dev_) hipSetDevice(prev_);
  }

 private:
  int prev_ = -1, dev_ = 0;
};

// Timing brackets around a launch (only while profiling is enabled).
cce_status prof_begin(cce_ctx* ctx, hipStream_t s, int kind, int iter, double flops, double bytes,
                      int* slot);
cce_status prof_end(cce_ctx* ctx, hipStream_t s, int slot);

}  // namespace cce
