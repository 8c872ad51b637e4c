// checks.hpp -- what the C ABI's translation units for the blocks share:
// limits of sizes and launches, and the check of a call's arrays.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "hyena.h"

namespace hyena {

constexpr int64_t kMaxRows = (int64_t)1 << 30;   // B * D
constexpr int64_t kMaxDim = (int64_t)1 << 20;
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;   // workgroups of 256 threads in a launch (2^32 threads)

// Arrays of a call: null checks are the caller's, absent ones are skipped.
struct Span {
  const void* p;
  int64_t bytes;
  int64_t align;
};

inline hyena_status check_spans(const Span* out, int no, const Span* in, int ni) {
  for (int i = 0; i < no + ni; ++i) {
    const Span& s = i < no ? out[i] : in[i - no];
    if (s.p && reinterpret_cast<uintptr_t>(s.p) % (uintptr_t)s.align) return HYENA_ERR_ALIGN;
  }
  const auto meet = [](const Span& a, const Span& b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
  };
  for (int i = 0; i < no; ++i) {
    for (int k = 0; k < ni; ++k)
      if (meet(out[i], in[k])) return HYENA_ERR_ALIAS;
    for (int k = 0; k < i; ++k)
      if (meet(out[i], out[k])) return HYENA_ERR_ALIAS;
  }
  return HYENA_OK;
}

template <int NO, int NI>
hyena_status check_spans(const Span (&out)[NO], const Span (&in)[NI]) {
  return check_spans(out, NO, in, NI);
}

inline bool io_ok(hyena_dtype io) { return io == HYENA_FP32 || io == HYENA_BF16; }
inline int64_t size_of(hyena_dtype io) { return io == HYENA_FP32 ? 4 : 2; }
inline bool batch_ok(int64_t B, int64_t D, int64_t L) {
  return B >= 1 && B <= kMaxDim && D >= 1 && D <= kMaxDim && B * D <= kMaxRows && L >= 1 && L <= HYENA_MAX_L;
}
inline hyena_status from_hip(hipError_t e) { return e == hipSuccess ? HYENA_OK : HYENA_ERR_HIP; }

}  // namespace hyena
