// Argument checks and status helpers shared by the C entry points.
#pragma once

#include "../../include/convrot.h"
#include "common.h"
#include "internal.h"

namespace convrot {

// Set the calling thread's error string and return `s`.
convrot_status fail(convrot_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clear it and return CONVROT_OK.
convrot_status ok();
convrot_status hip_status(hipError_t e, const char* what);

SignMask make_signs(uint64_t seed, int g);

// shape checks of the MXFP4 product (api_mx4.hip)
convrot_status check_mx4_gemm(const char* fn, int64_t m, int64_t n, int64_t k);

inline bool valid_group(int g) { return g == 4 || g == 16 || g == 64 || g == 256; }

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x0 = (uintptr_t)a, x1 = x0 + na, y0 = (uintptr_t)b, y1 = y0 + nb;
  return x0 < y1 && y0 < x1;
}

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

constexpr int64_t kMaxDim = (int64_t)1 << 31;

// enum argument of the entry points that take a 16-bit format
inline bool dtype_of(int v, DType* dt) {
  if (v != CONVROT_DTYPE_BF16 && v != CONVROT_DTYPE_F16) return false;
  *dt = v == CONVROT_DTYPE_F16 ? DType::kF16 : DType::kBF16;
  return true;
}

}  // namespace convrot
