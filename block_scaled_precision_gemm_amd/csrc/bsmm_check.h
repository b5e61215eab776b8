// Argument checks shared by the host entry points.
#pragma once

#include <cstdint>

#include "bsmm.h"

namespace bsmm {

// Record a printf-style message as this thread's last error; returns s.
bsmm_status fail(bsmm_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

constexpr int64_t kMaxDim = (int64_t)1 << 31;

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
// rows of bf16 or fp32 at 16-byte aligned addresses
inline bool aligned_rows(const void* p, int64_t ld, bsmm_dtype d) {
  return aligned(p, 16) && ld % (d == BSMM_BF16 ? 8 : 4) == 0;
}

}  // namespace bsmm

#define CHECK(cond, status, ...) \
  do { if (!(cond)) return fail(status, __VA_ARGS__); } while (0)
