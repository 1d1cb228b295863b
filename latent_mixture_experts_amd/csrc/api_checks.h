// api_checks.h -- argument checks that the entry points of rows and products
// share (internal to libmoe).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

constexpr int32_t kMaxRows = 1 << 28;
constexpr int32_t kMaxWidth = 65536;
constexpr int64_t kMaxPitch = int64_t{1} << 22;    // elements (of codes: bytes) between rows
constexpr int64_t kDescriptor = int64_t{1} << 31;  // bytes one buffer descriptor spans
constexpr int kMaxExperts = 256;                   // four experts per lane of the group search

inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline int need(const void* p, size_t n) {
  if (!p) return MOE_EINVAL;
  return aligned(p, n) ? MOE_OK : MOE_EALIGN;
}

inline int type_ok(int32_t type) { return type == MOE_TYPE_BF16 || type == MOE_TYPE_F32 ? MOE_OK : MOE_EINVAL; }
inline size_t type_size(int32_t type) { return type == MOE_TYPE_F32 ? 4 : 2; }

#define MOE_TRY(expr)              \
  do {                             \
    const int rc_ = (expr);        \
    if (rc_ != MOE_OK) return rc_; \
  } while (0)

}  // namespace moe
