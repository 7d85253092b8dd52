// Argument checks that the C-ABI files of the operators around the layer share.
#pragma once

#include "pw_internal.h"

namespace pw {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline pw_status hip_status(hipError_t e) { return e == hipSuccess ? PW_OK : PW_ERR_HIP; }

// Bytes of an element of a row type, 0 if it is none.
inline int64_t row_type_bytes(int32_t dtype) { return dtype == PW_F32 ? 4 : (dtype == PW_F16 || dtype == PW_BF16) ? 2 : 0; }

// A matrix of T rows of H elements: 16-byte aligned rows `stride` elements
// apart.  Rows that are written must not overlap.
inline pw_status check_rows(const void* p, int64_t stride, int64_t T, int64_t H, int64_t bytes, bool written) {
  if (!p) return PW_ERR_INVALID_ARG;
  if (stride < 0 || (written && T > 1 && stride < H)) return PW_ERR_INVALID_ARG;
  if (!aligned(p, 16) || (stride * bytes) % 16) return PW_ERR_ALIGNMENT;
  return PW_OK;
}

#define PW_TRY(expr)                     \
  do {                                   \
    const pw_status st_ = (expr);        \
    if (st_ != PW_OK) return st_;        \
  } while (0)

}  // namespace pw
