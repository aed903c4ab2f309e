// api_common.h -- what the C entry points of the operators share: status codes, alignment, element sizes.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/muon.h"
#include "error.h"

namespace muon {

inline int bad(const char* what) { return set_error(MUON_ERR_INVALID_ARGUMENT, "%s", what); }
inline int hip_result(hipError_t e, const char* what) {
  if (e == hipSuccess) return set_error(MUON_OK, "%s", "");
  return set_error(MUON_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

#define MUON_TRY(x)                   \
  do {                                \
    const int rc_ = (x);              \
    if (rc_ != MUON_OK) return rc_;   \
  } while (0)

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int elem(int dtype) { return dtype == MUON_BF16 ? 2 : 4; }

}  // namespace muon
