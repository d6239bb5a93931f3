// Token numbers by type.
#pragma once

#include "../common.h"

namespace mm {

__device__ __forceinline__ int64_t load_index(const void *p, int t, int64_t i) {
  return t == MM_I32 ? (int64_t)static_cast<const int32_t *>(p)[i] : static_cast<const int64_t *>(p)[i];
}
// The token at i, or `vocab` where it is none of 0 .. vocab - 1.
__device__ __forceinline__ int64_t load_token(const void *p, int t, int64_t i, int64_t vocab) {
  const int64_t v = load_index(p, t, i);
  return v >= 0 && v < vocab ? v : vocab;
}

}  // namespace mm
