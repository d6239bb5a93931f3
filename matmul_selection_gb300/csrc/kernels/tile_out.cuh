// Tiles on their way from TMEM to global memory through boxes in shared memory: 32
// rows of 128 bytes, 16-byte pieces exchanged as the 128-byte swizzle has them.
#pragma once

#include "values.cuh"

namespace mm {
namespace {

constexpr uint32_t kBoxB = 32 * 128;

__device__ __forceinline__ uint32_t pack2(int tc, float lo, float hi) {
  if (tc == MM_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// A box of rows of 128 swizzled bytes to a matrix of ES-byte elements, from
// element i on, `left` columns: a row an access of up to 128 bytes, which for
// 2-byte elements is two a lane; where the row starts between two, its first
// element goes alone.
template <int ES>
__device__ __forceinline__ void store_box(const uint8_t *box, void *out, int64_t i, int64_t ldc, int rows, int left) {
  const int lane = threadIdx.x & 31;
  constexpr int U = 8;  // rows read before the first of them is stored
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += U) {
    uint32_t v[U], next[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const auto word = [&](int k) {
        return *reinterpret_cast<const uint32_t *>(box + (r0 + u) * 128 + (((k >> 2) ^ u) << 4) + (k & 3) * 4);
      };
      v[u] = word(lane);
      if (ES == 2) next[u] = word((lane + 1) & 31);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r0 + u >= rows) break;
      char *to = static_cast<char *>(out) + (i + (r0 + u) * ldc) * ES;
      if constexpr (ES == 4) {
        if (lane < left) reinterpret_cast<uint32_t *>(to)[lane] = v[u];
      } else {
        uint16_t *const row = reinterpret_cast<uint16_t *>(to);
        const int odd = (int)((uintptr_t)to >> 1) & 1, j = 2 * lane + odd;
        if (odd && lane == 0) row[0] = (uint16_t)v[u];
        const uint32_t x = __funnelshift_r(v[u], next[u], odd * 16);
        if (j + 1 < left) *reinterpret_cast<uint32_t *>(row + j) = x;
        else if (j < left) row[j] = (uint16_t)x;
      }
    }
  }
}

}  // namespace
}  // namespace mm
