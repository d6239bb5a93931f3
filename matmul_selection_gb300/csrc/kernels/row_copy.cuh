// Rows of bytes that lie anywhere, moved in 16-byte pieces.
#pragma once

#include <cstdint>

namespace mm {
namespace {

// Bytes shift .. shift + 15 of the 32 that two pieces hold.
__device__ __forceinline__ uint4 shifted_bytes(uint4 first, uint4 second, int shift) {
  uint32_t w[8] = {first.x, first.y, first.z, first.w, second.x, second.y, second.z, second.w};
  const int words = shift >> 2, bits = (shift & 3) * 8;
#pragma unroll
  for (int b = 2; b > 0; b /= 2)
#pragma unroll
    for (int j = 0; j + b < 8; ++j) w[j] = words & b ? w[j + b] : w[j];
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// Bytes b .. b + 15 of a row of `bytes`, zeros past its end.  Whole 16-byte words are
// read where the two that hold a piece lie inside the row; else single elements of
// ES bytes.
template <int ES>
__device__ __forceinline__ uint4 row_piece(const uint8_t *row, int64_t bytes, int64_t b) {
  const int shift = (int)(reinterpret_cast<uintptr_t>(row + b) & 15);
  if (shift == 0 && b + 16 <= bytes) return *reinterpret_cast<const uint4 *>(row + b);
  if (b >= shift && b - shift + 32 <= bytes) {
    const uint4 *at = reinterpret_cast<const uint4 *>(row + b - shift);
    return shifted_bytes(at[0], at[1], shift);
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 16; e += ES)
    if (b + e < bytes) {
      const uint32_t v = ES == 1 ? row[b + e] : *reinterpret_cast<const uint16_t *>(row + b + e);
      w[e >> 2] |= v << (8 * (e & 3));
    }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace
}  // namespace mm
