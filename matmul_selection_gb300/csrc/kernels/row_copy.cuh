// Rows of bytes that lie anywhere, moved in 16-byte pieces.
#pragma once

#include <cstdint>

#include "../pack_shape.h"

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
// read where those that hold the piece lie inside the row; else single elements of ES
// bytes.  load() reads the words and value() makes the piece, so that the reads of
// several pieces can be issued before the first is waited for.
template <int ES>
struct RowPiece {
  uint4 first, second;
  static __device__ __forceinline__ int shift_of(const uint8_t *row, int64_t b) {
    return (int)(reinterpret_cast<uintptr_t>(row + b) & 15);
  }
  static __device__ __forceinline__ bool in_words(const uint8_t *row, int64_t bytes, int64_t b) {
    const int shift = shift_of(row, b);
    return b >= shift && b - shift + (shift ? 32 : 16) <= bytes;
  }
  __device__ __forceinline__ void load(const uint8_t *row, int64_t bytes, int64_t b) {
    const int shift = shift_of(row, b);
    const uint4 *at = reinterpret_cast<const uint4 *>(row + b - shift);
    first = second = make_uint4(0, 0, 0, 0);
    if (in_words(row, bytes, b)) {
      first = at[0];
      if (shift) second = at[1];
    }
  }
  __device__ __forceinline__ uint4 value(const uint8_t *row, int64_t bytes, int64_t b) const {
    if (in_words(row, bytes, b)) return shifted_bytes(first, second, shift_of(row, b));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 16; e += ES)
      if (b + e < bytes) {
        const uint32_t v = ES == 1 ? row[b + e] : *reinterpret_cast<const uint16_t *>(row + b + e);
        w[e >> 2] |= v << (8 * (e & 3));
      }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// `rows` rows of `bytes` bytes, ld apart, to rows of ld16 bytes that start on 16, the last
// piece of each filled up with zeros.  `threads`: those that take part, of which this is
// number `thread`; a power of two of them to a row, no more than there are.
struct PackRows {
  const uint8_t *from;
  int64_t ld, rows, bytes;
  uint8_t *to;
  int64_t ld16;
  int log_threads;
};
inline PackRows pack_job(const void *from, int64_t ld, int64_t rows, int64_t bytes, void *to, int64_t ld16, int log_threads) {
  return {static_cast<const uint8_t *>(from), ld, rows, bytes, static_cast<uint8_t *>(to), ld16, log_threads};
}
__device__ __forceinline__ void pack_rows(const PackRows &p, int64_t thread, int64_t threads) {
  constexpr int U = 4;  // pieces read before the first is stored
  const int row_threads = 1 << p.log_threads, t = (int)thread & (row_threads - 1);
  // (a last, incomplete group of threads writes what others write too)
  for (int64_t r = thread >> p.log_threads; r < p.rows; r += threads >> p.log_threads) {
    const uint8_t *from = p.from + r * p.ld;
    uint8_t *to = p.to + r * p.ld16;
    for (int64_t b0 = t * 16; b0 < p.ld16; b0 += row_threads * 16 * U) {
      RowPiece<1> v[U];
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (b0 + k * row_threads * 16 < p.ld16) v[k].load(from, p.bytes, b0 + k * row_threads * 16);
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (b0 + k * row_threads * 16 < p.ld16)
          *reinterpret_cast<uint4 *>(to + b0 + k * row_threads * 16) = v[k].value(from, p.bytes, b0 + k * row_threads * 16);
    }
  }
}

}  // namespace
}  // namespace mm
