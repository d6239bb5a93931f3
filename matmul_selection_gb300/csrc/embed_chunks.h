// Chunks of sorted places, of the embedding's gradient: which places a chunk reads.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MM_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MM_HOST_DEVICE inline
#endif

namespace mm {

// A border between two chunks moves up to kSnap places on, to where a token ends; inside a
// longer run it stays.  (8192 x 4096 66 -> 63 us, 65536 x 1024 151 -> 147: fewer parts to
// join; 32 places make the chunks too unequal.)
constexpr int kSnap = 8;
constexpr int kMinChunk = 8, kMaxChunk = 64;

// How many places there are from i0, where a chunk begins, on: its own, those that it may
// take over, and the one that they are compared with.  0 past the last place, where the
// last block's other groups are.
MM_HOST_DEVICE int places_left(int64_t rows, int64_t i0, int chunk) {
  const int64_t left = rows - i0, most = (int64_t)chunk + kSnap + 1;
  return left <= 0 ? 0 : (int)(left < most ? left : most);
}
// Whether place i0 + i, i from -1 (the place before, which tells whether a token comes from
// there) to chunk + kSnap, is one that the chunk reads.
MM_HOST_DEVICE bool reads_place(int64_t i0, int i, int left) { return left > 0 && i < left && i0 + i >= 0; }

}  // namespace mm
