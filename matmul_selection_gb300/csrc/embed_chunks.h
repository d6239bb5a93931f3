// Chunks of sorted places, of the embedding's gradient: how they are laid out over threads
// and which places each reads.
#pragma once

#include <algorithm>
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

// The sums over threads: a power of two of them to a chunk, a piece of the columns each, in
// slabs where there are more pieces; and chunks that fill the device once (65536 x 1024 in
// chunks of 54 40 us; of 32, 1.7 times, 48).
constexpr int kMinLogThreads = 3, kSumThreads = 256;
constexpr int kSumBlocks = 4;  // an SM, at once
struct SumShape {
  int log_threads, chunk, chunks;
  int64_t slabs, across;  // blocks for all chunks of a slab
  bool fits;              // in a grid
};
inline SumShape sum_shape(int64_t rows, int64_t pieces, int sms) {
  SumShape s;
  s.log_threads = kMinLogThreads;
  while (s.log_threads < 8 && (1ll << s.log_threads) < pieces) ++s.log_threads;
  s.slabs = (pieces + (1 << s.log_threads) - 1) >> s.log_threads;
  const int64_t per_block = kSumThreads >> s.log_threads;
  const int64_t groups = std::max<int64_t>(1, kSumBlocks * sms / s.slabs) * per_block;
  s.chunk = (int)std::max<int64_t>(kMinChunk, std::min<int64_t>(kMaxChunk, (rows + groups - 1) / groups));
  s.chunks = (int)((rows + s.chunk - 1) / s.chunk);
  s.across = (s.chunks + per_block - 1) / per_block;
  s.fits = s.across * s.slabs < 1 << 30;
  return s;
}

}  // namespace mm
