// The chunks of the embedding's gradient: the places that they read are every one that
// they need and none that is not there, and their grid is one that a launch takes.
#include <algorithm>
#include <cstdio>

#include "embed_chunks.h"

using namespace mm;

int main() {
  for (int64_t rows = 1; rows < 700; ++rows)
    for (int chunk = kMinChunk; chunk <= kMaxChunk; chunk += chunk < 12 ? 1 : 13) {
      const int64_t chunks = (rows + chunk - 1) / chunk;
      for (int per_block = 1; per_block <= 32; per_block *= 2) {  // (groups in a block)
        const int64_t groups = (chunks + per_block - 1) / per_block * per_block;
        for (int64_t c = 0; c < groups; ++c) {
          const int64_t i0 = c * chunk;
          const int left = places_left(rows, i0, chunk);
          for (int i = -1; i <= chunk + kSnap; ++i) {
            const bool there = i0 + i >= 0 && i0 + i < rows, wanted = c < chunks && there;
            if (reads_place(i0, i, left) != wanted) {
              std::printf("rows %lld, chunk %d of %lld, %d long: place %d\n", (long long)rows, (int)c, (long long)chunks,
                          chunk, i);
              return 1;
            }
          }
        }
      }
    }
  // far ones
  const int64_t rows = (1LL << 30) - 1, i0 = rows - 3;
  if (places_left(rows, i0, 64) != 3 || places_left(rows, i0 + 3, 64) != 0 || places_left(rows, 0, 64) != 64 + kSnap + 1) {
    std::printf("far places\n");
    return 1;
  }
  // the grid of the sums: one that a launch takes, or refused as such (before any launch)
  const int64_t most = (1LL << 30) - 1, most_cols = (1LL << 23) - 1;
  for (int sms : {1, 132, 152})
    for (int64_t r = 1;; r = std::min(most, r < 100 ? r + 1 : r * 5 / 4)) {
      for (int64_t pieces = 1;; pieces = std::min(most_cols, pieces < 100 ? pieces + 1 : pieces * 5 / 4)) {
        const SumShape s = sum_shape(r, pieces, sms);
        const int64_t per_block = kSumThreads >> s.log_threads;
        const bool good = s.chunk >= kMinChunk && s.chunk <= kMaxChunk && (int64_t)s.chunk * s.chunks >= r &&
                          (int64_t)s.chunk * (s.chunks - 1) < r && s.across * per_block >= s.chunks &&
                          (s.slabs << s.log_threads) >= pieces && s.fits == (s.across * s.slabs < (1LL << 30)) &&
                          (s.fits || r * pieces >= 1LL << 40);  // (as many elements never lie in memory)
        if (!good) {
          std::printf("%lld rows of %lld pieces\n", (long long)r, (long long)pieces);
          return 1;
        }
        if (pieces == most_cols) break;
      }
      if (r == most) break;
    }
  std::printf("ok\n");
}
