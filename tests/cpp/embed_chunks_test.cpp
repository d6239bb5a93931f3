// Places that the chunks of the embedding's gradient read: every one that they need, none
// that is not there.
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
  std::printf("ok\n");
}
