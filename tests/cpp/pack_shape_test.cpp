// How copied rows are shared out: no more threads to a row than there are, as many threads as
// the pieces keep busy, and no row left out.
#include <cstdio>

#include "pack_shape.h"

using namespace mm;

int main() {
  for (int block : {256, 512})
    for (int64_t most : {1, 3, 608, 1216, 2432})
      for (int64_t rows = 1; rows < 1ll << 30; rows = rows < 40 ? rows + 1 : rows * 7 / 4)
        for (int64_t pieces = 1; pieces < 1ll << 28; pieces = pieces < 40 ? pieces + 1 : pieces * 7 / 4) {
          const PackShape s = pack_shape(rows, pieces * 16, block, most);
          const int64_t threads = s.blocks * block, at_once = threads >> s.log_threads;
          // four pieces a thread (of which the last group may lack half), or every thread there is
          const int64_t busy = std::min((rows * pieces + 3) / 4, most * block);
          if (s.blocks < 1 || s.blocks > most || at_once < 1 || threads < std::min(busy, most * block / 2)) {
            std::printf("%lld rows of %lld pieces, %lld blocks of %d: %lld blocks, 2^%d threads a row\n", (long long)rows,
                        (long long)pieces, (long long)most, block, (long long)s.blocks, s.log_threads);
            return 1;
          }
        }
  if (pack_shape(0, 16, 256, 2432).blocks != 0) {
    std::printf("no rows\n");
    return 1;
  }
  std::printf("ok\n");
}
