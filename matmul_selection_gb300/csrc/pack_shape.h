// How rows that are copied are shared out over threads.
#pragma once

#include <algorithm>
#include <cstdint>

namespace mm {

struct PackShape {
  int log_threads;  // a power of two of threads to a row, with up to four pieces of 16 bytes each
  int64_t blocks;   // of `block` threads
};
// `rows` rows of ld16 bytes by at most `most` blocks of `block` threads (a power of two).  Few
// long rows take the threads of many blocks each (by 256 threads a row, products of 32 and 16
// rows of a million bytes 304 -> 180 us, 20 and 64 of four million 1300 -> 870).
inline PackShape pack_shape(int64_t rows, int64_t ld16, int block, int64_t most) {
  PackShape s{0, 0};
  // (2^20 at most, so that a step of all of a row's threads counts in 32 bits)
  while (s.log_threads < 20 && (2ll << s.log_threads) <= most * block && (64ll << s.log_threads) < ld16) ++s.log_threads;
  s.blocks = std::min(((rows << s.log_threads) + block - 1) / block, most);
  return s;
}

}  // namespace mm
