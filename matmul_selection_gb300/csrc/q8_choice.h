// Which of the e4m3 product's forms takes a size.
#pragma once

#include <cstdint>

namespace mm {

enum Q8Form { Q8_GEMV, Q8_SWAP, Q8_PAIR };
struct Q8Choice {
  Q8Form form;
  int bn;     // swap: rows of A a tile
  int ranks;  // swap: CTAs that split K
};

constexpr int64_t kQ8SwapRowTiles = 65535;  // a grid's third dimension

// M, N > 0; K as num_kb blocks of 128 bytes; a device of `sms` SMs that holds
// `clusters` pairs of CTAs.
inline Q8Choice choose_q8(int64_t M, int64_t N, int64_t num_kb, int sms, int clusters) {
  // At most 8 rows of A and too few rows of weights to fill the SMs with tiles
  // of 128: the GEMV form, whose tiles are of 16 to 64.  us, GEMV / swap: 1 x
  // 4096 x 4096 5.4 / 6.5, 1 x 2048 x 16384 9.2 / 13.9, 4 x 6144 x 6144 10.6 /
  // 10.4, 1 x 8192 x 8192 16.1 / 14.2, 1 x 16384 x 8192 29.0 / 23.5; 16 rows:
  // 16 x 4096 x 4096 7.6 / 6.7.
  if (M <= 8 && N <= 6144) return {Q8_GEMV, 0, 0};
  // swap: a tile of as few rows as hold A, and K over as many CTAs as fill the SMs
  const int bn = M <= 32 ? 32 : M <= 64 ? 64 : 128;
  const int64_t row_tiles = (M + bn - 1) / bn, tiles = (N + 127) / 128 * row_tiles;
  int ranks = 1;
  while (ranks < 8 && tiles * ranks * 2 <= sms && num_kb >= 4 * ranks) ranks *= 2;
  const Q8Choice swap{Q8_SWAP, bn, ranks}, pair{Q8_PAIR, 0, 0};
  if (M <= 128) return swap;
  if (row_tiles > kQ8SwapRowTiles) return pair;
  // Above 128 rows of A, pair or swap, whichever its waves say takes less: a
  // wave costs its stages (0.29 us of a pair's, 0.18 of a swap's, the measured
  // slopes) and what surrounds them.  us, pair / swap: 300 x 4096 x 4096 17.5 /
  // 13.4, 512 x 4096 x 4096 18.4 / 14.3.
  const int64_t pairs = ((M + 255) / 256) * ((N + 255) / 256);
  const double pair_us = (double)((pairs + clusters - 1) / clusters) * (double)num_kb * 0.29 + 8.0;
  const double swap_us = (double)((tiles * ranks + sms - 1) / sms) *
                             ((double)((num_kb + ranks - 1) / ranks) * 0.183 + 2.5) + 5.0;
  return pair_us < swap_us ? pair : swap;
}

}  // namespace mm
