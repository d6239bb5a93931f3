// The e4m3 product's choice of form: what it chooses can take the size.
#include <cstdio>
#include <initializer_list>

#include "q8_choice.h"

#define CHECK(x)                                                                            \
  do {                                                                                      \
    if (!(x)) {                                                                             \
      std::printf("line %d: %s (M %lld N %lld kb %lld)\n", __LINE__, #x, (long long)M, (long long)N, (long long)kb); \
      return 1;                                                                             \
    }                                                                                       \
  } while (0)

int main() {
  using namespace mm;
  const int64_t most = (1LL << 30) - 1;
  for (int sms : {8, 132, 152})
    for (int64_t M = 1; M <= most; M = M < 300 ? M + 1 : M * 9 / 8)
      for (int64_t N : {(int64_t)1, (int64_t)128, (int64_t)129, (int64_t)4096, (int64_t)6144, (int64_t)6145, most})
        for (int64_t kb : {1, 8, 24, 32, 512, 8388607}) {
          const Q8Choice c = choose_q8(M, N, kb, sms, sms / 2);
          if (c.form == Q8_GEMV) CHECK(M <= 8 && N <= 6144);
          if (c.form == Q8_PAIR) CHECK(M > 128);
          if (c.form == Q8_SWAP) {
            CHECK(c.bn == 32 || c.bn == 64 || c.bn == 128);
            CHECK(M > 128 || c.bn >= M || c.bn == 128);
            CHECK((M + c.bn - 1) / c.bn <= kQ8SwapRowTiles);
            CHECK(c.ranks == 1 || c.ranks == 2 || c.ranks == 4 || c.ranks == 8);
            // a cluster's CTAs fill a wave at most, and each has some of K's blocks to begin with
            if (c.ranks > 1) CHECK((N + 127) / 128 * ((M + c.bn - 1) / c.bn) * c.ranks <= sms && kb >= 2 * c.ranks);
          }
        }
  const int64_t M = 0, N = 0, kb = 0;
  // 8.4 million rows, N = 128: more row tiles than a grid's third dimension has
  CHECK(choose_q8(8400000, 128, 24, 152, 76).form == Q8_PAIR);
  CHECK(choose_q8(65535 * 128, 128, 24, 152, 76).form == Q8_SWAP);
  // the measured ones
  CHECK(choose_q8(1, 4096, 32, 152, 76).form == Q8_GEMV && choose_q8(1, 8192, 64, 152, 76).form == Q8_SWAP);
  CHECK(choose_q8(300, 4096, 32, 152, 76).form == Q8_SWAP && choose_q8(512, 4096, 32, 152, 76).form == Q8_SWAP);
  CHECK(choose_q8(8192, 8192, 64, 152, 76).form == Q8_PAIR);
  std::puts("ok");
}
