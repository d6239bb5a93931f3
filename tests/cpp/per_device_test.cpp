// What is kept for each device, with made-up devices.
#include <cstdio>
#include <thread>
#include <vector>

#include "per_device.h"

#define CHECK(x)                                  \
  do {                                            \
    if (!(x)) {                                   \
      std::printf("line %d: %s\n", __LINE__, #x); \
      return 1;                                   \
    }                                             \
  } while (0)

int main() {
  {  // each device its own value, made once
    static mm::PerDevice<int> per;
    int made = 0, v = 0;
    for (int round = 0; round < 3; ++round)
      for (int d : {0, 1, 7}) {
        CHECK(per.get(d, &v, [&](int *x) { return ++made, *x = 100 + d, 0; }) == 0);
        CHECK(v == 100 + d);
      }
    CHECK(made == 3);
  }
  {  // a failure is returned and tried again
    static mm::PerDevice<int> per;
    int v = -1;
    CHECK(per.get(0, &v, [](int *) { return 5; }) == 5);
    CHECK(per.get(0, &v, [](int *x) { return *x = 3, 0; }) == 0 && v == 3);
    CHECK(per.get(0, &v, [](int *) { return 5; }) == 0 && v == 3);
  }
  {  // ordinals past the table
    static mm::PerDevice<int> per;
    int made = 0, v = 0;
    for (int k = 0; k < 2; ++k) CHECK(per.get(1000, &v, [&](int *x) { return ++made, *x = 9, 0; }) == 0 && v == 9);
    CHECK(made == 2);
  }
  {  // threads at one time: made once, everyone sees it
    static mm::PerDevice<int> per;
    std::atomic<int> made{0}, bad{0};
    std::vector<std::thread> all;
    for (int t = 0; t < 8; ++t)
      all.emplace_back([&] {
        for (int k = 0; k < 2000; ++k) {
          int v = 0;
          if (per.get(k % 64, &v, [&](int *x) { return ++made, *x = k % 64 + 1, 0; }) != 0 || v != k % 64 + 1) ++bad;
        }
      });
    for (auto &t : all) t.join();
    CHECK(made == 64 && bad == 0);
  }
  std::puts("ok");
}
