// The growth rules of the library's scratch buffers, with fake memory.
#include <cstdio>
#include <cstdlib>
#include <map>

#include "scratch.h"

using mm::Scratch;
using mm::ScratchBuffer;

#define CHECK(x)                                             \
  do {                                                       \
    if (!(x)) {                                              \
      std::printf("line %d: %s\n", __LINE__, #x);            \
      return 1;                                              \
    }                                                        \
  } while (0)

struct Memory {
  std::map<void *, size_t> live;
  size_t limit = ~(size_t)0;
  int waits = 0, next = 1;
  size_t total() const {
    size_t n = 0;
    for (auto &b : live) n += b.second;
    return n;
  }
  bool allocate(void **p, size_t n) {
    if (total() + n > limit) return false;
    *p = reinterpret_cast<void *>((size_t)next++ << 12);
    live[*p] = n;
    return true;
  }
  void release(void *p) { live.erase(p) || (std::printf("released twice\n"), std::exit(1), 0); }
  bool wait() { return ++waits, true; }
};

int main() {
  const size_t MB = 1u << 20;
  {  // eager calls: one buffer, the stream waited for before the old one goes
    Memory m;
    ScratchBuffer b;
    void *p = nullptr, *q = nullptr;
    CHECK(mm::scratch_request(b, 100, false, m, &p) == Scratch::GROWN && m.live.count(p) && b.bytes == 2 * MB);
    CHECK(mm::scratch_request(b, 2 * MB, false, m, &q) == Scratch::READY && q == p);
    CHECK(mm::scratch_request(b, 2 * MB + 1, false, m, &q) == Scratch::GROWN && m.waits == 1);
    CHECK(m.live.size() == 1 && m.live.count(q) && m.live[q] == 4 * MB);
    mm::scratch_release(b, m);
    CHECK(m.live.empty());
  }
  {  // a buffer that a captured call was given outlives larger requests
    Memory m;
    ScratchBuffer b;
    void *p = nullptr, *q = nullptr;
    CHECK(mm::scratch_request(b, MB, false, m, &p) == Scratch::GROWN);
    CHECK(mm::scratch_request(b, MB, true, m, &q) == Scratch::READY && q == p);
    CHECK(mm::scratch_request(b, 5 * MB, true, m, &q) == Scratch::IN_CAPTURE);
    CHECK(mm::scratch_request(b, 5 * MB, false, m, &q) == Scratch::GROWN && q != p);
    CHECK(m.live.count(p) && m.live.count(q) && m.live[q] == 6 * MB);
    // not captured itself: it goes when it is outgrown
    void *r = nullptr;
    CHECK(mm::scratch_request(b, 9 * MB, false, m, &r) == Scratch::GROWN);
    CHECK(m.live.count(p) && !m.live.count(q) && m.live.count(r));
    mm::scratch_release(b, m);
    CHECK(m.live.empty());
  }
  {  // a graph for each size, smallest first: what is kept stays below the last
    Memory m;
    ScratchBuffer b;
    std::map<void *, int> given;
    for (int k = 1; k <= 300; ++k) {
      void *p = nullptr, *q = nullptr;
      CHECK(mm::scratch_request(b, k * MB, false, m, &p) != Scratch::FAILED);
      CHECK(mm::scratch_request(b, k * MB, true, m, &q) == Scratch::READY && q == p);
      given[p] = k;
      for (auto &g : given) CHECK(m.live.count(g.first));
      CHECK(m.total() < 2 * b.bytes);
    }
    mm::scratch_release(b, m);
    CHECK(m.live.empty());
  }
  {  // little memory: the exact size where twice does not fit, else a failure that loses nothing
    Memory m;
    m.limit = 11 * MB;
    ScratchBuffer b;
    void *p = nullptr, *q = nullptr;
    CHECK(mm::scratch_request(b, 4 * MB, false, m, &p) == Scratch::GROWN);
    CHECK(mm::scratch_request(b, 4 * MB, true, m, &p) == Scratch::READY);
    CHECK(mm::scratch_request(b, 5 * MB, false, m, &q) == Scratch::GROWN && m.live[q] == 6 * MB && m.live.count(p));
    CHECK(mm::scratch_request(b, 6 * MB, true, m, &q) == Scratch::READY);
    CHECK(mm::scratch_request(b, 7 * MB, false, m, &p) == Scratch::FAILED);
    CHECK(b.ptr == q && m.live.count(q));
    mm::scratch_release(b, m);
    CHECK(m.live.empty());
  }
  std::puts("ok");
}
