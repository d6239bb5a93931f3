// How a scratch buffer of the library grows, apart from CUDA (the memory calls
// come as `Mem`), so that the rules can be tested on the host.
#pragma once

#include <algorithm>
#include <cstddef>
#include <vector>

namespace mm {

struct ScratchBuffer {
  void *ptr = nullptr;
  size_t bytes = 0;
  bool captured = false;      // handed to a call that was captured into a graph
  std::vector<void *> kept;   // outgrown buffers that graphs still hold
};

enum class Scratch { READY, GROWN, IN_CAPTURE, FAILED };

// A pointer to at least `need` bytes in *out: READY, or GROWN where the buffer
// is new (its contents undefined).  IN_CAPTURE: it would have to grow while the
// stream is captured, which memory calls would end.  FAILED: a Mem call failed.
//   bool Mem::allocate(void **, size_t), void Mem::release(void *),
//   bool Mem::wait()  the stream's queued work, which may read the old buffer
// A graph keeps the address that a captured call was given, so a buffer that was
// handed to one is never given back before the library shuts down.  Its successor
// has at least twice its size (where memory allows), so what is kept so stays
// below the buffer in use.
template <typename Mem>
Scratch scratch_request(ScratchBuffer &b, size_t need, bool capturing, Mem &&mem, void **out) {
  static constexpr size_t kUnit = (size_t)2 << 20;
  const auto whole = [](size_t n) { return std::max(kUnit, (n + kUnit - 1) / kUnit * kUnit); };
  if (b.ptr && b.bytes >= need) {
    b.captured |= capturing;
    *out = b.ptr;
    return Scratch::READY;
  }
  if (capturing) return Scratch::IN_CAPTURE;
  size_t size = whole(need);
  void *p = nullptr;
  if (b.ptr && b.captured) {
    const size_t twice = std::max(size, 2 * b.bytes);
    if (mem.allocate(&p, twice)) size = twice;
    else if (twice == size || !mem.allocate(&p, size)) return Scratch::FAILED;
    b.kept.push_back(b.ptr);
  } else {
    if (b.ptr) {
      if (!mem.wait()) return Scratch::FAILED;
      mem.release(b.ptr);
      b.ptr = nullptr;
      b.bytes = 0;
    }
    if (!mem.allocate(&p, size)) return Scratch::FAILED;
  }
  b.ptr = p;
  b.bytes = size;
  b.captured = false;
  *out = p;
  return Scratch::GROWN;
}

template <typename Mem>
void scratch_release(ScratchBuffer &b, Mem &&mem) {
  for (void *p : b.kept) mem.release(p);
  if (b.ptr) mem.release(b.ptr);
  b = ScratchBuffer{};
}

}  // namespace mm
