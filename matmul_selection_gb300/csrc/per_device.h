// What is worked out once for each device and kept: kernel attributes, which
// belong to a device's copy of a kernel, and occupancies.
#pragma once

#include <atomic>
#include <mutex>

namespace mm {

// get() gives the device's value; the first call on a device makes it with
// make(T *) -> status, 0 for success.  A failure is returned and not kept: the next
// call tries again.  Devices past kDevices are made on every call.
template <typename T>
class PerDevice {
  static constexpr int kDevices = 64;
  struct Slot {
    std::atomic<bool> ready{false};
    std::mutex mu;
    T value{};
  } slots_[kDevices];

 public:
  template <typename Make>
  auto get(int device, T *out, Make &&make) -> decltype(make(out)) {
    if (device < 0 || device >= kDevices) return make(out);
    Slot &s = slots_[device];
    if (!s.ready.load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> lk(s.mu);
      if (!s.ready.load(std::memory_order_relaxed)) {
        T v{};
        const auto st = make(&v);
        if (st != 0) return st;
        s.value = v;
        s.ready.store(true, std::memory_order_release);
      }
    }
    *out = s.value;
    return {};
  }
};

}  // namespace mm
