// sv_device.cuh -- host-side set-up that a device needs once (plain C++).
#pragma once
#include <atomic>

namespace sv {

// Runs a set-up once for each device: it returns 0 when it took, and is tried again at the
// next call otherwise. (Two threads may both run it: it must not matter how often it runs.)
class OncePerDevice {
 public:
  template <typename F>
  int run(int dev, F set) {
    const bool known = dev >= 0 && dev < MAX;
    if (known && done_[dev].load(std::memory_order_acquire)) return 0;
    const int e = set();
    if (known && e == 0) done_[dev].store(true, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int MAX = 64;  // devices beyond are set up at every call
  std::atomic<bool> done_[MAX] = {};
};

}  // namespace sv
