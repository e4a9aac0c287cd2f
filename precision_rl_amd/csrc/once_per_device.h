// Something to do once on each device of the process (host only, no HIP).
#pragma once

#include <stdint.h>

#include <atomic>

namespace w4a4 {

// Calls set() for a device until it has returned true there; threads may call
// it at the same time (set() can then run twice).  Devices past the 64th are
// set at every call.
class OncePerDevice {
 public:
  template <class F>
  bool operator()(int device, F set) {
    const uint64_t bit = device >= 0 && device < 64 ? uint64_t{1} << device : 0;
    if (done_.load(std::memory_order_acquire) & bit) return true;
    if (!set()) return false;
    done_.fetch_or(bit, std::memory_order_release);
    return true;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

}  // namespace w4a4
