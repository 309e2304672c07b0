// A setting that belongs to one device's copy of a kernel (its shared-memory limit),
// made on a device's first call.  Host threads may make it at the same time; a failure
// is returned and tried again by the next call.
#pragma once

#include <atomic>

namespace moe {

class OncePerDevice {
 public:
  // f's result, whose zero is success, or success where f has succeeded on `dev` before
  template <class F>
  auto operator()(int dev, F&& f) -> decltype(f()) {
    using R = decltype(f());
    const bool known = dev >= 0 && dev < kDevices;
    if (known && done_[dev].load(std::memory_order_acquire)) return R{};
    const R rc = f();
    if (known && rc == R{}) done_[dev].store(true, std::memory_order_release);
    return rc;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<bool> done_[kDevices]{};
};

}  // namespace moe
