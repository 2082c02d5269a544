// State that belongs to a device, kept once for each (host code).
#pragma once

#include <atomic>
#include <mutex>

namespace mla {

constexpr int kMaxDevices = 64;  // the library refuses others

// A setup that every device needs once, such as a kernel's attributes (a process
// may call the library on several devices).  A setup that fails is not
// remembered: the next call on that device runs it again.
class OncePerDevice {
 public:
  // setup() returns 0 for success.  0, or what setup() returned.
  template <class Setup>
  auto run(int device, Setup setup) -> decltype(setup()) {
    using Status = decltype(setup());
    std::atomic<bool>& done = done_[device];
    if (done.load(std::memory_order_acquire)) return Status(0);
    std::lock_guard<std::mutex> lock(mu_);
    if (done.load(std::memory_order_relaxed)) return Status(0);
    const Status status = setup();
    if (status == Status(0)) done.store(true, std::memory_order_release);
    return status;
  }

 private:
  std::mutex mu_;
  std::atomic<bool> done_[kMaxDevices] = {};
};

}  // namespace mla
