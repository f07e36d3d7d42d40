// Work that a process does once per device before its first launch of a kernel
// (function attributes), from whichever host thread comes first.
#pragma once

#include <atomic>
#include <mutex>

namespace w4a16 {

constexpr int kMaxDevices = 64;

class OncePerDevice {
  public:
    // Runs prepare() unless it has succeeded for `dev` (0 <= dev < kMaxDevices) before; its result (0: success).
    // A call that finds it done takes no lock and sees all that prepare() wrote.
    template <class F>
    int run(int dev, F&& prepare) {
        if (done_[dev].load(std::memory_order_acquire)) return 0;
        std::lock_guard<std::mutex> lock(mu_);
        if (done_[dev].load(std::memory_order_relaxed)) return 0;
        const int rc = prepare();
        if (rc == 0) done_[dev].store(true, std::memory_order_release);
        return rc;
    }

  private:
    std::mutex mu_;
    std::atomic<bool> done_[kMaxDevices] = {};
};

}  // namespace w4a16
