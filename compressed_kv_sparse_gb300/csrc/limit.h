// A limit per device that launches need raised (a kernel's dynamic shared memory), kept by host
// threads together: it is set under a lock and only ever to more, so that a launch finds at
// least what it asked for, whatever the others asked for meanwhile. Host code without CUDA.
#pragma once
#include <atomic>
#include <cstddef>
#include <mutex>

namespace ds4a {

class RaisedLimit {
 public:
  static constexpr int kDevices = 64;
  // set(bytes): sets the limit of the current device, `dev` (0 .. kDevices - 1); its result (0:
  // done) is the call's.
  template <typename Set>
  auto raise(int dev, size_t bytes, Set set) -> decltype(set(bytes)) {
    std::atomic<size_t> &done = done_[dev];
    if (done.load(std::memory_order_acquire) >= bytes) return {};
    std::lock_guard<std::mutex> lock(mu_);
    if (done.load(std::memory_order_relaxed) >= bytes) return {};
    const auto e = set(bytes);
    if (!e) done.store(bytes, std::memory_order_release);
    return e;
  }

 private:
  std::mutex mu_;
  std::atomic<size_t> done_[kDevices] = {};
};

}  // namespace ds4a
