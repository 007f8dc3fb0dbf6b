// How much dynamic shared memory a kernel may be launched with: a limit per
// device that only grows, where calls of one kernel differ in what they need.
#pragma once

#include <atomic>
#include <cstddef>
#include <mutex>

namespace pa {

template <int DEVICES>
class SmemLimit {
 public:
  // At least `bytes` from now on.  set(bytes) sets the kernel's attribute; its
  // failure is this call's.  The lock keeps one thread's smaller limit from
  // being set behind another's larger one.
  template <typename Set>
  bool raise(int device, size_t bytes, Set set) {
    if (have_[device].load() >= bytes) return true;
    const std::lock_guard<std::mutex> hold(lock_);
    if (have_[device].load() >= bytes) return true;
    if (!set(bytes)) return false;
    have_[device].store(bytes);
    return true;
  }

 private:
  std::atomic<size_t> have_[DEVICES] = {};
  std::mutex lock_;
};

}  // namespace pa
