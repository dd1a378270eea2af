// The kernels whose dynamic shared-memory limit has been raised, by device.
// Plain C++, so that a host test can build it.
#pragma once

#include <new>
#include <unordered_map>

namespace abw {

// Holds any number of kernels: some hundred instances raise their limit on each
// device that they run on.  An entry counts in the context it was made in alone.
// Not synchronised.
class SmemLimits {
 public:
  // The limit of `func` on device `dev` is at least `bytes` in context `ctx` (0: unknown).
  bool reaches(int dev, const void *func, unsigned long long ctx, int bytes) const {
    const auto d = devices_.find(dev);
    if (ctx == 0 || d == devices_.end()) return false;
    const auto f = d->second.find(func);
    return f != d->second.end() && f->second.ctx == ctx && f->second.bytes >= bytes;
  }
  // It has been raised to `bytes`.  Without memory for the entry it is raised again at the next call.
  void raised(int dev, const void *func, unsigned long long ctx, int bytes) {
    try {
      devices_[dev][func] = Entry{ctx, bytes};
    } catch (const std::bad_alloc &) {
    }
  }

 private:
  struct Entry {
    unsigned long long ctx;
    int bytes;
  };
  std::unordered_map<int, std::unordered_map<const void *, Entry>> devices_;
};

}  // namespace abw
