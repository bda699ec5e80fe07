// A value that belongs to a device (how much of a kernel fits there, and that its
// limits have been set there), made on the first use on each: a process may have
// handles on several.
#pragma once

#include <cuda_runtime.h>

#include <mutex>

namespace rcu {

template <typename V>
class PerDevice {
 public:
  // The current device's value, from make() at first.
  template <typename Make>
  V here(Make make) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= MAX) return make();
    std::call_once(made_[dev], [&] { of_[dev] = make(); });
    return of_[dev];
  }

 private:
  static constexpr int MAX = 64;  // devices beyond it make theirs every time
  std::once_flag made_[MAX];
  V of_[MAX] = {};
};

}  // namespace rcu
