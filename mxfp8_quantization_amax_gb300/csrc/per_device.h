// per_device.h -- what is set or found out once for each device of a process: a
// kernel's attributes and its occupancy belong to the device that was current.
#pragma once

#include <mutex>

namespace fp8q {

// A value for each device.  get() makes it with make(T*), true on success, when
// a device first asks; what failed is not kept, and the next call tries again.
template <typename T>
class PerDevice {
 public:
  static constexpr int kDevices = 64;  // beyond them every call makes its own

  template <typename F>
  bool get(int device, T* out, F make) {
    if (device < 0 || device >= kDevices) return make(out);
    std::lock_guard<std::mutex> lock(mu_);
    if (!have_[device]) {
      if (!make(&value_[device])) return false;
      have_[device] = true;
    }
    *out = value_[device];
    return true;
  }

  // Shows change(T*) the device's value, T{} at first, alone.
  template <typename F>
  void update(int device, F change) {
    if (device < 0 || device >= kDevices) {
      T v{};
      return change(&v);
    }
    std::lock_guard<std::mutex> lock(mu_);
    change(&value_[device]);
  }

 private:
  std::mutex mu_;
  bool have_[kDevices] = {};
  T value_[kDevices] = {};
};

}  // namespace fp8q
