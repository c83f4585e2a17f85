// per_device.h -- a number that belongs to a device, worked out at its first use
// there.  Host code.
#pragma once

#include <atomic>

namespace moe {

class PerDevice {
 public:
  // *out = what ask(int*) gives on `device`, asked for until it gives a number
  // above 0 without an error.  Threads that ask at once get the same number.
  template <typename Ask>
  auto get(int device, int* out, Ask ask) -> decltype(ask(out)) {
    using Error = decltype(ask(out));
    const bool kept = device >= 0 && device < kDevices;
    *out = kept ? known_[device].load(std::memory_order_acquire) : 0;
    if (*out > 0) return Error(0);
    const Error e = ask(out);
    if (e == Error(0) && kept) known_[device].store(*out, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kDevices = 64;  // those beyond are asked every time
  std::atomic<int> known_[kDevices] = {};
};

}  // namespace moe
