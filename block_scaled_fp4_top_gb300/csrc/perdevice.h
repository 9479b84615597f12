// A host value that belongs to a device (a kernel attribute that was set, an occupancy), kept once it is known.
#pragma once

#include <atomic>

namespace fp4moe {

constexpr int kMaxDevices = 64;

// `ask` answers for the current device: a positive value, or 0 where a call failed. A failure is not kept, so a later
// call asks again. Threads that ask at the same time get the same answer.
struct PerDevice {
  std::atomic<int> known[kMaxDevices] = {};

  template <typename Ask>
  int get(int device, Ask ask) {
    if (device < 0 || device >= kMaxDevices) return 0;
    int v = known[device].load(std::memory_order_acquire);
    if (v > 0) return v;
    v = ask();
    if (v > 0) known[device].store(v, std::memory_order_release);
    return v;
  }
};

}  // namespace fp4moe
