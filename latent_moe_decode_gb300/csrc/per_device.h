// Counts that are asked of each device once (plain C++).
#pragma once

#include <atomic>

namespace moe {

constexpr int kMaxKnownDevices = 64;

// get(device, i, ask): what ask() gave for the i-th of N counts on that device. A negative answer (the query failed)
// is passed on and not kept: the next call asks again.
template <int N>
class PerDevice {
  std::atomic<int> known_[kMaxKnownDevices][N] = {};  // 0: not asked; else the count and one

 public:
  template <typename Ask>
  int get(int device, int i, Ask ask) {
    if (device < 0 || device >= kMaxKnownDevices || i < 0 || i >= N) return -1;
    const int k = known_[device][i].load(std::memory_order_relaxed);
    if (k != 0) return k - 1;
    const int n = ask();
    if (n >= 0) known_[device][i].store(n + 1, std::memory_order_relaxed);
    return n;
  }
};

}  // namespace moe
