// What a query says of a device, kept per device: the answers of one are not those of another, and a
// query that failed is made again at the next call.
#pragma once
#include <atomic>

namespace moe_host {

// Whether this process sees one GPU alone; count(&n): the query, true on success.  Loads that a cluster shares
// (TMA multicast) are for such runs only: where there are several GPUs every block loads its own tiles.
template <typename Query>
bool sole_device(Query count) {
  int n = 0;
  return count(&n) && n == 1;
}

template <int N>
class PerDevice {
 public:
  // Value i of `device` (0 <= i < N): query() once, > 0 on success; `fallback`, not kept, if it fails.
  // A device outside the table is asked every time.
  template <typename Query>
  int get(int device, int i, int fallback, Query query) {
    const bool known = device >= 0 && device < kDevices;
    if (known) {
      const int v = v_[device][i].load(std::memory_order_relaxed);
      if (v > 0) return v;
    }
    const int v = query();
    if (v <= 0) return fallback;
    if (known) v_[device][i].store(v, std::memory_order_relaxed);
    return v;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> v_[kDevices][N] = {};
};

}  // namespace moe_host
