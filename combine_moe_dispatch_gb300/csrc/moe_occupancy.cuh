// moe_occupancy.cuh -- what the driver answered about each kernel's resident blocks,
// kept per kernel, device, block size and shared memory.  Host code alone.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <mutex>

namespace moe {

// The library has about 140 kernels, each launched one way: a device's worth is
// found in one or two probes, and there is room for several devices.  (A list of
// 64 was full after one process had used the norm's and the products' forms;
// every further kernel's call then asked the driver.)  Entries are never removed;
// when three quarters of the places are taken new kernels are asked about each time.
class OccupancyTable {
 public:
  static constexpr int kPlaces = 2048;       // a power of two

  // The kept answer, or ask()'s.
  template <class Ask>
  int get(const void *kern, int dev, int threads, size_t smem, const Ask &ask) {
    std::lock_guard<std::mutex> lock(mu_);
    uint64_t h = (uint64_t)(uintptr_t)kern * 0x9E3779B97F4A7C15ull;
    h = (h ^ (uint64_t)dev ^ ((uint64_t)threads << 8) ^ ((uint64_t)smem << 24)) * 0x9E3779B97F4A7C15ull;
    int i = (int)(h >> 53);
    for (; place_[i].kern; i = (i + 1) & (kPlaces - 1))
      if (place_[i].kern == kern && place_[i].dev == dev && place_[i].threads == threads &&
          place_[i].smem == smem)
        return place_[i].blocks;
    const int blocks = ask();
    if (used_ < kPlaces / 4 * 3) {
      place_[i] = Entry{kern, dev, threads, smem, blocks};
      ++used_;
    }
    return blocks;
  }

 private:
  struct Entry {
    const void *kern;                        // null: free
    int dev, threads;
    size_t smem;
    int blocks;
  };
  Entry place_[kPlaces] = {};
  int used_ = 0;
  std::mutex mu_;
};
static_assert(OccupancyTable::kPlaces == 1 << (64 - 53), "a place is the upper bits of the product");

}  // namespace moe
