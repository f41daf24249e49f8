// The dynamic shared-memory limit that each kernel has been given on each device (host only).
#pragma once

#include <cstddef>
#include <cstdint>

namespace moe {

// Open addressing over a fixed number of slots, so that nothing is allocated.  The library has about
// 110 kernels that ask for a limit, each once per device: kSlots holds them on nine devices.  A full table
// is no error: find() then has no slot to give and the caller sets the limit anew.
class SmemTable {
 public:
  struct Entry {
    const void* func;
    int dev;
    size_t bytes;    // 0: none yet
  };
  static constexpr size_t kSlots = 1024;

  // The entry of (func, dev), made if it is new; nullptr when the table is full.
  Entry* find(const void* func, int dev) {
    const uint64_t key = reinterpret_cast<uintptr_t>(func) / 16 + static_cast<uint64_t>(dev) * 0x9E3779B97F4A7C15ull;
    const size_t first = static_cast<size_t>((key * 0x9E3779B97F4A7C15ull) >> 54);
    for (size_t i = 0; i < kSlots; ++i) {
      Entry& e = slots_[(first + i) % kSlots];
      if (e.func == nullptr) {
        e.func = func;
        e.dev = dev;
        return &e;
      }
      if (e.func == func && e.dev == dev) return &e;
    }
    return nullptr;
  }

 private:
  Entry slots_[kSlots] = {};
};

}  // namespace moe
