// The dynamic shared-memory limit that each kernel has been given on each device (host only).
#pragma once

#include <cstddef>
#include <cstdint>

namespace moe {

// Open addressing over a fixed number of slots, so that nothing is allocated.  The library has about
// 370 kernels that may ask for a limit (260 of them the normalisation's, by types and sizes), each once per device:
// kSlots holds them on eleven devices.  A full table is no error: find() then has no slot to give, and the limit that
// is in force is asked for at each call (raise_limit).
class SmemTable {
 public:
  struct Entry {
    const void* func;
    int dev;
    size_t bytes;    // 0: none yet
  };
  static constexpr int kSlotBits = 12;
  static constexpr size_t kSlots = size_t{1} << kSlotBits;

  // The entry of (func, dev), made if it is new; nullptr when the table is full.
  Entry* find(const void* func, int dev) {
    const uint64_t key = reinterpret_cast<uintptr_t>(func) / 16 + static_cast<uint64_t>(dev) * 0x9E3779B97F4A7C15ull;
    const size_t first = static_cast<size_t>((key * 0x9E3779B97F4A7C15ull) >> (64 - kSlotBits));
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

// Raises a kernel's limit to `bytes` and never lowers it: another thread may be about to launch with what was set
// before.  entry: the kernel's, or nullptr from a full table.  get(&bytes) and set(bytes) are the driver's calls, 0
// from either is success.
template <typename Error, typename Get, typename Set>
Error raise_limit(SmemTable::Entry* entry, size_t bytes, const Get& get, const Set& set) {
  size_t held = 0;
  if (entry) {
    held = entry->bytes;
  } else {
    const Error err = get(&held);
    if (err != Error{}) return err;
  }
  if (held >= bytes) return Error{};
  const Error err = set(bytes);
  if (err == Error{} && entry) entry->bytes = bytes;
  return err;
}

}  // namespace moe
