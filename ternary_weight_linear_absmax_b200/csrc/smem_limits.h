// Which dynamic shared-memory limit each kernel has been given on each device.
// Plain host code; the caller holds a lock.
#pragma once

#include <cstddef>
#include <cstdint>

namespace bl {

// A limit holds for a kernel, not for a launch: a call that lowered it between
// another thread's call and its launch would make that launch fail. So there is
// one entry per kernel and device, and a limit only ever rises.
class SmemLimits {
 public:
  // Makes sure that `fn` may have `bytes` on `dev`; set(bytes) is called where the
  // limit has to rise, and returns whether it did. False: set failed, or there
  // are more kernels and devices than entries.
  template <typename Set>
  bool ensure(const void* fn, int dev, size_t bytes, Set&& set) {
    const uintptr_t mix = (reinterpret_cast<uintptr_t>(fn) >> 4) * 0x9E3779B97F4A7C15ull + (uintptr_t)dev * 131;
    for (size_t i = 0; i < kEntries; ++i) {
      Entry& e = table_[((mix >> 20) + i) % kEntries];
      if (e.fn != nullptr && (e.fn != fn || e.dev != dev)) continue;
      if (e.fn != nullptr && e.bytes >= bytes) return true;
      if (!set(bytes)) return false;
      e = Entry{fn, dev, bytes};
      return true;
    }
    return false;
  }

  static constexpr size_t kEntries = 4096;

 private:
  struct Entry {
    const void* fn;
    int dev;
    size_t bytes;
  };
  Entry table_[kEntries] = {};
};

}  // namespace bl
