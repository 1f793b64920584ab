// Setting up once for each device of a process. Not part of the C ABI; no CUDA headers.
#pragma once
#include <atomic>
#include <cstdint>

namespace mlora {

// Runs set() (0 on success) unless it has succeeded for this device before; a failure is returned and not kept. Devices from
// 64 on are set up at every call. Two threads may both run it for a device's first call.
template <class Error, class Set>
Error once_per_device(std::atomic<uint64_t>& done, int device, Set set) {
  const uint64_t bit = device >= 0 && device < 64 ? uint64_t(1) << device : 0;
  if (done.load(std::memory_order_acquire) & bit) return Error(0);
  const Error e = set();
  if (e == Error(0)) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace mlora
