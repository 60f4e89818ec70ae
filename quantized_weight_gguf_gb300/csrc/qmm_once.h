// qmm_once.h -- what is set up once per device (a kernel's shared-memory limit).
// Host code without CUDA headers.
#pragma once

#include <atomic>
#include <cstdint>

namespace qmm {

// `run` calls set() unless it has returned `ok` for this device before, and
// returns its status. Only success is remembered: a failure is tried again by
// the next call. Two threads may both call set() the first time.
class OncePerDevice {
  public:
    template <class Status, class Set>
    Status run(int device, Status ok, Set set) {
        const uint64_t bit = (uint64_t)1 << (device & 63);
        if (done_.load(std::memory_order_acquire) & bit) return ok;
        const Status st = set();
        if (st == ok) done_.fetch_or(bit, std::memory_order_release);
        return st;
    }

  private:
    std::atomic<uint64_t> done_{0};  // a bit per device; device_info takes indexes below 64 only
};

}  // namespace qmm
