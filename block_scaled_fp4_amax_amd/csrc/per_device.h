// per_device.h -- what has to be done once on each device of a process (plain C++).
#pragma once

#include <stdint.h>

#include <atomic>

namespace fp4q {

// Runs `set` (an int of 0 on success) unless it has succeeded on this device before.  Devices beyond 63
// run it every time.
struct OncePerDevice {
    std::atomic<uint64_t> done{0};

    template <class Set>
    int operator()(int device, Set set)
    {
        const uint64_t bit = device >= 0 && device < 64 ? (uint64_t)1 << device : 0;
        if (done.load(std::memory_order_acquire) & bit) return 0;
        const int st = set();
        if (st == 0) done.fetch_or(bit, std::memory_order_release);
        return st;
    }
};

}  // namespace fp4q
