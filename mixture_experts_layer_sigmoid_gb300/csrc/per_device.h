// per_device.h -- what the first call of a kernel on a device works out and later ones reuse.
#pragma once
#include <atomic>

namespace moe {

constexpr int kMaxDevices = 64;        // slots; on further devices every call is a first one

// The number (not 0) that `first` gives on device `dev`. Only a success is kept: after an error,
// which may be a passing one, the next call tries again.
template <typename Error, typename First>
Error per_device(std::atomic<int> (&slots)[kMaxDevices], int dev, First first, int* out)
{
    int n = dev < kMaxDevices ? slots[dev].load(std::memory_order_acquire) : 0;
    if (n == 0) {
        const Error e = first(&n);
        if (e != Error{}) return e;
        if (dev < kMaxDevices) slots[dev].store(n, std::memory_order_release);
    }
    *out = n;
    return Error{};
}

}  // namespace moe
