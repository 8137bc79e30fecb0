// q4k_per_device.h -- values made on first need, once per device, and kept.
#pragma once

#include <atomic>
#include <driver_types.h>
#include <mutex>

namespace q4k {

// A failed attempt is not kept: its caller gets the error, the next call tries
// again (memory may be free by then). Callers on several threads get one value.
template <class T>
class PerDevice {
public:
    // The value of device `dev`, made by make(T*) -> cudaError_t.
    template <class Make>
    cudaError_t get(int dev, T* out, Make make) {
        if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
        Entry& entry = entries_[dev];
        if (!entry.made.load(std::memory_order_acquire)) {
            std::lock_guard<std::mutex> lock(entry.mutex);
            if (!entry.made.load(std::memory_order_relaxed)) {
                T value{};
                const cudaError_t e = make(&value);
                if (e != cudaSuccess) return e;
                entry.value = value;
                entry.made.store(true, std::memory_order_release);
            }
        }
        *out = entry.value;
        return cudaSuccess;
    }

private:
    static constexpr int kDevices = 64;
    struct Entry {
        std::mutex mutex;
        std::atomic<bool> made{false};
        T value{};
    };
    Entry entries_[kDevices];
};

}  // namespace q4k
