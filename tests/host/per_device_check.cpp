// q4k_per_device.h on the host: one value per device, and a failed attempt is
// tried again.
#include <atomic>
#include <cstdio>
#include <thread>
#include <vector>

#include "q4k_per_device.h"

static int failures = 0;

static void check(bool ok, const char* what) {
    if (ok) return;
    std::printf("failed: %s\n", what);
    ++failures;
}

int main() {
    static q4k::PerDevice<int> values;
    int calls = 0, v = -1;
    auto fails = [&](int*) { ++calls; return cudaErrorMemoryAllocation; };
    auto makes = [&](int* out) { ++calls; *out = 7; return cudaSuccess; };
    check(values.get(3, &v, fails) == cudaErrorMemoryAllocation && v == -1, "the first attempt's error is returned");
    check(values.get(3, &v, makes) == cudaSuccess && v == 7, "the next call tries again");
    check(values.get(3, &v, fails) == cudaSuccess && v == 7 && calls == 2, "a made value is kept");
    check(values.get(4, &v, fails) == cudaErrorMemoryAllocation, "devices have their own");
    check(values.get(-1, &v, makes) == cudaErrorInvalidDevice && values.get(64, &v, makes) == cudaErrorInvalidDevice,
          "no such device");

    static q4k::PerDevice<int> shared;
    std::atomic<int> made{0}, wrong{0};
    std::vector<std::thread> threads;
    for (int i = 0; i < 8; ++i)
        threads.emplace_back([&] {
            int got = 0;
            for (int k = 0; k < 1000; ++k)
                if (shared.get(0, &got, [&](int* out) { *out = 40 + ++made; return cudaSuccess; }) != cudaSuccess || got != 41)
                    ++wrong;
        });
    for (auto& t : threads) t.join();
    check(made == 1 && wrong == 0, "threads share one value");
    if (failures == 0) std::printf("per device ok\n");
    return failures;
}
