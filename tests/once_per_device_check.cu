// Host check of csrc/once_per_device.h: prints "ok" when each device gets its step once, a failed
// step is taken again by the next call, one device's failure is not another's, and devices out of
// range are refused without a step.  Built and run on the host by test_once_per_device.py.
#include <cstdio>
#include <thread>
#include <vector>

#include "once_per_device.h"

using namespace relation;

int main() {
    OncePerDevice once;
    int taken[64] = {};
    auto on = [&](int device, cudaError_t result) {
        return once.run(device, [&] { return ++taken[device], result; });
    };
    if (on(0, cudaErrorInvalidValue) != cudaErrorInvalidValue || taken[0] != 1) return std::printf("the error\n"), 1;
    if (on(1, cudaSuccess) != cudaSuccess || taken[1] != 1) return std::printf("another device\n"), 1;
    if (on(0, cudaSuccess) != cudaSuccess || taken[0] != 2) return std::printf("after an error\n"), 1;
    for (int k = 0; k < 3; ++k)
        if (on(0, cudaErrorInvalidValue) != cudaSuccess || taken[0] != 2) return std::printf("again\n"), 1;
    if (on(63, cudaSuccess) != cudaSuccess || taken[63] != 1) return std::printf("the last device\n"), 1;
    for (int device : {-1, 64})
        if (once.run(device, [] { return std::printf("a step\n"), cudaSuccess; }) != cudaErrorInvalidDevice)
            return std::printf("device %d\n", device), 1;
    std::vector<std::thread> threads;
    for (int k = 0; k < 8; ++k) threads.emplace_back([&] { on(5, cudaSuccess); });
    for (auto& t : threads) t.join();
    if (taken[5] != 1) return std::printf("threads: %d\n", taken[5]), 1;
    std::printf("ok\n");
    return 0;
}
