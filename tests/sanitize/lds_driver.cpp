// lds_driver.cpp — allow_lds (csrc/launch.hpp) over several devices and host
// threads: every thread may launch only after its own device has been asked,
// which happens again after a failure and otherwise not. The runtime's two calls
// are the ones below. Built with ThreadSanitizer for the host by
// tests/test_lds_host.py; no GPU is touched.
#include <atomic>
#include <cstdio>
#include <thread>
#include <vector>

#include "../../weight_only_quantized_qgemv_amd/csrc/launch.hpp"

static thread_local int t_device = 0;
static std::atomic<int> asked[4];
static std::atomic<bool> failing{false};

extern "C" hipError_t hipGetDevice(int* dev)
{
    *dev = t_device;
    return hipSuccess;
}
extern "C" hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int bytes)
{
    if (failing.load() || bytes != 98304)
        return hipErrorInvalidValue;
    asked[t_device].fetch_add(1);
    return hipSuccess;
}

int main()
{
    int kernel = 0, failures = 0;
    std::atomic<uint64_t> done{0};
    failing = true;
    if (qp::allow_lds(done, &kernel, 98304) == hipSuccess || done.load() != 0)
        ++failures;
    failing = false;
    std::atomic<int> early{0};
    std::vector<std::thread> threads;
    for (int i = 0; i < 16; ++i)
        threads.emplace_back([&, i] {
            t_device = i % 4;
            for (int j = 0; j < 100; ++j)
                if (qp::allow_lds(done, &kernel, 98304) != hipSuccess || asked[t_device].load() == 0)
                    early.fetch_add(1);
        });
    for (auto& t : threads)
        t.join();
    for (auto& a : asked)
        failures += a.load() < 1 || a.load() > 4;   // four threads a device may ask at once
    const int before = asked[0].load();
    if (qp::allow_lds(done, &kernel, 98304) != hipSuccess || asked[0].load() != before)
        ++failures;
    failures += early.load();
    std::printf(failures ? "FAIL %d\n" : "asked once per device\n", failures);
    return failures != 0;
}
