// per_device.h -- what a kernel's first launch on a device sets up or finds out,
// kept for the later ones.
#pragma once
#include <atomic>

namespace fp8ll {

// One value per device, safe for any number of host threads: as a static object,
// all values start unknown.
class PerDevice {
public:
    // The device's value, 0 or more: what find() returns on the first use.  A
    // negative one is an error: it is returned and not kept.  Threads that come
    // first together each call find(), which has to give the same value every time.
    template <typename F>
    int get(int device, F&& find) {
        if (device < 0 || device >= kDevices) return -3;
        const int known = value_[device].load(std::memory_order_acquire);
        if (known != 0) return known - 1;
        const int v = find();
        if (v >= 0) value_[device].store(v + 1, std::memory_order_release);
        return v;
    }

private:
    static constexpr int kDevices = 64;
    std::atomic<int> value_[kDevices];  // value + 1; 0: unknown
};

}  // namespace fp8ll
