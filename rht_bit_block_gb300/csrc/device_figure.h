// A figure of each device that is asked for once and kept.
#pragma once

#include <atomic>

namespace ufp4 {

// Several host threads may need the figure at the same time: each that finds
// none asks, and what they keep is the same.  Figures are positive; 0 (a
// failed query, or a device index out of range) is not kept.
class DeviceFigure {
public:
    template <typename Ask>
    int get(int device, Ask ask) {
        if (device < 0 || device >= kDevices) return 0;
        int v = kept_[device].load(std::memory_order_relaxed);
        if (v > 0) return v;
        v = ask();
        if (v > 0) kept_[device].store(v, std::memory_order_relaxed);
        return v > 0 ? v : 0;
    }

private:
    static constexpr int kDevices = 64;
    std::atomic<int> kept_[kDevices] = {};
};

}  // namespace ufp4
