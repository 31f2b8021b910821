// resident.h -- how many clusters of a kernel run at once on each device: asked for once, by
// whichever host thread comes first (the answer is the same for all).
#pragma once

#include <atomic>

namespace lnq {

class ResidentClusters {
public:
    // query() gives the count, 0 if it failed; then the call uses `fallback`, and the next one asks
    // again.
    template <typename Query>
    int get(int device, int fallback, Query query)
    {
        const bool kept = device >= 0 && device < kDevices;
        int n = kept ? count_[device].load(std::memory_order_relaxed) : 0;
        if (n == 0) {
            n = query();
            if (n <= 0)
                return fallback;
            if (kept)
                count_[device].store(n, std::memory_order_relaxed);
        }
        return n;
    }

private:
    static constexpr int kDevices = 64;
    std::atomic<int> count_[kDevices] = {};
};

}  // namespace lnq
