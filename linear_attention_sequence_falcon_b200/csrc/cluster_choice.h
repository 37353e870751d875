// cluster_choice.h -- how many blocks of the gated recurrence's kernels form a
// cluster (host code without CUDA calls; scan_parts.cuh asks the device).
#pragma once

#include <mutex>

namespace falcon {
namespace scan {

constexpr int kMaxCluster = 16;  // beyond 8: not portable, allowed per kernel

// What the device answers: clusters held at once (0: this size does not fit),
// or, below 0, that it could not be asked.
constexpr int kNotAsked = -1;

// The answers so far, per (kernel, device, size).  A question that failed is
// asked again.
class ClustersHeld {
    static constexpr int kDevices = 16, kKernels = 64;
    std::mutex guard_;
    struct {
        const void *kernel;
        int known[kDevices][kMaxCluster + 1];  // the answer + 1
    } kept_[kKernels] = {};

public:
    template <typename Ask> int get(const void *kernel, int device, int cs, Ask ask) {
        std::lock_guard<std::mutex> lock(guard_);
        int *slot = nullptr;
        for (auto &e : kept_) {
            if (e.kernel == nullptr) e.kernel = kernel;
            if (e.kernel == kernel) {
                if (device >= 0 && device < kDevices) slot = &e.known[device][cs];
                break;
            }
        }
        if (slot && *slot) return *slot - 1;
        const int held = ask();
        if (slot && held >= 0) *slot = held + 1;
        return held;
    }
};

// The cluster's size: blocks walk steps = tiles/cs tiles each, in as many waves
// as the device needs for all units' clusters.  A step takes a latency (its
// exchange) and a share of the SM that grows with the blocks on it, a wave its
// start: waves x (steps x (1.5 + blocks per SM) + 4.5) fits what was measured
// over sizes 1 to 16 of six shapes; the least, the smallest size of equals.
// Least waves x steps took 5 for the forward pass at 8x2048x768 (21.1 us; 4
// takes 19.3); without the waves' start the backward pass at 16x1024x1024 took
// 16 (69 us; 3 takes 39).  held(cs): clusters at once; a size of which none
// fits is not taken, blocks without neighbours always are.
template <typename Held> int choose_cluster(long long units, int tiles, Held held) {
    int best = 1;
    long long cost = 0;
    for (int cs = 1; cs <= kMaxCluster && cs <= tiles; ++cs) {
        int fit = held(cs);
        if (fit < 1) {
            if (cs > 1) continue;
            fit = 1;
        }
        const long long waves = (units + fit - 1) / fit;
        const long long blocks = (units < fit ? units : fit) * cs;  // at once
        const long long here = waves * ((tiles + cs - 1) / cs * (3 * 148 + 2 * blocks) + 9 * 148);
        if (cs == 1 || here < cost) { best = cs; cost = here; }
    }
    return best;
}

}  // namespace scan
}  // namespace falcon
