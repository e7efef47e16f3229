// How many clusters of a kernel a device holds at once, asked once per kernel,
// device and cluster size (plain C++: the question itself is the caller's).
#pragma once

#include <atomic>

namespace smoe {

class ClusterTable {
public:
    // The answer for clusters of csize (2, 4 or 8) CTAs on device dev, from
    // query() the first time.  Below 1 the query has failed: the answer is 0, and
    // the next call asks again.
    template <typename Query>
    int get(int dev, int csize, Query query)
    {
        if (dev < 0 || dev >= kDevices) return 0;
        std::atomic<int> &slot = kept_[dev][csize == 2 ? 0 : (csize == 4 ? 1 : 2)];
        int n = slot.load(std::memory_order_relaxed);
        if (n > 0) return n;
        n = query();
        if (n < 1) return 0;
        slot.store(n, std::memory_order_relaxed);
        return n;
    }

private:
    static constexpr int kDevices = 64;
    std::atomic<int> kept_[kDevices][3] = {};
};

// The table of one kernel: of the function itself, since the instantiations of a
// kernel template share one type.
template <auto Kernel>
ClusterTable &cluster_table()
{
    static ClusterTable table;
    return table;
}

}  // namespace smoe
