// The 8-bit products' plan of a launch, apart from CUDA.
#pragma once

#include <atomic>

namespace coc {

// A count that is asked for once; none is an answer too.
class KnownCount {
public:
    bool get(int* n) const {
        const int v = held_.load(std::memory_order_acquire);
        *n = v - 1;
        return v > 0;
    }
    void set(int n) { held_.store(n + 1, std::memory_order_release); }

private:
    std::atomic<int> held_{0};      // the count + 1; 0: not asked yet
};

// Ranges that a tile's contraction of `total` runs is cut into: the most, up to
// 8, whose clusters all find an SM for every block.  room(k, &n): how many
// clusters of k blocks run at once; 0 or an error.
template <class Room>
auto f8_ranges(long long tiles, int total, int sm_count, Room&& room, int* ranges) -> decltype(room(1, ranges)) {
    *ranges = 1;
    for (int k = 2; k <= 8 && k <= total && tiles * k <= sm_count; ++k) {
        int n = 0;
        if (const auto e = room(k, &n)) return e;
        if (tiles <= n) *ranges = k;
    }
    return {};
}

}  // namespace coc
