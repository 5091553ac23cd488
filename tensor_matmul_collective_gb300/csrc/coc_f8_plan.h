// The 8-bit products' plan of a launch, apart from CUDA.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstdint>

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

// Tiles of CTA pairs or slabs of weight rows, by the time either takes for its
// rounds of k-blocks (us, measured): a tile 6 and 0.31 a k-block (summed over
// ranks 7, gated 8), a slab of 128 rows (gated: of 64) 5 and 0.28 (0.39) where it
// has an SM to itself, 0.5 (0.83) where two share one, and 2.5 to join ranges.  Up
// to 128 rows (gated: 64) the weights' bytes decide, and slabs stream them better.
// Over 3253 random sizes above that the rule costs 0.7% against the better one of
// each; 2.6% of them lose more than 7%, most in 7 to 11 us, the worst 31% (n 12960, k
// 736, m 546: 17.2 / 13.1). Measured, slab / tile (us): n 8192, k 8 x 3584, m 64 38 /
// 74, 128 42 / 79, 256 65 / 81, 384 106 / 88, 512 117 / 94, 1024 223 / 178, 4096 858 / 592;
// n 1024, k 4096, m 512 9.6 / 15.1, 2048 13.0 / 15.7, 4096 21.9 / 17.7; n 4096, k 1024, m 512
// 7.6 / 9.5, 1024 10.1 / 10.2; n 2 x 1384, m 666, k 4096 13.0 / 16.0, 4112 19.2 / 18.5,
// 4128 14.6 / 16.4; gated, 8 x 3584, k 8192, m 64 76 / 83, 96 106 / 85, 256 151 / 92,
// 4096 2075 / 1206; 1376, k 4096, m 64 9.6 / 17.1, 128 10.0 / 17.1, 512 15.8 / 17.8; 3584, k
// 8192, m 128 18.4 / 27.6, 256 26.0 / 28.0 (tiles are taken there).
inline bool f8_tiles_sooner(bool gathers, bool gated, int R, int64_t m, int64_t n, int64_t k, int sm_count) {
    const int64_t slab_m = gated ? 64 : 128;
    if (m <= slab_m) return false;
    const int64_t ranks = gathers ? R : 1, blocks = (k + 127) / 128 * (gathers ? 1 : R), n_tiles = (n + 127) / 128;
    const int64_t units = (m + 255) / 256 * (gated ? n_tiles : (n_tiles + 1) / 2) * ranks, slabs = (m + slab_m - 1) / slab_m * n_tiles * ranks;
    const int64_t runs = ((k + 127) / 128 + 3) / 4 * (gathers ? 1 : R);
    const int64_t pairs = std::max(1, sm_count / 2), split = std::max<int64_t>(1, std::min<int64_t>({8, sm_count / slabs, runs}));
    const int64_t rounds = slabs <= sm_count ? 1 : (slabs + 2 * sm_count - 1) / (2 * sm_count);
    // rows that start between L2's sectors (16 bytes) or lines are fetched in more of them, which costs slabs the more the
    // more SMs fetch
    const double fill = std::min(1.0, static_cast<double>(slabs * split) / sm_count);
    const double tile_rows = k % 32 ? 1.25 : k % 128 ? 1.03 : 1.0, slab_rows = 1.0 + (k % 32 ? 0.6 : k % 128 ? 0.1 : 0.0) * fill;
    const double each = slabs <= sm_count ? (gated ? 0.39 : 0.28) : (gated ? 0.83 : 0.5);
    const double tile = (gated ? 8.0 : !gathers && R > 1 ? 7.0 : 6.0) + 0.31 * tile_rows * static_cast<double>((units + pairs - 1) / pairs * blocks);
    const double slab = 5.0 + each * slab_rows * static_cast<double>(rounds * blocks) / static_cast<double>(split) + (split > 1 ? 2.5 : 0.0);
    return tile < slab;
}

}  // namespace coc
