// Tiles of the bf16 products of a gated feed-forward block (host side).
#pragma once

#include <algorithm>
#include <cstdint>

namespace sgemm_gb300 {

// One product: an M x N result in tiles, summed over nk blocks of 64.  `halves`: the
// tile's columns are two matrices' (gate and up), so N counts both.
struct FfnShape {
    int64_t m, n, nk;
};

struct FfnTile {
    int rows, cols;         // of the result, for each CTA or pair
    int ctas;               // 2: a pair of SMs
};

constexpr FfnTile kFfnTiles[] = {{256, 256, 2}, {128, 128, 1}, {128, 64, 1}};

// The tile that a launch of `count` products takes: the least of a model's time, the
// longest share of a CTA times what a block of 64 k costs it, and the epilogue of
// its last tile.  `whole_groups`: only tiles with 128 columns of gate and of up.
inline int ffn_tile(const FfnShape *s, int count, bool whole_groups, int sms) {
    // clocks for a block of k, and for a tile's start and end
    constexpr double per_block[] = {560, 660, 500}, per_tile[] = {6000, 4000, 3000};
    int best = 0;
    double least = 0;
    for (int v = 0; v < (whole_groups ? 1 : 3); ++v) {
        const FfnTile &t = kFfnTiles[v];
        double blocks = 0, longest = 0;
        int64_t tiles = 0;
        for (int i = 0; i < count; ++i) {
            const int64_t n = ((s[i].m + t.rows - 1) / t.rows) * ((s[i].n + t.cols - 1) / t.cols);
            tiles += n;
            blocks += (double)n * s[i].nk;
            longest = std::max(longest, (double)s[i].nk);
        }
        const int64_t lanes = std::max<int64_t>(1, sms / t.ctas);
        const double waves = (double)((tiles + lanes - 1) / lanes);
        const double share = std::max(longest, waves * blocks / tiles);
        const double time = share * per_block[v] + per_tile[v];
        if (v == 0 || time < least) {
            least = time;
            best = v;
        }
    }
    return best;
}

}  // namespace sgemm_gb300
