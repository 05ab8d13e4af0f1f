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

// Lanes that a launch of `units` tiles runs on: CTAs or pairs, one each SM or two.
inline int ffn_lanes(int ctas, int64_t units, int sms) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(units, sms / ctas));
}

// Clocks of a lane for a tile among others, and for the last one's epilogue: the MMAs and
// loads of a block of 64 k, or the epilogue where the sum is short.  Fitted to products of
// 64 .. 4096 tokens: 4096 x 4096 x 8192 us, down 164, 225 and 350 with the three tiles; 64 x 2048 x 4096,
// slope 25, 20 and 17.
constexpr double kFfnBlock[] = {560, 450, 350}, kFfnEpilogue[] = {14000, 7000, 3500};
inline double ffn_tile_time(int variant, double nk) { return std::max(nk * kFfnBlock[variant], kFfnEpilogue[variant]); }

// The tile that a launch of `count` products takes: the shortest time of that model, a
// lane's share of the tiles, or the longest tile with what its lane gets beside it.
// `whole_groups`: only tiles with 128 columns of gate and of up.
inline int ffn_tile(const FfnShape *s, int count, bool whole_groups, int sms) {
    int best = 0;
    double least = 0;
    for (int v = 0; v < (whole_groups ? 1 : 3); ++v) {
        const FfnTile &t = kFfnTiles[v];
        double total = 0, longest = 0;
        int64_t tiles = 0;
        for (int i = 0; i < count; ++i) {
            const int64_t n = ((s[i].m + t.rows - 1) / t.rows) * ((s[i].n + t.cols - 1) / t.cols);
            const double one = ffn_tile_time(v, (double)s[i].nk);
            tiles += n;
            total += (double)n * one;
            longest = std::max(longest, one);
        }
        const int64_t lanes = ffn_lanes(t.ctas, tiles, sms);
        const double rounds = (double)((tiles + lanes - 1) / lanes);
        const double time = std::max(longest, count > 1 ? total / lanes : rounds * longest) + kFfnEpilogue[v];
        if (v == 0 || time < least) {
            least = time;
            best = v;
        }
    }
    return best;
}

// Tokens up to which the forward pass, where nothing is kept, takes the products of few
// rows (few.h).
constexpr int64_t kFfnFewTokens = 16;

}  // namespace sgemm_gb300
