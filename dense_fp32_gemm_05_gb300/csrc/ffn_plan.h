// Tiles of the bf16 products of a gated feed-forward block (host side).
#pragma once

#include <algorithm>
#include <cstdint>

namespace sgemm_gb300 {

// One product: an m x n result in tiles, summed over nk blocks of 64.  Of the gated product n
// counts the columns of both matrices, gate and up, which share its tiles.
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

// Clocks of a lane for a tile among others: the MMAs and loads of a block of 64 k, or the
// epilogue where the sum is short; and of a launch before its first block is there.  Fitted
// to products of 64 .. 4096 tokens: 4096 x 4096 x 8192 us, down 164, 225 and 350 with the
// three tiles; 64 x 2048 x 4096 us, weights 17, 17 and 21, first backward launch 21, 15 and 11.
constexpr double kFfnBlock[] = {560, 450, 350}, kFfnStart = 6000;
enum FfnKind { FFN_STORE, FFN_GATED, FFN_SLOPE };
constexpr double kFfnEpilogue[][3] = {{5600, 3100, 2000}, {5600, 3100, 2000}, {16000, 7500, 4300}};
inline double ffn_tile_time(FfnKind kind, int variant, double nk) {
    return std::max(nk * kFfnBlock[variant], kFfnEpilogue[kind][variant]);
}

// How a launch is cut: its tile, and the CTAs of a cluster that share each tile's sum.
struct FfnCut {
    int variant, ks;
    double clocks;
};

// The cut of a launch of `count` products: the shortest time of that model, a lane's share
// of the tiles, or the longest tile with what its lane gets beside it.  One product with
// few tiles may be cut along the sum, over clusters that the GPU holds at once (clusters
// of 8 whole SMs: 14 of 19, as a GB300 answers; the plan is also asked for without a GPU. One
// that held fewer would run the rest after them); they add the partial sums in 1500 clocks.
// `whole_groups`: only tiles with 128 columns of gate and of up.
inline FfnCut ffn_cut(FfnKind kind, const FfnShape *s, int count, bool whole_groups, bool may_split, int sms) {
    FfnCut best{0, 1, 0};
    for (int v = 0; v < (whole_groups ? 1 : 3); ++v) {
        const FfnTile &t = kFfnTiles[v];
        double total = 0, longest = 0;
        int64_t tiles = 0;
        for (int i = 0; i < count; ++i) {
            const int64_t n = ((s[i].m + t.rows - 1) / t.rows) * ((s[i].n + t.cols - 1) / t.cols);
            const double one = ffn_tile_time(kind, v, (double)s[i].nk);
            tiles += n;
            total += (double)n * one;
            longest = std::max(longest, one);
        }
        const int64_t lanes = ffn_lanes(t.ctas, tiles, sms);
        const double rounds = (double)((tiles + lanes - 1) / lanes);
        const double time = std::max(longest, count > 1 ? total / lanes : rounds * longest) + kFfnEpilogue[kind][v] + kFfnStart;
        if (v == 0 || time < best.clocks) best = FfnCut{v, 1, time};
        if (!may_split || count > 1 || t.ctas > 1) continue;
        for (int ks = 2; ks <= 8 && 4 * ks <= s[0].nk; ks *= 2) {
            if (tiles * ks > (ks == 8 ? sms * 3 / 4 : ks == 4 ? sms * 9 / 10 : sms)) break;
            const double split = (double)s[0].nk / ks * kFfnBlock[v] + kFfnEpilogue[kind][v] + kFfnStart + 1500;
            if (split < best.clocks) best = FfnCut{v, ks, split};
        }
    }
    return best;
}

// Tokens up to which the forward pass, where nothing is kept, takes the products of few
// rows (few.h): 4096 x 8192 us, 8 tokens 40 (with tiles 54), 16 42 (43), 24 51 (44); 2048 x 4096
// 8 tokens 15 (28), 16 20 (26), 32 23 (21).
constexpr int64_t kFfnFewTokens = 16;

}  // namespace sgemm_gb300
