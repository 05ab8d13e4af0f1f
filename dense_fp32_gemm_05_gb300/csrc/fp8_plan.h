// The selector of the 8-bit product: pure C++, also reachable without a GPU.
#pragma once

#include <algorithm>
#include <cstdint>

namespace sgemm_gb300 {

struct Fp8Plan {
    int by = 256;       // rows of C per tile
    int bx = 256;       // columns of C per tile: 256 the wide kernel, 128 the narrow one
    int ksplit = 1;     // CTAs of a cluster that share a tile's sum (narrow)
};

// Takes the tile and cluster size with the least time by a model in microseconds,
// fitted to GB300: a call's fixed time, and for each wave of tiles a time for each
// block of 128 k and one for the epilogue.
//
//            fixed   block   epilogue   (block with a scale for each row of B)
//   16 rows   4.2    0.17     1.0        0.19
//   32        4.9    0.20     1.4        0.24
//   64        6.1    0.24     2.0        0.32
//   128       8.4    0.375    3.0        0.53
//   256 x 256 4.0    0.42     1.1        0.65
//
// A cluster of k CTAs takes 1/k of the blocks and 1.5 us to add; clusters have to be
// resident at once (more than ~136 CTAs in clusters take two waves and more: 512 x
// 4096 x 4096 with 128 rows and 2 CTAs 10 -> 41 us).  Measured (us, model / GPU), the
// choices in turn: 256^3 16 rows 4.5 / 4.5, 128 rows (the rule before) 9.2 / 8.8; 1024^3
// 64 rows 8.0 / 8.3, 256 x 256 8.5 / 9.0, 16 rows 12.4 / 12.4; 128 x 4096 x 4096 32 rows
// 11.3 / 11.4, 128 rows in clusters of 4 12.9 / 14.7; 100 x 16384 x 8192 128 rows 32.4 / 34.5,
// 32 rows 61 / 60; 300 x 300 x 8192 64 rows in clusters of 8 9.5 / 9.0; 2048 x 1024 x 4096
// 256 x 256 18.5 / 18.5, 128 rows 20.4 / 21.2; the same with a scale for each row of B
// 256 x 256 25.9 / 25.7, 128 rows 25.4 / 21.4.
inline Fp8Plan fp8_plan(int64_t M, int64_t N, int64_t K, int b_group, int sms) {
    constexpr int kClusterCtas = 136;
    const int64_t nkb = (K + 127) / 128;
    auto ceil_div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    Fp8Plan best;
    const bool vec = b_group == 1;
    const double block = vec ? 0.65 : 0.42;
    double best_us = M > 128 && N > 128
                         ? 4.0 + (double)ceil_div(ceil_div(M, 256) * ceil_div(N, 256), std::max(sms / 2, 1)) * (block * (double)nkb + 1.1)
                         : 1e30;
    const struct { int by; double fixed, block, vec_block, epilogue; } narrow[] = {
        {16, 4.2, 0.17, 0.19, 1.0}, {32, 4.9, 0.20, 0.24, 1.4}, {64, 6.1, 0.24, 0.32, 2.0}, {128, 8.4, 0.375, 0.53, 3.0}};
    for (const auto &n : narrow) {
        if (n.by > 16 && n.by >= 2 * M) break;
        const int64_t tiles = ceil_div(N, 128) * ceil_div(M, n.by);
        for (int ks = 1; ks <= 8 && ks <= nkb; ks *= 2) {
            if (ks > 1 && tiles * ks > std::min(sms, kClusterCtas)) break;
            const double us = n.fixed - n.epilogue + (ks > 1 ? 1.5 : 0.0) +
                              (double)ceil_div(tiles * ks, sms) * ((double)ceil_div(nkb, ks) * (vec ? n.vec_block : n.block) + n.epilogue);
            if (us < best_us) {
                best_us = us;
                best.by = n.by;
                best.bx = 128;
                best.ksplit = ks;
            }
        }
    }
    return best;
}

}  // namespace sgemm_gb300
