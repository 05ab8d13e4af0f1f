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

inline Fp8Plan fp8_plan(int64_t M, int64_t N, int64_t K, int sms) {
    Fp8Plan pl;
    const int64_t nkb = (K + 127) / 128;
    const int64_t wide = ((M + 255) / 256) * ((N + 255) / 256);
    if (M > 128 && N > 128 && wide * 2 >= sms / 2) return pl;
    pl.bx = 128;
    pl.by = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    const int64_t tiles = ((N + 127) / 128) * ((M + pl.by - 1) / pl.by);
    while (pl.ksplit < 8 && tiles * pl.ksplit * 2 <= sms && nkb >= 4 * pl.ksplit) pl.ksplit *= 2;
    return pl;
}

}  // namespace sgemm_gb300
