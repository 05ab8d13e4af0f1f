// Products of few rows with a matrix read once, bf16 or 4-bit (host side).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

namespace sgemm_gb300 {

// C(m, n) = sum_k x(m, k) W(n, k), or with a second matrix act(x W^T) * (x W2^T).  W is
// bf16 (group 0), or 4-bit codes with scales (and zero codes) for each `group` (32, 64
// or 128) along k.  Rows of W start on 16 bytes, ldw bytes apart.
struct FewCall {
    int64_t M, N, K;
    const void *x;
    int x_f32;                     // else bf16
    int64_t ldx;
    const void *w, *w2;            // w2 null: one matrix
    int64_t ldw;
    int group;
    const float *s, *s2;
    const uint8_t *z, *z2;         // null: 8
    int64_t lds;
    int act;
    void *c;
    int c_f32;
    int64_t ldc;
};

// early: the kernel before it in the stream is the library's, and writes none of its weights:
// they may be read while that one still runs.
int run_few(const FewCall &c, cudaStream_t s, bool early);

// How a call is cut: blocks of 8 nt columns (rows of x, times their parts), wk warps of a
// CTA and ks CTAs of a cluster along the sum, `depth` stages of k that a CTA holds of x at a
// time, `ring` stages of weights that each warp has under way.
struct FewPlan {
    int nt, wk, ks, depth, ring;
};

constexpr int kFewWarps = 8;
constexpr int kFewStage = 4096;        // bytes of weights: 128 of each of 32 rows
// Stages of each warp under way, 64 KB of an SM's with one CTA, 128 with two.  (A third made
// the block of one token 4096 x 8192 43.8 us, not 35.5; one stage 39.8.)
constexpr int kFewRing = 2;

inline int64_t few_stage_k(int group) { return group ? 256 : 64; }
inline int few_parts(int group, bool x_f32) { return group && x_f32 ? 2 : 1; }
// Shared memory of a stage of x: its pieces for `cols` columns, and for 4 bits their units for
// all columns of a block; and of the partial sums, the warps' and the CTA's.
inline int64_t few_x_bytes(int group, int64_t cols, int nt) { return few_stage_k(group) * 2 * cols + (group ? 8 * 16 + 2 * 32 * nt : 0); }
inline int64_t few_sums_bytes(int nt, int64_t rows, int wk) {
    return (int64_t)kFewWarps * nt * 8 * 36 * 4 + 32 * (kFewWarps / wk) * rows * 4;
}

// Shared memory of a CTA, which has half an SM's with few columns.
inline int64_t few_most_smem(int nt) { return (nt <= 2 ? 110 : 216) * 1024; }

// The clusters of `ks` CTAs of nt tiles of columns that the current device, dev, runs together
// (0: an error).
int few_clusters(int dev, int nt, int ks);

// clusters(nt, ks): as few_clusters.
template <typename Clusters>
FewPlan few_plan(int64_t M, int64_t N, int64_t K, int parts, bool gated, int group, Clusters clusters) {
    FewPlan p;
    const int64_t stages = (K + few_stage_k(group) - 1) / few_stage_k(group);
    // columns for all rows of x, where their tiles' accumulators fit the registers
    const int64_t all = M * parts;
    p.nt = all <= 8 ? 1 : all <= 16 ? 2 : all <= 32 ? 4 : 8;
    const int64_t cols = std::min<int64_t>(M, 8 * p.nt / parts) * parts, x_stage = few_x_bytes(group, cols, p.nt);
    // Warps for the rows (32 each, or 16 of both matrices), times slices of the sum: the
    // fewest stages a warp that CTAs which run together allow (a second round of CTAs starts late:
    // 1 x 16384 x 8192 with 4 slices, 256 CTAs, 19.2 us, with 8 24.5, with 2 20.9; 1 x 20480 x
    // 8192 with 3 24.2, with 2 30.6).  How many do is asked, since a cluster's CTAs
    // are on neighbouring SMs: 48 clusters of 3 SMs, of the 50 that 152 SMs would hold, took
    // two rounds (32 x 6144 x 4096 29.1 us, with 32 clusters of 4 19.3).  Slices are
    // a CTA's warps where there is little to lay out of x for a stage (4 bits, M = 1 19.2 us,
    // not 20.0; bf16 block, 4 tokens 38.0, not 38.4), else a cluster's CTAs first, so that a CTA
    // lays out a part of x for more rows (M = 2 20.2 us, not 20.8, M = 8 23.0, not 34.9; bf16
    // block, 8 tokens 39.6, not 41.0).
    const bool little = cols * few_stage_k(group) <= 256;
    const int most_ks = p.nt <= 2 ? 8 : 4;
    int64_t fewest = stages + 1;
    p.wk = p.ks = 1;
    // Rows of x past a block's are blocks of CTAs beside it, and count (64 x 2048 x 4096 fp32 22.1 us, as
    // if each had the GPU to itself 33.1; 512 x 8192 x 4096 bf16 168 and 216).
    const int64_t blocks = (all + 8 * p.nt - 1) / (8 * p.nt);
    for (int i = 0; i < most_ks * 4; ++i) {
        const int wk = 1 << (little ? 3 - i % 4 : i / most_ks), ks = little ? 1 + i / 4 : most_ks - i % most_ks;
        const int64_t per_cta = (gated ? 16 : 32) * (kFewWarps / wk), each = ((stages + ks - 1) / ks + wk - 1) / wk;
        if (ks > stages || each >= fewest || (N + per_cta - 1) / per_cta * blocks > clusters(p.nt, ks)) continue;
        fewest = each;
        p.wk = wk;
        p.ks = ks;
    }
    // the ring, and x's whole range where it fits beside it
    const int64_t most = few_most_smem(p.nt), one = (int64_t)kFewWarps * kFewStage;
    const int64_t mine = (stages + p.ks - 1) / p.ks, each = (mine + p.wk - 1) / p.wk;
    p.depth = (int)std::max<int64_t>(1, std::min<int64_t>(mine, (most - kFewRing * one) / x_stage));
    p.ring = (int)std::max<int64_t>(1, std::min<int64_t>(each, kFewRing));
    return p;
}

}  // namespace sgemm_gb300
