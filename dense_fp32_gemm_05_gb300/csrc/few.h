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

// dep: launched as the programmatic dependent of a kernel that writes nothing but x.
int run_few(const FewCall &c, int sms, cudaStream_t s, bool dep);

// How a call is cut: blocks of 8 nt columns (rows of x, times their parts), wk warps of a
// CTA and ks CTAs of a cluster along the sum, `depth` chunks of k that a CTA holds of x at a time.
struct FewPlan {
    int nt, wk, ks, depth;
};

constexpr int kFewWarps = 8;

inline int64_t few_chunk(int group) { return group ? 128 : 32; }       // k: 64 bytes of a row

inline FewPlan few_plan(int64_t M, int64_t N, int64_t K, int parts, bool gated, int group, int sms) {
    FewPlan p;
    const int64_t chunks = (K + few_chunk(group) - 1) / few_chunk(group);
    // columns for all rows of x, where their tiles' accumulators fit the registers
    const int64_t cols = M * parts;
    const int tiles[] = {1, 2, 4, 6, 8};
    p.nt = 8;
    for (int t : tiles)
        if (cols <= 8 * t) {
            p.nt = t;
            break;
        }
    // Warps for the rows (32 each, or 16 of both matrices), times slices of the sum until
    // there are twelve for each SM.
    const int64_t rows = (N + (gated ? 15 : 31)) / (gated ? 16 : 32);
    int64_t slices = 1;
    while (slices < 64 && rows * slices < (int64_t)sms * 12 && 2 * slices <= chunks) slices *= 2;
    p.wk = (int)std::min<int64_t>(slices, kFewWarps);
    p.ks = (int)(slices / p.wk);
    // x in shared memory: the CTA's whole range where it fits
    const int64_t chunk_bytes = few_chunk(group) * 16 * p.nt, most = p.nt <= 2 ? 65536 : 131072;
    const int64_t mine = (chunks + p.ks - 1) / p.ks;
    p.depth = (int)std::max<int64_t>(1, std::min<int64_t>(mine, most / chunk_bytes));
    return p;
}

}  // namespace sgemm_gb300
