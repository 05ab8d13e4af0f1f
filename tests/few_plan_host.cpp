// few_plan's cuts, one line of "nt wk ks depth ring bytes" for each line of "M N K group f32 gated"; the
// arguments are the clusters of 1, 2, .. 8 CTAs that the GPU holds with two CTAs an SM, then with one.
#include <cstdio>
#include <cstdlib>

#include "../dense_fp32_gemm_05_gb300/csrc/few.h"

int main(int argc, char **argv) {
    using namespace sgemm_gb300;
    if (argc != 17) return 1;
    int held[2][9] = {};
    for (int i = 0; i < 16; ++i) held[i / 8][i % 8 + 1] = std::atoi(argv[1 + i]);
    long long M, N, K;
    int group, f32, gated;
    while (std::scanf("%lld %lld %lld %d %d %d", &M, &N, &K, &group, &f32, &gated) == 6) {
        const int parts = few_parts(group, f32 != 0);
        const FewPlan p = few_plan(M, N, K, parts, gated != 0, group, [&](int nt, int ks) { return held[nt > 2][ks]; });
        const int64_t rows = std::min<int64_t>(M, 8 * p.nt / parts);
        const int64_t hold = (int64_t)p.ring * kFewWarps * kFewStage + p.depth * few_x_bytes(group, rows * parts, p.nt);
        std::printf("%d %d %d %d %d %lld\n", p.nt, p.wk, p.ks, p.depth, p.ring,
                    (long long)std::max(hold, few_sums_bytes(p.nt, rows, p.wk)));
    }
    return 0;
}
