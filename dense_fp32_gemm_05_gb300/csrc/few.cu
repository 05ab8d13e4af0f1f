// Products of few rows: how a call is cut (see few_kernel.cuh for the kernel).
#include <algorithm>
#include <cstdint>

#include "few_kernel.cuh"

namespace sgemm_gb300 {

template <>
int launch_few<0>(int nt, const few::Params &p, int grid_x, int grid_y, int smem, cudaStream_t s, bool dep);
template <>
int launch_few<32>(int nt, const few::Params &p, int grid_x, int grid_y, int smem, cudaStream_t s, bool dep);
template <>
int launch_few<64>(int nt, const few::Params &p, int grid_x, int grid_y, int smem, cudaStream_t s, bool dep);
template <>
int launch_few<128>(int nt, const few::Params &p, int grid_x, int grid_y, int smem, cudaStream_t s, bool dep);

int run_few(const FewCall &c, int sms, cudaStream_t s, bool dep) {
    const bool gated = c.w2 != nullptr;
    const int parts = c.x_f32 ? 3 : 1;
    const FewPlan pl = few_plan(c.M, c.N, c.K, parts, gated, c.group, sms);
    few::Params p{};
    p.x = c.x;
    p.ldx = c.ldx;
    for (int i = 0; i < 2; ++i) {
        p.w[i] = static_cast<const uint8_t *>(gated && i ? c.w2 : c.w);
        p.s[i] = gated && i ? c.s2 : c.s;
        p.z[i] = gated && i ? c.z2 : c.z;
    }
    p.ldw = c.ldw;
    p.lds = c.lds;
    p.c = c.c;
    p.ldc = c.ldc;
    p.M = (int)c.M;
    p.N = (int)c.N;
    p.K = (int)c.K;
    p.gated = gated;
    p.act = c.act;
    p.c_f32 = c.c_f32;
    p.x_f32 = c.x_f32;
    p.x_vec = aligned16(c.x) && (c.ldx % (c.x_f32 ? 4 : 8) == 0 || c.M == 1);
    p.per_block = 8 * pl.nt / parts;
    p.wk = pl.wk;
    p.ks = pl.ks;
    p.chunks = (int)((c.K + few_chunk(c.group) - 1) / few_chunk(c.group));
    p.depth = pl.depth;
    const int per_cta = (gated ? 16 : 32) * (kFewWarps / pl.wk);
    const int64_t grid_x = (c.N + per_cta - 1) / per_cta * pl.ks, grid_y = (c.M + p.per_block - 1) / p.per_block;
    // (rows are addressed in 16 bytes, in 32 bits, and bytes in a row in int)
    if (c.K > INT32_MAX / 2 - 256 || grid_x > INT32_MAX || grid_y > 65535 || c.N * (c.ldw / 16) > UINT32_MAX) return SGEMM_ERR_UNSUPPORTED;
    const int smem = std::max((int)(pl.depth * few_chunk(c.group) * 16 * pl.nt), few::WARPS * pl.nt * 8 * few::RED * 4);
    const int gx = (int)grid_x, gy = (int)grid_y;
    switch (c.group) {
    case 0: return launch_few<0>(pl.nt, p, gx, gy, smem, s, dep);
    case 32: return launch_few<32>(pl.nt, p, gx, gy, smem, s, dep);
    case 64: return launch_few<64>(pl.nt, p, gx, gy, smem, s, dep);
    default: return launch_few<128>(pl.nt, p, gx, gy, smem, s, dep);
    }
}

}  // namespace sgemm_gb300
