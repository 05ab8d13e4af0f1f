// Products of few rows: how a call is cut and launched (the kernel is few_kernel.cuh's).
#include <algorithm>
#include <cstdint>

#include "few_kernel.cuh"

namespace sgemm_gb300 {

template <>
int launch_few<0>(const FewLaunch &l, cudaStream_t s);
template <>
int launch_few<32>(const FewLaunch &l, cudaStream_t s);
template <>
int launch_few<64>(const FewLaunch &l, cudaStream_t s);
template <>
int launch_few<128>(const FewLaunch &l, cudaStream_t s);

namespace few {
__device__ unsigned int g_error;               // sticky device error word of this path

// Rows of bytes in boxes of 128 bytes (swizzled) x box_rows; outside reads as zeros.
static bool byte_map(CUtensorMap *m, const void *base, int64_t rows, int64_t bytes, int64_t ld, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld};
    cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace few

int few_take_device_error() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, few::g_error, sizeof(v)) != cudaSuccess) return SGEMM_ERR_CUDA;
    if (v != 0 && cudaMemcpyToSymbol(few::g_error, &zero, sizeof(zero)) != cudaSuccess) return SGEMM_ERR_CUDA;
    return v == 0 ? SGEMM_OK : (int)v;
}

int run_few(const FewCall &c, cudaStream_t s, bool early) {
    const bool gated = c.w2 != nullptr;
    const int parts = few_parts(c.group, c.x_f32);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return launch_status();
    const FewPlan pl = few_plan(c.M, c.N, c.K, parts, gated, c.group, [dev](int nt, int ks) { return few_clusters(dev, nt, ks); });
    FewLaunch l{};
    few::Params &p = l.p;
    p.x = c.x;
    p.ldx = c.ldx;
    p.s[0] = c.s;
    p.s[1] = c.s2;
    p.z[0] = c.z;
    p.z[1] = c.z2;
    p.lds = (uint32_t)c.lds;
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
    p.c_vec = reinterpret_cast<uintptr_t>(c.c) % (c.c_f32 ? 16 : 8) == 0 && (c.ldc % 4 == 0 || c.M == 1);
    p.per_block = 8 * pl.nt / parts;
    p.wk = pl.wk;
    p.ks = pl.ks;
    p.stages = (int)((c.K + few_stage_k(c.group) - 1) / few_stage_k(c.group));
    p.depth = pl.depth;
    p.ring = pl.ring;
    p.groups = c.group ? (int)((c.K + c.group - 1) / c.group) : 0;
    p.early = early;
    p.wait_ns = tc_wait_limit();
    void *word = nullptr;
    if (cudaGetSymbolAddress(&word, few::g_error) != cudaSuccess) return launch_status();
    p.error = static_cast<unsigned int *>(word);
    const int per_cta = (gated ? 16 : 32) * (kFewWarps / pl.wk);
    const int64_t grid_x = (c.N + per_cta - 1) / per_cta * pl.ks, grid_y = (c.M + p.per_block - 1) / p.per_block;
    // (bytes of a row and k in int, scales addressed in 32 bits)
    if (c.K > INT32_MAX / 2 - 512 || grid_x > INT32_MAX || grid_y > 65535 ||
        (c.group && (c.K + c.group - 1) / c.group * c.lds > UINT32_MAX))
        return SGEMM_ERR_UNSUPPORTED;
    const int64_t bytes = c.group ? (c.K + 1) / 2 : 2 * c.K;
    const int box = gated ? 16 : 32;
    if (!few::byte_map(&l.map[0], c.w, c.N, bytes, c.ldw, box)) return SGEMM_ERR_UNSUPPORTED;
    l.map[1] = l.map[0];
    if (gated && !few::byte_map(&l.map[1], c.w2, c.N, bytes, c.ldw, box)) return SGEMM_ERR_UNSUPPORTED;
    const int64_t cols = std::min<int64_t>(c.M, p.per_block) * parts;
    const int64_t hold = (int64_t)pl.ring * kFewWarps * kFewStage + pl.depth * few_x_bytes(c.group, cols, pl.nt);
    l.smem = 1024 + (int)std::max<int64_t>(hold, few_sums_bytes(pl.nt, std::min<int64_t>(c.M, p.per_block), pl.wk));
    l.nt = pl.nt;
    l.grid_x = (int)grid_x;
    l.grid_y = (int)grid_y;
    switch (c.group) {
    case 0: return launch_few<0>(l, s);
    case 32: return launch_few<32>(l, s);
    case 64: return launch_few<64>(l, s);
    default: return launch_few<128>(l, s);
    }
}

}  // namespace sgemm_gb300
