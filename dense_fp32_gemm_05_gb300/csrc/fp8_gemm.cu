// Matrix product of two quantised operands (8-bit codes, one fp32 scale for
// each group of 128 along the sum):
//
//   C(m,n) = alpha * sum_b sA(m,b) sB(b,n) P_b(m,n) + beta * C(m,n),
//   P_b(m,n) = sum over the 128 k of block b of A(m,k) B(k,n)
//
// P_b is what tcgen05.mma kind::f8f6f4 adds up in tensor memory (products of
// codes are exact in fp32); the scales differ from block to block, so each
// P_b is brought into registers once and added there with its scales.
//
// Two kernels.  Large results take 256 x 256 tiles on SM pairs (fp8_wide_kernel,
// below), the others narrow tiles (fp8_gemm_kernel), by the rule in fp8_plan.h.
//
// Narrow tiles: the MMA's M (tensor-memory lanes) is the result's N, its N (columns)
// the result's M.  A warp then holds 32 neighbouring columns of C for each row m, so
// that C is stored straight from registers, whole sectors at a time; and few rows
// (decode) become a narrow MMA, BY = 16 .. 128 columns, against 128 full rows of the
// weights, which are read once.  352 threads, one CTA per SM:
//   warp 0      TMA producer: per block of 128 k one 128 x 128 tile of B (the
//               "X" operand) and a BY x 128 tile of A ("Y") into a ring of
//               stages.  Either operand may be stored along k or across it
//               (MN-major descriptors read the tile as it lies);
//   warp 1      tensor memory, and the 4 MMAs of a block into one of two buffers of
//               BY columns;
//   warp 2      the block's scales, sA(m,b) for each column (times sB where
//               that is one value for the CTA's 128 rows), in a small ring;
//   warps 3-10  add a block's P_b to the accumulators: tcgen05.ld, then one
//               fused multiply-add for each value (two where B has a scale for each
//               row).  128 x BY fp32 accumulators live in their registers: warp w has
//               lanes 32 (w % 4) .. + 31 and half of the columns.  They release the
//               buffer as soon as it is read.
// Each CTA walks tiles of C (grouped raster), the rings run on across tiles.
// Few tiles: a cluster of KS CTAs shares a tile's blocks in contiguous ranges
// and adds the partial sums through distributed shared memory in ascending
// order, each CTA its share of the columns: no workspace, no atomics.
// Decode is bound by the weights' stream: 16 x 16384 x 8192 25.1 us on the GPU alone, 5.4
// TB/s (0.81 of the measured copy), 26.7 us among other calls, of which ~4 us are the
// launch, the first loads and the last tile; small ones by latency (256^3 4.3 us).
//
// Every wait is bounded, as in the tensor-core GEMM: on expiry the device error
// word is set, the role stops, copies and MMAs in flight are waited for (again
// bounded) and the CTA frees its tensor memory and exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <new>

#include "fp8.cuh"
#include "fp8_plan.h"
#include "plan.h"
#include "ptx_util.cuh"
#include "tc_gemm.h"
#include "tc_ptx.cuh"

namespace sgemm_gb300 {
namespace fp8g {

using namespace tc;

constexpr int BX = 128;                    // rows of X (columns of C) per CTA
constexpr int BK = fp8::GROUP;             // k per block
constexpr int X_BYTES = BX * BK;
constexpr int PROMOTERS = 8;               // warps 3..10
constexpr int THREADS = 32 * (3 + PROMOTERS);
constexpr int MAX_STAGES = 12;
constexpr int SCALE_SLOTS = 4;
constexpr int SMEM_MAX = 232448;           // opt-in dynamic shared memory per block
constexpr int BAR_BYTES = 512;
constexpr uint64_t kDrainNs = 1000000000ull;

__device__ unsigned int g_error;           // sticky device error word of this path

struct Params {
    void *C;
    int64_t ldc;
    int c_bf16;
    int M, N;
    float alpha, beta;
    const float *SX, *SY;                  // scales of B (X) and A (Y)
    int64_t x_mn, x_k, y_mn, y_k;          // strides of the scales along N / M (per group) and per block of k
    int x_shift, y_shift;                  // a scale for each 1 << shift rows
    int c_vec;                             // quads of C may be accessed whole
    int c_tma;                             // wide tiles: columns of C from 0 that TMA writes (0: none)
    int c_add;                             // it adds them to what is there
    int x_mnmajor, y_mnmajor;              // operand stored across k
    int y_bytes;                           // bytes of Y per stage
    uint32_t idesc;
    int tiles_x, tiles_y, group_y;
    int nkb;                               // blocks of 128 k
    int stages, ksplit;
    unsigned long long wait_ns;
};

// Bounded wait by a converged warp: true when every lane's was.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit) {
    return __all_sync(0xffffffffu, mbar_wait_for(bar, parity, limit, &g_error));
}

// Tile u of the grouped raster: group_y tile rows of C at a time, so that the
// tiles in flight share operand panels in L2.
__device__ __forceinline__ void tile_of(const Params &p, int u, int &tx, int &ty) {
    const int per = p.group_y * p.tiles_x;
    const int g = u / per, r = u - g * per;
    const int h = min(p.group_y, p.tiles_y - g * p.group_y);
    tx = r / h;
    ty = g * p.group_y + (r - tx * h);
}

__device__ __forceinline__ float load_c(const Params &p, int64_t at) {
    return p.c_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.C)[at])
                    : static_cast<const float *>(p.C)[at];
}

// alpha * acc, or fma(alpha, acc, beta * c), to be rounded once to C's type
__device__ __forceinline__ float epilogue(const Params &p, float acc, float old) {
    return p.beta == 0.0f ? __fmul_rn(p.alpha, acc) : __fmaf_rn(p.alpha, acc, __fmul_rn(p.beta, old));
}

__device__ __forceinline__ void store_c(const Params &p, int64_t at, float acc, float old) {
    const float v = epilogue(p, acc, old);
    if (p.c_bf16) static_cast<__nv_bfloat16 *>(p.C)[at] = __float2bfloat16_rn(v);
    else static_cast<float *>(p.C)[at] = v;
}

// A CTA's own address of `local` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(uint32_t local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ void store_cluster(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ float load_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// ---------------------------------------------------------------- narrow tiles
// BY: columns of the MMA (rows of C) per tile, 16 .. 128.  XVEC: B has a scale for each
// of its rows (else one for the CTA's 128).
template <int BY, bool XVEC>
__global__ void __launch_bounds__(THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_y,
                    const Params p) {
    constexpr int PC = BY / 2;                     // columns per promoting thread
    constexpr int CH = PC < 16 ? PC : 16;          // columns per tensor-memory load
    constexpr uint32_t COLS = 2 * BY < 32 ? 32 : 2 * BY;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stage_bytes = X_BYTES + p.y_bytes;
    const uint32_t smem0 = smem_u32(smem);
    float *scales = reinterpret_cast<float *>(smem + p.stages * stage_bytes);
    uint64_t *bars = reinterpret_cast<uint64_t *>(scales + SCALE_SLOTS * BY);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * MAX_STAGES + 4 + 2 * SCALE_SLOTS);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (MAX_STAGES + s); };
    auto tfull = [&](int b) { return bar0 + 8u * (2 * MAX_STAGES + b); };
    auto tempty = [&](int b) { return bar0 + 8u * (2 * MAX_STAGES + 2 + b); };
    auto sfull = [&](int s) { return bar0 + 8u * (2 * MAX_STAGES + 4 + s); };
    auto sempty = [&](int s) { return bar0 + 8u * (2 * MAX_STAGES + 4 + SCALE_SLOTS + s); };

    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int ks = p.ksplit;
    const int rank = ks > 1 ? (int)cluster_rank() : 0;
    const int group = (int)blockIdx.x / ks, groups = (int)gridDim.x / ks;
    const int kb0 = (int)((int64_t)p.nkb * rank / ks), kb1 = (int)((int64_t)p.nkb * (rank + 1) / ks);
    const int units = p.tiles_x * p.tiles_y;
    const uint64_t lim = p.wait_ns;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tempty(b), PROMOTERS);
        }
        for (int s = 0; s < SCALE_SLOTS; ++s) {
            mbar_init(sfull(s), 1);
            mbar_init(sempty(s), PROMOTERS);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&tm_x);
        prefetch_map(&tm_y);
    }
    if (warp == 1) tmem_alloc<false>(smem_u32(tmem_slot), COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();                                    // a copy of an operand may precede this kernel

    float2 acc[PC / 2];
    bool ok = true;
    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        {
            int s = 0, filled = 0;
            uint32_t ph = 1;                       // an empty stage's first wait passes
            for (int u = group; ok && u < units; u += groups) {
                int tx, ty;
                tile_of(p, u, tx, ty);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!warp_wait(empty(s), ph, lim)) { ok = false; break; }
                    const uint32_t x = smem0 + (uint32_t)(s * stage_bytes), y = x + X_BYTES;
                    const int k = kb * BK, n = tx * BX, m = ty * BY;
                    if (elect_one()) {
                        mbar_expect_tx(full(s), (uint32_t)stage_bytes);
                        tma_load_2d(x, &tm_x, full(s), p.x_mnmajor ? n : k, p.x_mnmajor ? k : n);
                        tma_load_2d(y, &tm_y, full(s), p.y_mnmajor ? m : k, p.y_mnmajor ? k : m);
                    }
                    ++filled;
                    if (++s == p.stages) { s = 0; ph ^= 1; }
                }
            }
            // copies in flight land before the CTA's shared memory goes (on an
            // early stop nobody else has waited for them)
            for (int i = 0; i < min(filled, p.stages); ++i) {
                if (s == 0) { s = p.stages; ph ^= 1; }
                --s;
                mbar_wait_for(full(s), ph ^ 1u, kDrainNs, &g_error);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        {
            int s = 0, b = 0, issued = 0;
            uint32_t ph = 0, bph = 1;
            const uint64_t dx0 = smem_desc_8bit(smem0, X_BYTES);
            const uint32_t x_step = p.x_mnmajor ? 4096u >> 4 : 32u >> 4;
            const uint32_t y_step = p.y_mnmajor ? 4096u >> 4 : 32u >> 4;
            for (int u = group; ok && u < units; u += groups) {
                for (int kb = kb0; kb < kb1; ++kb) {
                    // (the two tests overlap: few columns leave little time for a block)
                    const bool t0 = mbar_test(full(s), ph), t1 = mbar_test(tempty(b), bph);
                    if (!__all_sync(0xffffffffu, t0 && t1) &&
                        (!warp_wait(full(s), ph, lim) || !warp_wait(tempty(b), bph, lim))) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t dx = dx0 + (uint32_t)(s * (stage_bytes >> 4)), dy = dx + (X_BYTES >> 4);
                    const uint32_t d = tmem + (uint32_t)(b * BY);
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < BK / 32; ++i)
                            umma_8bit<false>(d, dx + i * x_step, dy + i * y_step, p.idesc, i > 0);
                        umma_commit(tfull(b));
                    }
                    ++issued;
                    if (++s == p.stages) { s = 0; ph ^= 1; }
                    if (++b == 2) { b = 0; bph ^= 1; }
                }
            }
            // MMAs retire before tensor memory is freed
            if (issued > 0) {
                const int last = (issued - 1) & 1;
                mbar_wait_for(tfull(last), (uint32_t)((issued - 1) >> 1) & 1u, kDrainNs, &g_error);
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------ scales
        constexpr int J = (BY + 31) / 32;          // columns per lane
        constexpr int AHEAD = 4;                   // blocks loaded at a time
        int slot = 0;
        uint32_t ph = 1;
        for (int u = group; ok && u < units; u += groups) {
            int tx, ty;
            tile_of(p, u, tx, ty);
            const float *sx = XVEC ? nullptr : p.SX + (int64_t)tx * p.x_mn;   // BX = the block's width
            float v[AHEAD][J], w[AHEAD];
            auto fetch = [&](int kb) {
#pragma unroll
                for (int a = 0; a < AHEAD; ++a) {
                    const bool in = kb + a < kb1;
                    w[a] = !XVEC && in ? __ldg(sx + (int64_t)(kb + a) * p.x_k) : 1.0f;
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        const int m = ty * BY + 32 * j + lane;
                        v[a][j] = in && m < p.M && 32 * j + lane < BY
                                      ? __ldg(p.SY + (int64_t)(m >> p.y_shift) * p.y_mn + (int64_t)(kb + a) * p.y_k)
                                      : 0.0f;
                    }
                }
            };
            fetch(kb0);
            for (int kb = kb0; ok && kb < kb1; kb += AHEAD) {
                float t[AHEAD][J];
#pragma unroll
                for (int a = 0; a < AHEAD; ++a)
#pragma unroll
                    for (int j = 0; j < J; ++j) t[a][j] = XVEC ? v[a][j] : __fmul_rn(v[a][j], w[a]);
                fetch(kb + AHEAD);
#pragma unroll
                for (int a = 0; a < AHEAD; ++a) {
                    if (kb + a >= kb1) break;
                    if (!warp_wait(sempty(slot), ph, lim)) { ok = false; break; }
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        if (32 * j + lane < BY) scales[slot * BY + 32 * j + lane] = t[a][j];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sfull(slot));
                    if (++slot == SCALE_SLOTS) { slot = 0; ph ^= 1; }
                }
            }
        }
    } else {
        // ------------------------------------------------ promotion and epilogue
        const int q = warp & 3, half = (warp - 3) >> 2;
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * PC);
        int stage = 0, b = 0, slot = 0;
        uint32_t bph = 0, sph = 0;
        for (int u = group; ok && u < units; u += groups) {
            int tx, ty;
            tile_of(p, u, tx, ty);
            const int n = tx * BX + q * 32 + lane;
            const float *sx = p.SX + (XVEC ? (int64_t)min(n, p.N - 1) : 0);
#pragma unroll
            for (int i = 0; i < PC / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
            float sx_next = XVEC ? __ldg(sx + (int64_t)kb0 * p.x_k) : 0.0f;
            for (int kb = kb0; kb < kb1; ++kb) {
                const float2 sx2 = make_float2(sx_next, sx_next);
                if (XVEC && kb + 1 < kb1) sx_next = __ldg(sx + (int64_t)(kb + 1) * p.x_k);
                ok = mbar_wait_for(sfull(slot), sph, lim, &g_error) &&
                     mbar_wait_for(tfull(b), bph, lim, &g_error);
                if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
                tc_fence_after();
                // the block's MMAs are done with its stage
                if (warp == 3 && lane == 0) mbar_arrive(empty(stage));
                if (++stage == p.stages) stage = 0;
                const float *sc = scales + slot * BY + half * PC;
                uint32_t r[2][CH];
                tmem_ld_async(taddr + (uint32_t)(b * BY), r[0]);
#pragma unroll
                for (int c = 0; c < PC / CH; ++c) {
                    tmem_ld_wait(r[c & 1]);
                    if (c + 1 < PC / CH) {
                        tmem_ld_async(taddr + (uint32_t)(b * BY + (c + 1) * CH), r[(c + 1) & 1]);
                    } else {                       // the buffer is read: hand it back
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(tempty(b));
                    }
#pragma unroll
                    for (int i = 0; i < CH; i += 4) {
                        const float4 s4 = *reinterpret_cast<const float4 *>(sc + c * CH + i);
                        float2 t0 = make_float2(__uint_as_float(r[c & 1][i]), __uint_as_float(r[c & 1][i + 1]));
                        float2 t1 = make_float2(__uint_as_float(r[c & 1][i + 2]), __uint_as_float(r[c & 1][i + 3]));
                        float2 &a0 = acc[(c * CH + i) / 2], &a1 = acc[(c * CH + i) / 2 + 1];
                        if (XVEC) {
                            t0 = __fmul2_rn(t0, make_float2(s4.x, s4.y));
                            t1 = __fmul2_rn(t1, make_float2(s4.z, s4.w));
                            a0 = __ffma2_rn(t0, sx2, a0);
                            a1 = __ffma2_rn(t1, sx2, a1);
                        } else {
                            a0 = __ffma2_rn(t0, make_float2(s4.x, s4.y), a0);
                            a1 = __ffma2_rn(t1, make_float2(s4.z, s4.w), a1);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sempty(slot));
                if (++slot == SCALE_SLOTS) { slot = 0; sph ^= 1; }
                if (++b == 2) { b = 0; bph ^= 1; }
            }
            if (!ok || ks > 1) break;
            if (n < p.N) {
                const int m0 = ty * BY + half * PC;
#pragma unroll
                for (int c = 0; c < PC; c += CH) {
                    // a batch's loads of C are all under way before its first store
                    float old[CH];
#pragma unroll
                    for (int i = 0; i < CH; ++i)
                        old[i] = p.beta != 0.0f && m0 + c + i < p.M ? load_c(p, (int64_t)(m0 + c + i) * p.ldc + n) : 0.0f;
#pragma unroll
                    for (int i = 0; i < CH; ++i)
                        if (m0 + c + i < p.M) {
                            const float2 a = acc[(c + i) / 2];
                            store_c(p, (int64_t)(m0 + c + i) * p.ldc + n, i % 2 ? a.y : a.x, old[i]);
                        }
                }
            }
        }
    }

    if (ks > 1) {
        // every MMA of this CTA has completed (the promoters saw the last one),
        // so its stages hold the partial sums now: [column][128 rows of X]
        float *part = reinterpret_cast<float *>(smem);
        const int q = warp & 3, half = (warp - 3) >> 2;
        __syncthreads();                           // (on an early stop: copies have landed)
        if (warp >= 3) {
#pragma unroll
            for (int i = 0; i < PC / 2; ++i) {
                part[(half * PC + 2 * i) * BX + q * 32 + lane] = acc[i].x;
                part[(half * PC + 2 * i + 1) * BX + q * 32 + lane] = acc[i].y;
            }
        }
        cluster_sync_all();
        if (warp >= 3) {
            int tx, ty;
            tile_of(p, group, tx, ty);
            const int n = tx * BX + q * 32 + lane;
            const int c1 = BY * (rank + 1) / ks;
            for (int c = BY * rank / ks + half; c < c1; c += 2) {
                const int m = ty * BY + c;
                if (m >= p.M) break;
                const uint32_t at = smem0 + 4u * (uint32_t)(c * BX + q * 32 + lane);
                float sum = 0.0f;
                for (int r = 0; r < ks; ++r) sum = __fadd_rn(sum, load_cluster(peer_addr(at, (uint32_t)r)));
                const int64_t to = (int64_t)m * p.ldc + n;
                if (n < p.N) store_c(p, to, sum, p.beta != 0.0f ? load_c(p, to) : 0.0f);
            }
        }
        cluster_sync_all();                        // no CTA leaves while a peer reads its sums
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free<false>(tmem, COLS);
    }
}

// ---------------------------------------------------------------- wide tiles
// 256 x 256 tiles of C on a pair of SMs (cta_group::2): each CTA holds its 128
// rows of A ("X"), half of the tile's 256 columns of B ("Y") and its 128 rows of
// the two tensor-memory buffers.  Here the lanes are C's rows: a row's scale is one
// register, and where B has one scale for its 128 x 128 block the product of the
// two is one value for each thread and block of k, so that promotion is one
// multiply-add per value and nothing else.  (With C's columns on the lanes every
// column's scale comes from shared memory for every block, beside the MMAs' own
// reads: 820 us at 8192^3, on single SMs.)  128 accumulators per promoting thread
// need more registers than an equal share: the first warpgroup hands its over
// (setmaxnreg).
// 8192^3 NT 392 us in short runs, 2.80 PFLOP/s (0.73 of twice the measured bf16 rate),
// 435 us under the power cap.  What bounds
// it is the turn-round of the two buffers, which fill tensor memory: release to the
// MMA's start 230 clocks, the MMAs (512) and their commit's arrival 900, reading 580,
// for two blocks; the MMAs fed by TMA alone would take 671 a block, not 857.
// With a scale for each row of B promotion is a multiply and a multiply-add, and the
// columns' scales come from shared memory.  There a thread reads pairs of columns in
// four rows, so that a pair of scales is loaded once for four pairs of values and the
// rows' scales are four registers: with a row in each thread, as above, the loads of
// 16 bytes for every four values took shared memory's whole rate (4096 x 4096 x 8192
// TN, beta = 1: 225 -> 192 us; 168 us, 1.64 PFLOP/s, with the waits below).  The
// promoting warps bound it.
constexpr int WT = 256;                        // tile rows and columns
constexpr int W_STAGE = 2 * X_BYTES;           // per CTA

template <bool YVEC>
struct Wide {
    static constexpr int WARPS = 8;                        // promoting: 32 rows x 128 columns each
    static constexpr int THREADS = 32 * (4 + WARPS);       // after TMA, MMA, scales, idle: a warpgroup
    static constexpr int PC = WT / (WARPS / 4);            // columns per promoting warp
    static constexpr int CH = 32;                          // columns read or stored at a time
    static constexpr int REGS_ISSUE = 40, REGS_PROMOTE = 232;   // 384 x 168 = 128 x 40 + 256 x 232
    static constexpr int OUT = 32 * CH * 4;                // epilogue staging per warp
    static constexpr int BATCH = 4;                        // blocks of k whose scales are fetched together
    // YVEC: the scales of the CTA's rows and the tile's columns for a block of k in a slot
    static constexpr int SLOTS = YVEC ? 6 : 0;
    static constexpr int BLOCK = BX + WT;                  // floats for a block
    static constexpr int RING = SLOTS * BLOCK;
    static constexpr int FIXED = 1024 + WARPS * OUT + RING * 4 + BAR_BYTES;
    static constexpr int STAGES = (SMEM_MAX - FIXED) / W_STAGE;
    static constexpr int SMEM = FIXED + STAGES * W_STAGE;
    static_assert(STAGES >= 4 && STAGES <= MAX_STAGES, "stages");
};

// The 16-byte chunk of a staged row of `bytes` (32, 64 or 128) where chunk c lies: TMA's
// swizzle over that span.
template <int BYTES>
__device__ __forceinline__ int staged_chunk(int row, int c) {
    return BYTES == 128 ? c ^ (row & 7) : BYTES == 64 ? c ^ ((row >> 1) & 3) : c ^ ((row >> 2) & 1);
}

__device__ __forceinline__ float4 load4(const float *c) { return *reinterpret_cast<const float4 *>(c); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *c) {
    const uint2 u = *reinterpret_cast<const uint2 *>(c);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void store4(float *c, float4 v) { *reinterpret_cast<float4 *>(c) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *c, float4 v) {
    *reinterpret_cast<uint2 *>(c) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
}
__device__ __forceinline__ float load1(const float *c) { return *c; }
__device__ __forceinline__ float load1(const __nv_bfloat16 *c) { return __bfloat162float(*c); }
__device__ __forceinline__ void store1(float *c, float v) { *c = v; }
__device__ __forceinline__ void store1(__nv_bfloat16 *c, float v) { *c = __float2bfloat16_rn(v); }

// A staged block of 32 rows x 32 columns of sums to C, through the epilogue: quads of
// columns where C allows, else a row's columns across the lanes.  Eight rows' (or
// quads') loads of C are under way together, where it is read at all; pointers are
// stepped, not multiplied (4095 x 3073 x 1537: 5600 instructions a tile of each warp
// otherwise, 32 of the 67 us).
template <typename T, bool READ>
__device__ __forceinline__ void write_block(T *C, int64_t ldc, float alpha, float beta, bool vec, const float *stg,
                                            int rows, int cols) {
    const int lane = threadIdx.x & 31;
    if (vec && cols >= 32) {
        const int r0 = lane >> 3, c = lane & 7;
        T *at = C + r0 * ldc + 4 * c;
        const int64_t step = 4 * ldc;
        float4 old[8];
        if (READ) {
            const T *from = at;
#pragma unroll
            for (int i = 0; i < 8; ++i, from += step)
                old[i] = 4 * i + r0 < rows ? load4(from) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i, at += step) {
            const int r = 4 * i + r0;
            float4 v = *reinterpret_cast<const float4 *>(stg + r * 32 + 4 * staged_chunk<128>(r, c));
            if (READ)
                v = make_float4(__fmaf_rn(alpha, v.x, __fmul_rn(beta, old[i].x)), __fmaf_rn(alpha, v.y, __fmul_rn(beta, old[i].y)),
                                __fmaf_rn(alpha, v.z, __fmul_rn(beta, old[i].z)), __fmaf_rn(alpha, v.w, __fmul_rn(beta, old[i].w)));
            else
                v = make_float4(__fmul_rn(alpha, v.x), __fmul_rn(alpha, v.y), __fmul_rn(alpha, v.z), __fmul_rn(alpha, v.w));
            if (r < rows) store4(at, v);
        }
    } else {
        if (lane >= cols) return;
        T *at = C + lane;
        const float *src = stg + (lane & 3);
#pragma unroll 1
        for (int i0 = 0; i0 < 32; i0 += 8, src += 8 * 32) {
            float old[8];
            if (READ) {
                const T *from = at;
#pragma unroll
                for (int i = 0; i < 8; ++i, from += ldc) old[i] = i0 + i < rows ? load1(from) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i, at += ldc) {
                const float v = src[i * 32 + 4 * ((lane >> 2) ^ i)];
                if (i0 + i < rows)
                    store1(at, READ ? __fmaf_rn(alpha, v, __fmul_rn(beta, old[i])) : __fmul_rn(alpha, v));
            }
        }
    }
}

// YVEC: B has a scale for each of its rows (else one for each 128 x 128 block).
template <bool YVEC>
__global__ void __launch_bounds__(Wide<YVEC>::THREADS, 1) __cluster_dims__(2, 1, 1)
    fp8_wide_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_y,
                    const __grid_constant__ CUtensorMap tm_c, const Params p) {
    using K_ = Wide<YVEC>;
    constexpr int S = K_::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t smem0 = smem_u32(smem);
    float *staging = reinterpret_cast<float *>(smem + S * W_STAGE);
    float *scales = staging + K_::WARPS * K_::OUT / 4;
    uint64_t *bars = reinterpret_cast<uint64_t *>(scales + K_::RING);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * S + 4 + 2 * K_::SLOTS);
    uint32_t *counts = tmem_slot + 1;              // stages filled by either CTA, blocks the leader multiplied
    static_assert((2 * S + 4 + 2 * K_::SLOTS) * 8 + 16 <= BAR_BYTES, "barriers");
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };
    auto tfull = [&](int b) { return bar0 + 8u * (2 * S + b); };
    auto tempty = [&](int b) { return bar0 + 8u * (2 * S + 2 + b); };
    auto sfull = [&](int s) { return bar0 + 8u * (2 * S + 4 + s); };
    auto sempty = [&](int s) { return bar0 + 8u * (2 * S + 4 + K_::SLOTS + s); };

    const int warp = warp_index(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int group = (int)blockIdx.x >> 1, groups = (int)gridDim.x >> 1;
    const int units = p.tiles_x * p.tiles_y;
    const uint64_t lim = p.wait_ns;
    auto publish = [&](int which, int n) {         // to both CTAs
        if (lane == 0) {
            counts[which] = (uint32_t)n;
            store_cluster(peer_addr(smem_u32(counts + which), rank ^ 1u), (uint32_t)n);
        }
    };

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tempty(b), 2 * K_::WARPS);   // of both CTAs, on the leader's
        }
        for (int s = 0; s < K_::SLOTS; ++s) {
            mbar_init(sfull(s), 32);               // each lane's copies
            mbar_init(sempty(s), K_::WARPS);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&tm_x);
        prefetch_map(&tm_y);
    }
    if (warp == 1) tmem_alloc<true>(smem_u32(tmem_slot), 512);
    tc_fence_before();
    cluster_sync_all();                            // the peer's barriers exist before anything arrives on them
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();                                    // a copy of an operand may precede this kernel

    bool ok = true;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(K_::REGS_ISSUE));
        if (warp == 0) {
            // ------------------------------------------------ TMA producer
            {
                int s = 0, filled = 0;
                uint32_t ph = 1;
                const uint32_t lead_full0 = leader_addr(full(0));
                for (int u = group; ok && u < units; u += groups) {
                    int tx, ty;
                    tile_of(p, u, tx, ty);
                    const int m = ty * WT + (int)rank * BX, n = tx * WT + (int)rank * BX;
                    for (int kb = 0; kb < p.nkb; ++kb) {
                        if (!warp_wait(empty(s), ph, lim)) { ok = false; break; }
                        const uint32_t x = smem0 + (uint32_t)(s * W_STAGE), y = x + X_BYTES;
                        const uint32_t bar = lead_full0 + 8u * s;
                        const int k = kb * BK;
                        if (elect_one()) {
                            if (rank == 0) mbar_expect_tx(full(s), 2 * W_STAGE);
                            tma_load_2d_pair(x, &tm_x, bar, p.x_mnmajor ? m : k, p.x_mnmajor ? k : m);
                            tma_load_2d_pair(y, &tm_y, bar, p.y_mnmajor ? n : k, p.y_mnmajor ? k : n);
                        }
                        ++filled;
                        if (++s == S) { s = 0; ph ^= 1; }
                    }
                }
                publish((int)rank, filled);
            }
        } else if (warp == 1) {
            // ------------------------------------------------ MMA issuer (the leader's)
            if (rank == 0) {
                int s = 0, b = 0, issued = 0;
                uint32_t ph = 0, bph = 1;
                const uint32_t x_step = p.x_mnmajor ? 4096u >> 4 : 32u >> 4;
                const uint32_t y_step = p.y_mnmajor ? 4096u >> 4 : 32u >> 4;
                for (int u = group; ok && u < units; u += groups) {
                    for (int kb = 0; kb < p.nkb; ++kb) {
                        if (!warp_wait(full(s), ph, lim) || !warp_wait(tempty(b), bph, lim)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t x = smem0 + (uint32_t)(s * W_STAGE), y = x + X_BYTES;
                        const uint64_t dx = smem_desc_8bit(x, X_BYTES), dy = smem_desc_8bit(y, X_BYTES);
                        const uint32_t d = tmem + (uint32_t)(b * WT);
                        if (elect_one()) {
#pragma unroll
                            for (int i = 0; i < BK / 32; ++i)
                                umma_8bit<true>(d, dx + i * x_step, dy + i * y_step, p.idesc, i > 0);
                            umma_commit_pair(empty(s));
                            umma_commit_pair(tfull(b));
                        }
                        ++issued;
                        if (++s == S) { s = 0; ph ^= 1; }
                        if (++b == 2) { b = 0; bph ^= 1; }
                    }
                }
                if (issued > 0)                    // MMAs retire before tensor memory is freed
                    mbar_wait_for(tfull((issued - 1) & 1), (uint32_t)((issued - 1) >> 1) & 1u, kDrainNs, &g_error);
                publish(2, issued);
            }
        } else if (YVEC && warp == 2) {
            // ------------------------------------------------ scales
            // copied asynchronously, up to SLOTS blocks' under way.  Scales of single
            // rows or columns are neighbours in memory; rows and columns past the
            // matrix take its last: any valid one will do.
            const uint32_t to = smem_u32(scales) + 4u * (uint32_t)lane;
            int slot = 0;
            uint32_t ph = 1;
            for (int u = group; ok && u < units; u += groups) {
                int tx, ty;
                tile_of(p, u, tx, ty);
                const int x0 = min(ty * WT + (int)rank * BX, p.M - 1), y0 = min(tx * WT, p.N - 1);
                const float *sx = p.SX + (int64_t)(x0 >> p.x_shift) * p.x_mn;
                const float *sy = p.SY + (int64_t)y0 * p.y_mn;
                for (int kb = 0; kb < p.nkb; ++kb) {
                    if (!warp_wait(sempty(slot), ph, lim)) { ok = false; break; }
                    const uint32_t at = to + 4u * (uint32_t)(slot * K_::BLOCK);
#pragma unroll
                    for (int j = 0; j < BX / 32; ++j)
                        cp_async_4(at + 128u * j, sx + (p.x_shift ? 0 : min(32 * j + lane, p.M - 1 - x0)), 4);
#pragma unroll
                    for (int j = 0; j < WT / 32; ++j)
                        cp_async_4(at + 4u * BX + 128u * j, sy + min(32 * j + lane, p.N - 1 - y0), 4);
                    sx += p.x_k;
                    sy += p.y_k;
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(sfull(slot)) : "memory");
                    if (++slot == K_::SLOTS) { slot = 0; ph ^= 1; }
                }
            }
            cp_async_wait_all();
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ promotion and epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(K_::REGS_PROMOTE));
        constexpr int PC = K_::PC, CH = K_::CH, NC = PC / CH;
        constexpr int BATCH = K_::BATCH;
        const int q = warp & 3, part = (warp - 4) >> 2;
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(part * PC);
        const uint32_t lead_tempty0 = leader_addr(tempty(0));
        float *stg = staging + (warp - 4) * (K_::OUT / 4);

        // One scale of B for the columns: it and the row's are fetched a batch ahead into
        // registers, across tiles, so that nothing here waits for memory: what a block
        // of k costs beside reading and adding its sums is what bounds this role.
        int fu = group, fkb = 0;                   // the batch to fetch next
        const float *fx = nullptr, *fy = nullptr;
        float nx[BATCH], ny[BATCH];
        auto fetch = [&]() {
            if (YVEC || fu >= units) return;
            if (fkb == 0) {
                int tx, ty;
                tile_of(p, fu, tx, ty);
                const int m = min(ty * WT + (int)rank * BX + q * 32 + lane, p.M - 1);
                const int n = min(tx * WT + part * PC, p.N - 1);
                fx = p.SX + (int64_t)(m >> p.x_shift) * p.x_mn;
                fy = p.SY + (int64_t)(n >> p.y_shift) * p.y_mn;
            }
#pragma unroll
            for (int a = 0; a < BATCH; ++a) {
                if (fkb + a < p.nkb) {
                    nx[a] = __ldg(fx);
                    ny[a] = __ldg(fy);
                    fx += p.x_k;
                    fy += p.y_k;
                }
            }
            fkb += BATCH;
            if (fkb >= p.nkb) { fkb = 0; fu += groups; }
        };
        fetch();

        int b = 0, slot = 0;
        uint32_t bph = 0, sph = 0;
        // (the reads under way while another chunk is added are held by the compiler in
        // place: no accumulator or sum may spill)
        uint32_t r[2][CH];
        auto read = [&](int c, uint32_t(&v)[CH]) {
            const uint32_t at = taddr + (uint32_t)(b * WT + c * CH);
            if (YVEC) tmem_ld_rows_async(at, v);
            else tmem_ld_async(at, v);
        };
        // waits for the next buffer (and its block's scales) and starts reading it: one
        // branch for both, with no read under way across it (two waits, the scales'
        // at the block's start: 192 us, not 167, at 4096 x 4096 x 8192 TN)
        auto next_buffer = [&]() {
            bool there = mbar_test(tfull(b), bph) && (!YVEC || mbar_test(sfull(slot), sph));
            if (!there)
                there = mbar_wait_for(tfull(b), bph, lim, &g_error) &&
                        (!YVEC || mbar_wait_for(sfull(slot), sph, lim, &g_error));
            ok = __all_sync(0xffffffffu, there);
            if (ok) {
                tc_fence_after();
                read(0, r[0]);
            }
        };
        for (int u = group; ok && u < units; u += groups) {
            int tx, ty;
            tile_of(p, u, tx, ty);
            float2 acc[PC / 2];
#pragma unroll
            for (int i = 0; i < PC / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
            float sv[BATCH];
            // (no tensor-memory read is under way across the epilogue: its registers could be moved)
            next_buffer();
            if (!ok) break;
            for (int kb = 0; kb < p.nkb; ++kb) {
                float2 s2[YVEC ? 4 : 1];
                const float *sc = scales + slot * K_::BLOCK;
                if (YVEC) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float s = sc[q * 32 + 8 * i + lane / 4];
                        s2[i] = make_float2(s, s);
                    }
                } else {
                    if (kb % BATCH == 0) {
#pragma unroll
                        for (int a = 0; a < BATCH; ++a) sv[a] = __fmul_rn(nx[a], ny[a]);
                        fetch();
                    }
                    s2[0] = make_float2(sv[0], sv[0]);
#pragma unroll
                    for (int a = 0; a + 1 < BATCH; ++a) sv[a] = sv[a + 1];
                }
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    uint32_t(&v)[CH] = r[c & 1];
                    float2 y2[CH / 8];             // (loaded while the sums arrive)
                    if (YVEC) {
#pragma unroll
                        for (int g = 0; g < CH / 8; ++g)
                            y2[g] = *reinterpret_cast<const float2 *>(sc + BX + part * PC + c * CH + 8 * g + 2 * (lane & 3));
                    }
                    tmem_ld_wait(v);
                    if (c + 1 < NC) {
                        read(c + 1, r[(c + 1) & 1]);
                    } else {
                        // the buffer is read: hand it back, and start on the next one
                        // while this chunk is added
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) remote_arrive_relaxed(lead_tempty0 + 8u * b);
                        if (++b == 2) { b = 0; bph ^= 1; }
                        if (YVEC) {            // (its scales are in registers)
                            if (lane == 0) mbar_arrive(sempty(slot));
                            if (++slot == K_::SLOTS) { slot = 0; sph ^= 1; }
                        }
                        if (kb + 1 < p.nkb) next_buffer();
                    }
                    if (YVEC) {
#pragma unroll
                        for (int g = 0; g < CH / 8; ++g) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int k = 16 * (i / 2) + 4 * g + 2 * (i % 2);
                                const float2 t = make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
                                float2 &a = acc[(c * CH + k) / 2];
                                a = __ffma2_rn(__fmul2_rn(t, s2[i]), y2[g], a);
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < CH; i += 2) {
                            const float2 t = make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                            float2 &a = acc[(c * CH + i) / 2];
                            a = __ffma2_rn(t, s2[0], a);
                        }
                    }
                }
                if (!ok) break;
            }
            if (!ok) break;
            // blocks of 32 rows x CH columns through shared memory (lane = row in), from
            // there to C by a TMA store; by one that adds where C += sums; or, where C's
            // alignment or the scalars do not allow it, by this warp
            const int m0 = ty * WT + (int)rank * BX + q * 32, n0 = tx * WT + part * PC;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (m0 >= p.M || n0 + c * CH >= p.N) break;
                const float2 *a = acc + c * CH / 2;
                if (lane == 0) tma_store_read_wait();
                __syncwarp();
                if (n0 + c * CH < p.c_tma) {
                    uint8_t *row = reinterpret_cast<uint8_t *>(stg);
                    if (YVEC) {
                        // (pairs of columns, of four rows a group)
#pragma unroll
                        for (int i = 0; i < CH / 2; ++i) {
                            const int y = lane / 4 + 8 * (i / 8 * 2 + i % 2), g = i / 2 % 4;
                            const float2 v = make_float2(__fmul_rn(p.alpha, a[i].x), __fmul_rn(p.alpha, a[i].y));
                            if (p.c_bf16)
                                *reinterpret_cast<uint32_t *>(row + y * 2 * CH + 16 * staged_chunk<2 * CH>(y, g) +
                                                              4 * (lane & 3)) = pack2(v.x, v.y);
                            else
                                *reinterpret_cast<float2 *>(row + y * 4 * CH + 16 * staged_chunk<4 * CH>(y, 2 * g + (lane & 3) / 2) +
                                                            8 * (lane & 1)) = v;
                        }
                    } else if (p.c_bf16) {
                        row += lane * 2 * CH;
#pragma unroll
                        for (int i = 0; i < CH / 8; ++i)
                            *reinterpret_cast<uint4 *>(row + 16 * staged_chunk<2 * CH>(lane, i)) = make_uint4(
                                pack2(__fmul_rn(p.alpha, a[4 * i].x), __fmul_rn(p.alpha, a[4 * i].y)),
                                pack2(__fmul_rn(p.alpha, a[4 * i + 1].x), __fmul_rn(p.alpha, a[4 * i + 1].y)),
                                pack2(__fmul_rn(p.alpha, a[4 * i + 2].x), __fmul_rn(p.alpha, a[4 * i + 2].y)),
                                pack2(__fmul_rn(p.alpha, a[4 * i + 3].x), __fmul_rn(p.alpha, a[4 * i + 3].y)));
                    } else {
                        row += lane * 4 * CH;
#pragma unroll
                        for (int i = 0; i < CH / 4; ++i)
                            *reinterpret_cast<float4 *>(row + 16 * staged_chunk<4 * CH>(lane, i)) =
                                make_float4(__fmul_rn(p.alpha, a[2 * i].x), __fmul_rn(p.alpha, a[2 * i].y),
                                            __fmul_rn(p.alpha, a[2 * i + 1].x), __fmul_rn(p.alpha, a[2 * i + 1].y));
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        if (!p.c_add) tma_store_2d<false>(&tm_c, smem_u32(stg), n0 + c * CH, m0);
                        else tma_store_2d<true>(&tm_c, smem_u32(stg), n0 + c * CH, m0);
                    }
                } else {
                    if (YVEC) {
#pragma unroll
                        for (int i = 0; i < CH / 2; ++i) {
                            const int y = lane / 4 + 8 * (i / 8 * 2 + i % 2), g = i / 2 % 4;
                            *reinterpret_cast<float2 *>(stg + y * CH + 4 * staged_chunk<4 * CH>(y, 2 * g + (lane & 3) / 2) +
                                                        2 * (lane & 1)) = a[i];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < CH / 4; ++i)
                            *reinterpret_cast<float4 *>(stg + lane * CH + 4 * staged_chunk<4 * CH>(lane, i)) =
                                make_float4(a[2 * i].x, a[2 * i].y, a[2 * i + 1].x, a[2 * i + 1].y);
                    }
                    __syncwarp();
                    const int64_t at = (int64_t)m0 * p.ldc + n0 + c * CH;
                    const int rows = p.M - m0, cols = p.N - n0 - c * CH;
                    const bool vec = p.c_vec != 0;
                    if (p.c_bf16) {
                        __nv_bfloat16 *C = static_cast<__nv_bfloat16 *>(p.C) + at;
                        if (p.beta != 0.0f) write_block<__nv_bfloat16, true>(C, p.ldc, p.alpha, p.beta, vec, stg, rows, cols);
                        else write_block<__nv_bfloat16, false>(C, p.ldc, p.alpha, p.beta, vec, stg, rows, cols);
                    } else {
                        float *C = static_cast<float *>(p.C) + at;
                        if (p.beta != 0.0f) write_block<float, true>(C, p.ldc, p.alpha, p.beta, vec, stg, rows, cols);
                        else write_block<float, false>(C, p.ldc, p.alpha, p.beta, vec, stg, rows, cols);
                    }
                }
            }
        }
        if (lane == 0) tma_store_read_wait();
    }

    tc_fence_before();
    cluster_sync_all();                            // no CTA leaves while its peer may still signal it
    const int f0 = (int)counts[0], f1 = (int)counts[1], multiplied = (int)counts[2];
    if (f0 != multiplied || f1 != multiplied) {
        // A role gave up, and stages were filled that no MMA waited for.  A stage is
        // complete with both CTAs' copies (counted on the leader's barrier): the CTA that
        // filled fewer fills the missing ones, which are free, since the other was let
        // into them; then the leader waits for what no MMA did.  Commits that reach both
        // CTAs have done so.
        if (warp == 0) {
            const int most = max(f0, f1);
            for (int i = rank == 0 ? f0 : f1; i < most; ++i) {
                const uint32_t x = smem0 + (uint32_t)(i % S * W_STAGE);
                if (elect_one()) {
                    if (rank == 0) mbar_expect_tx(full(i % S), 2 * W_STAGE);
                    tma_load_2d_pair(x, &tm_x, leader_addr(full(i % S)), 0, 0);
                    tma_load_2d_pair(x + X_BYTES, &tm_y, leader_addr(full(i % S)), 0, 0);
                }
                __syncwarp();
            }
            for (int i = max(most - S, 0); rank == 0 && i < most; ++i)
                mbar_wait_for(full(i % S), (uint32_t)(i / S) & 1u, kDrainNs, &g_error);
            if (rank == 1 && multiplied > 0) {
                const int last = multiplied - 1;
                mbar_wait_for(empty(last % S), (uint32_t)(last / S) & 1u, kDrainNs, &g_error);
                mbar_wait_for(tfull(last & 1), (uint32_t)(last >> 1) & 1u, kDrainNs, &g_error);
            }
        }
        __syncwarp();
        cluster_sync_all();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_free<true>(tmem, 512);
    }
}

// C = beta * C (no product term)
__global__ void __launch_bounds__(256) scale_kernel(const Params p) {
    const int64_t total = (int64_t)p.M * p.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t at = i / p.N * p.ldc + i % p.N;
        const float v = p.beta == 0.0f ? 0.0f : __fmul_rn(p.beta, load_c(p, at));
        if (p.c_bf16) static_cast<__nv_bfloat16 *>(p.C)[at] = __float2bfloat16_rn(v);
        else static_cast<float *>(p.C)[at] = v;
    }
}

// Rows of bytes to rows that start on 16 bytes (what a TMA map asks for); one
// operand for blockIdx.y == 0, the other for 1.
struct CopyJob {
    const uint8_t *src;
    uint8_t *dst;
    int64_t ld_src, ld_dst;
    int rows, cols;
};
__global__ void __launch_bounds__(256) align_rows_kernel(const CopyJob j0, const CopyJob j1) {
    const CopyJob j = blockIdx.y == 0 ? j0 : j1;
    const int per_row = (j.cols + 15) / 16;
    const int64_t total = (int64_t)j.rows * per_row;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per_row;
        const int c = (int)(i - row * per_row) * 16;
        const uint8_t *src = j.src + row * j.ld_src + c;
        uint32_t w[4];
        if (c >= 4 && c + 20 <= j.cols) {
            // five aligned words of this row hold the 16 bytes
            const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(src) & 3);
            const uint32_t *a = reinterpret_cast<const uint32_t *>(src - off);
            uint32_t v[5];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = __ldg(a + k);
            v[4] = off ? __ldg(a + 4) : 0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(v[k], v[k + 1], 8 * off);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w[k] = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (c + 4 * k + b < j.cols) w[k] |= (uint32_t)src[4 * k + b] << (8 * b);
            }
        }
        *reinterpret_cast<uint4 *>(j.dst + row * j.ld_dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace fp8g

// ---------------------------------------------------------------- host side
int fp8_take_device_error() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, fp8g::g_error, sizeof(v)) != cudaSuccess) return SGEMM_ERR_CUDA;
    if (v != 0 && cudaMemcpyToSymbol(fp8g::g_error, &zero, sizeof(zero)) != cudaSuccess)
        return SGEMM_ERR_CUDA;
    return v == 0 ? SGEMM_OK : (int)v;
}

// A row-major array of bytes, `rows` x `cols`, in boxes of box_rows x 128 bytes
// with the 128-byte swizzle; outside reads as zeros.
static bool byte_map(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld};
    cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One launch, with the shared-memory opt-in made once on each device (bit d of `done`).
template <typename Kern, typename... Args>
static int launch_kernel(Kern kern, uint64_t &done, int grid, int threads, int smem, int cluster, cudaStream_t s,
                         bool dep, const Args &...args) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SGEMM_ERR_CUDA;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (!bit || !(__atomic_load_n(&done, __ATOMIC_ACQUIRE) & bit)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, fp8g::SMEM_MAX) !=
            cudaSuccess)
            return launch_status();
        __atomic_fetch_or(&done, bit, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    if (dep) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    timing_mark(s, true);
    count_launch();
    cudaLaunchKernelEx(&cfg, kern, args...);
    timing_mark(s, false);
    return launch_status();
}

template <int BY, bool XVEC>
static int launch_fp8(const CUtensorMap &mx, const CUtensorMap &my, const fp8g::Params &p, int grid,
                      int smem, cudaStream_t s, bool dep) {
    static uint64_t done = 0;
    return launch_kernel(fp8g::fp8_gemm_kernel<BY, XVEC>, done, grid, fp8g::THREADS, smem, p.ksplit, s, dep, mx, my, p);
}

template <bool YVEC>
static int launch_wide(const CUtensorMap &mx, const CUtensorMap &my, fp8g::Params &p, int grid, cudaStream_t s,
                       bool dep) {
    using K_ = fp8g::Wide<YVEC>;
    static uint64_t done = 0;
    // C in boxes of 32 rows x CH columns, where TMA can write it: rows on 16 bytes,
    // and nothing to read, or C += sums in fp32 (one rounding, as the epilogue's;
    // subnormal numbers are kept, measured on GB300).  A
    // store writes all 16 bytes that hold C's last column (measured on GB300), so the last
    // box goes the other way where C ends inside them.
    const int esize = p.c_bf16 ? 2 : 4;
    CUtensorMap mc = mx;
    p.c_tma = 0;
    p.c_add = p.beta != 0.0f;
    if (aligned16(p.C) && p.ldc * esize % 16 == 0 &&
        (p.beta == 0.0f || (p.beta == 1.0f && p.alpha == 1.0f && !p.c_bf16))) {
        EncodeTiledFn enc = encode_fn();
        cuuint64_t dims[2] = {(cuuint64_t)p.N, (cuuint64_t)p.M};
        cuuint64_t strides[1] = {(cuuint64_t)(p.ldc * esize)};
        cuuint32_t box[2] = {(cuuint32_t)K_::CH, 32};
        cuuint32_t es[2] = {1, 1};
        const int bytes = K_::CH * esize;
        if (enc && enc(&mc, p.c_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p.C, dims,
                       strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       bytes == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                       : bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                     : CU_TENSOR_MAP_SWIZZLE_32B,
                       CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS)
            p.c_tma = (int64_t)p.N * esize % 16 == 0 ? p.N : p.N / K_::CH * K_::CH;
    }
    return launch_kernel(fp8g::fp8_wide_kernel<YVEC>, done, grid, K_::THREADS, K_::SMEM, 1, s, dep, mx, my, mc, p);
}

template <int BY>
static int launch_fp8(bool xvec, const CUtensorMap &mx, const CUtensorMap &my, const fp8g::Params &p,
                      int grid, int smem, cudaStream_t s, bool dep) {
    return xvec ? launch_fp8<BY, true>(mx, my, p, grid, smem, s, dep)
                : launch_fp8<BY, false>(mx, my, p, grid, smem, s, dep);
}

static int run_fp8(char ta, char tb, int64_t M, int64_t N, int64_t K, float alpha, const void *A,
                   int a_type, int64_t lda, const float *SA, int a_group, int64_t ldsa, const void *B,
                   int b_type, int64_t ldb, const float *SB, int b_group, int64_t ldsb, float beta,
                   void *C, int c_type, int64_t ldc, cudaStream_t s) {
    int sms = 0;
    int st = usable_device(&sms);
    if (st != SGEMM_OK) return st;
    fp8g::Params p{};
    p.C = C; p.ldc = ldc; p.c_bf16 = c_type == SGEMM_TYPE_BF16;
    p.M = (int)M; p.N = (int)N;
    p.alpha = alpha; p.beta = beta;
    if (K == 0 || alpha == 0.0f) {
        if (beta == 1.0f) return SGEMM_OK;
        const int64_t blocks = std::min<int64_t>((M * N + 255) / 256, (int64_t)sms * 8);
        count_launch();
        fp8g::scale_kernel<<<(unsigned)blocks, 256, 0, s>>>(p);
        return launch_status();
    }
    const bool a_mn = !is_notrans(ta), b_mn = is_notrans(tb);
    const int64_t a_rows = a_mn ? K : M, a_cols = a_mn ? M : K;
    const int64_t b_rows = b_mn ? K : N, b_cols = b_mn ? N : K;
    // an operand that TMA cannot read in place is copied with rows on 16 bytes
    auto in_place = [](const void *q, int64_t ld, int64_t rows) { return aligned16(q) && (ld % 16 == 0 || rows == 1); };
    auto up16 = [](int64_t v) { return (v + 15) / 16 * 16; };
    const bool copy_a = !in_place(A, lda, a_rows), copy_b = !in_place(B, ldb, b_rows);
    if (copy_a || copy_b) {
        const int64_t la = up16(a_cols), lb = up16(b_cols);
        const size_t bytes_a = copy_a ? ((size_t)a_rows * la + 255) / 256 * 256 : 0;
        const size_t bytes_b = copy_b ? (size_t)b_rows * lb : 0;
        void *ws = nullptr;
        st = workspace(s, bytes_a + bytes_b, &ws);
        if (st != SGEMM_OK) return st;
        uint8_t *w = static_cast<uint8_t *>(ws);
        fp8g::CopyJob j[2];
        int n = 0;
        int64_t most = 0;
        if (copy_a) {
            j[n++] = fp8g::CopyJob{static_cast<const uint8_t *>(A), w, lda, la, (int)a_rows, (int)a_cols};
            A = w;
            lda = la;
            most = a_rows * (la / 16);
        }
        if (copy_b) {
            j[n++] = fp8g::CopyJob{static_cast<const uint8_t *>(B), w + bytes_a, ldb, lb, (int)b_rows, (int)b_cols};
            B = w + bytes_a;
            ldb = lb;
            most = std::max(most, b_rows * (lb / 16));
        }
        const unsigned blocks = (unsigned)std::min<int64_t>((most + 255) / 256, (int64_t)sms * 16);
        count_launch();
        fp8g::align_rows_kernel<<<dim3(blocks, (unsigned)n), 256, 0, s>>>(j[0], j[n - 1]);
        st = launch_status();
        if (st != SGEMM_OK) return st;
    }
    // (a single row may have any leading dimension; its map takes a valid one)
    if (lda % 16 != 0) lda = up16(lda);
    if (ldb % 16 != 0) ldb = up16(ldb);

    const Fp8Plan pl = fp8_plan(M, N, K, b_group, sms);
    const bool dep = copy_a || copy_b;
    // scales: strides along M or N and along the sum, for each operand
    const int64_t a_mn_stride = a_group == 1 || a_mn ? 1 : ldsa, a_k_stride = a_group == 1 || a_mn ? ldsa : 1;
    const int64_t b_mn_stride = b_group == 1 || b_mn ? 1 : ldsb, b_k_stride = b_group == 1 || b_mn ? ldsb : 1;
    const int a_shift = a_group == 1 ? 0 : 7, b_shift = b_group == 1 ? 0 : 7;
    p.nkb = (int)fp8::blocks_of(K);
    p.c_vec = reinterpret_cast<uintptr_t>(C) % (p.c_bf16 ? 8 : 16) == 0 && ldc % 4 == 0;
    p.ksplit = pl.ksplit;
    p.wait_ns = tc_wait_limit();
    const int a5 = a_type == SGEMM_TYPE_E5M2, b5 = b_type == SGEMM_TYPE_E5M2;
    const int64_t tiles = ((N + pl.bx - 1) / pl.bx) * ((M + pl.by - 1) / pl.by);
    if (tiles > INT32_MAX / 16) return SGEMM_ERR_UNSUPPORTED;
    p.tiles_x = (int)((N + pl.bx - 1) / pl.bx);
    p.tiles_y = (int)((M + pl.by - 1) / pl.by);
    CUtensorMap mx, my;
    if (pl.bx == fp8g::WT) {
        // the wide kernel: X is A, Y is B
        p.SX = SA; p.x_mn = a_mn_stride; p.x_k = a_k_stride; p.x_shift = a_shift; p.x_mnmajor = a_mn;
        p.SY = SB; p.y_mn = b_mn_stride; p.y_k = b_k_stride; p.y_shift = b_shift; p.y_mnmajor = b_mn;
        p.group_y = 8;
        p.idesc = tc::idesc_8bit(a5, b5, a_mn, b_mn, fp8g::WT, fp8g::WT);
        if (!byte_map(&mx, A, a_rows, a_cols, lda, 128) || !byte_map(&my, B, b_rows, b_cols, ldb, 128))
            return SGEMM_ERR_UNSUPPORTED;
        const int grid = 2 * (int)std::min<int64_t>(tiles, std::max(sms / 2, 1));
        return b_group == 1 ? launch_wide<true>(mx, my, p, grid, s, dep)
                            : launch_wide<false>(mx, my, p, grid, s, dep);
    }
    // the narrow kernel: X is B, Y is A
    p.SX = SB; p.x_mn = b_mn_stride; p.x_k = b_k_stride; p.x_shift = b_shift; p.x_mnmajor = b_mn;
    p.SY = SA; p.y_mn = a_mn_stride; p.y_k = a_k_stride; p.y_shift = a_shift; p.y_mnmajor = a_mn;
    p.group_y = 16;
    p.y_bytes = a_mn ? fp8g::X_BYTES : pl.by * fp8g::BK;
    const int fixed = 1024 + fp8g::SCALE_SLOTS * pl.by * 4 + fp8g::BAR_BYTES;
    p.stages = std::min(fp8g::MAX_STAGES, (fp8g::SMEM_MAX - fixed) / (fp8g::X_BYTES + p.y_bytes));
    p.idesc = tc::idesc_8bit(b5, a5, b_mn, a_mn, fp8g::BX, pl.by);
    if (!byte_map(&mx, B, b_rows, b_cols, ldb, 128) || !byte_map(&my, A, a_rows, a_cols, lda, a_mn ? 128 : pl.by))
        return SGEMM_ERR_UNSUPPORTED;
    const int grid = p.ksplit > 1 ? (int)tiles * p.ksplit : (int)std::min<int64_t>(tiles, sms);
    const int smem = fixed + p.stages * (fp8g::X_BYTES + p.y_bytes);
    const bool xvec = b_group == 1;
    switch (pl.by) {
    case 16: return launch_fp8<16>(xvec, mx, my, p, grid, smem, s, dep);
    case 32: return launch_fp8<32>(xvec, mx, my, p, grid, smem, s, dep);
    case 64: return launch_fp8<64>(xvec, mx, my, p, grid, smem, s, dep);
    default: return launch_fp8<128>(xvec, mx, my, p, grid, smem, s, dep);
    }
}

}  // namespace sgemm_gb300

using namespace sgemm_gb300;

extern "C" int sgemm_fp8(char transA, char transB, int64_t M, int64_t N, int64_t K, float alpha,
                         const void *A, int a_type, int64_t lda, const float *SA, int a_group,
                         int64_t ldsa, const void *B, int b_type, int64_t ldb, const float *SB,
                         int b_group, int64_t ldsb, float beta, void *C, int c_type, int64_t ldc,
                         sgemm_stream_t stream) {
    const int64_t lim = INT32_MAX - 255;           // tiles are rounded up in int
    if (!is_notrans(transA) && !is_trans(transA)) return -1;
    if (!is_notrans(transB) && !is_trans(transB)) return -2;
    if (M < 0 || M > lim) return -3;
    if (N < 0 || N > lim) return -4;
    if (K < 0 || K > lim) return -5;
    const bool an = is_notrans(transA), bn = is_notrans(transB);
    const bool need = M > 0 && N > 0 && K > 0 && alpha != 0.0f;
    auto scales_row = [&](int group, int64_t mn, int64_t stored_cols) {
        return std::max<int64_t>(1, group == 1 ? mn : fp8::blocks_of(stored_cols));
    };
    if (need && A == nullptr) return -7;
    if (!fp8::is_code_type(a_type)) return -8;
    if (lda < std::max<int64_t>(1, an ? K : M)) return -9;
    if (need && (SA == nullptr || reinterpret_cast<uintptr_t>(SA) % 4 != 0)) return -10;
    if (a_group != 1 && a_group != fp8::GROUP) return -11;
    if (ldsa < scales_row(a_group, M, an ? K : M)) return -12;
    if (need && B == nullptr) return -13;
    if (!fp8::is_code_type(b_type)) return -14;
    if (ldb < std::max<int64_t>(1, bn ? N : K)) return -15;
    if (need && (SB == nullptr || reinterpret_cast<uintptr_t>(SB) % 4 != 0)) return -16;
    if (b_group != 1 && b_group != fp8::GROUP) return -17;
    if (ldsb < scales_row(b_group, N, bn ? N : K)) return -18;
    if (!fp8::is_float_type(c_type)) return -21;
    if (M > 0 && N > 0 && (C == nullptr || reinterpret_cast<uintptr_t>(C) % (c_type == SGEMM_TYPE_F32 ? 4 : 2) != 0))
        return -20;
    if (ldc < std::max<int64_t>(1, N)) return -22;
    if (M == 0 || N == 0) return SGEMM_OK;
    try {
        return run_fp8(transA, transB, M, N, K, alpha, A, a_type, lda, SA, a_group, ldsa, B, b_type, ldb,
                       SB, b_group, ldsb, beta, C, c_type, ldc, reinterpret_cast<cudaStream_t>(stream));
    } catch (const std::bad_alloc &) {
        return SGEMM_ERR_NOMEM;
    }
}

extern "C" int sgemm_fp8_plan(int64_t M, int64_t N, int64_t K, int b_group, int num_sms, int *out_tile_m,
                              int *out_tile_n, int *out_ksplit) {
    if (M < 1 || M > INT32_MAX - 255) return -1;
    if (N < 1 || N > INT32_MAX - 255) return -2;
    if (K < 1 || K > INT32_MAX - 255) return -3;
    if (b_group != 1 && b_group != fp8::GROUP) return -4;
    if (num_sms <= 0) return -5;
    const Fp8Plan pl = fp8_plan(M, N, K, b_group, num_sms);
    if (out_tile_m) *out_tile_m = pl.by;
    if (out_tile_n) *out_tile_n = pl.bx;
    if (out_ksplit) *out_ksplit = pl.ksplit;
    return SGEMM_OK;
}
