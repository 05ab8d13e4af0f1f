// Few rows of x (decode) against a matrix that is read once from memory: bf16 weights of a
// feed-forward block, or 4-bit weights with group scales.
//
//   c(m,n) = sum over groups b of s(n,b) (sum_{k in b} x(m,k) (code(n,k) - zero(n,b)))
//
// Bound by the weights' stream, and with 4 bits nearly as much by the instructions that take
// them apart.  A warp holds 32 rows of W (or 16 of each of two matrices) and walks stages of
// 128 bytes of each row, brought by TMA into a ring of its own: what is under way does
// not depend on how far the warp is, and starts before x is there; a row's or the
// matrix's end reads as zeros.  The products are mma.sync (exact products, fp32 sums): W's
// rows are the MMA's 16 rows, x's rows its 8 columns.  Which k an MMA calls its first is
// free as long as both operands agree, so a lane's neighbouring bytes are its share of the
// fragments as they lie; x is laid out once in shared memory in the order in which
// lanes read it.
//   4 bits: the codes of a word come out by one shift and four logic operations, which also
//   set the exponent of 1024 in each half: 1024 + code, or 1024 + 16 code for the upper four
//   bits of a byte, exact in fp16; the same with the zero code is subtracted (exact), so that
//   nothing cancels and infinities in x keep their meaning; x is divided by 16 where codes
//   are 16 times larger.  x is held in fp16, each block of 128 of a row times a power of two
//   that brings its largest value to 2^14 .. 2^15: bf16 as it is, but for values below 2^-27 of
//   the block's largest; fp32 in two parts, in columns of their own, the second 2^11
//   times what the first leaves.  An MMA never spans two groups; a group's sum is scaled
//   into the fp32 accumulator.
//   (Integers made into numbers by the exponent's bits, and odd ones left 16 times larger, are a
//   published way with 4-bit weights: Kim, Henry, Fahim and Awadalla, "Who Says Elephants Can't
//   Run", 2022.  The order of k, the exact zero codes and the factor on x's side are this kernel's.)
//   Tried for 1 x 16384 x 8192 on earlier forms of the kernel, which took 33 us with weights loaded into
//   registers and 22.5 when the rings were new (18.9 now): codes as bf16 numbers, 128 + code (11
//   operations a word, not 9), 27 us; as E4M3 bytes (3) 29; zero codes taken off a group's sum
//   instead (5 a word, but fp32 results 2e-6 off, four times as much as fp32 arithmetic) 25,
//   with loads into registers.  A code's bits alone are an fp16 number, too, but a subnormal
//   one, and sums came out with up to 7 bits fewer (1.4e-6 off).  8-bit integer MMAs take 65
//   clocks each, 8 times these.
// The sum is cut over the warps of a CTA (which take stages in turn, so that neighbours in
// memory are read together) and over a cluster of CTAs; the partial sums meet
// through (distributed) shared memory in a fixed order: no workspace, no atomics.
// Waits for TMA are bounded; where one runs out the error word is set, and the warp leaves
// after what it has under way has landed (waited for, again bounded).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "act.cuh"
#include "few.h"
#include "plan.h"
#include "ptx_util.cuh"
#include "tc_gemm.h"
#include "tc_ptx.cuh"

namespace sgemm_gb300 {
namespace few {

using namespace tc;

constexpr int WARPS = kFewWarps;
constexpr int THREADS = 32 * WARPS;
constexpr int STAGE = kFewStage;
constexpr int RED = 36;                        // floats of a column of 32 partial sums: no bank twice
constexpr uint64_t kDrainNs = 1000000000ull;
// (4 bits) Sums are held this many times smaller than they are until a warp has its own: a group's, 15 *
// 128 times the largest of x at most, then stays below 2^128 before its scale is on it.  (What it
// costs is bits of results below 2^-115.  Without it x from 2^117 on and a small scale gave an
// infinity; scales multiplied first lose bits of results below 2^-101; found out and held smaller
// for a CTA's range of x only where x is that large, 2 to 5 % of the time of every call.)
constexpr float ACC = 2048.0f;

struct Params {
    const void *x;
    int64_t ldx;
    const float *s[2];
    const uint8_t *z[2];
    uint32_t lds;
    void *c;
    int64_t ldc;
    int M, N, K;
    int gated, act, c_f32, c_vec, x_f32, x_vec;
    int per_block;                             // rows of x in a block of columns
    int wk, ks, stages, depth, ring;
    int groups;
    int early;                                 // weights may be read before pdl_wait
    unsigned int *error;                       // device error word
    unsigned long long wait_ns;
};

// 16 rows of W times 8 columns of x over 16 of k: the first of a sum, and one added to it.
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (word & mask) | the exponents of 1024.
__device__ __forceinline__ uint32_t codes_of(uint32_t word, uint32_t mask) {
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(word), "r"(mask), "r"(0x64006400u));
    return v;
}
__device__ __forceinline__ uint32_t subtract(uint32_t a, uint32_t b) {
    uint32_t v;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(v) : "r"(a), "r"(b));
    return v;
}

// G: 0 bf16, else the group.  A stage is two chunks of 64 bytes of a row, of which a lane
// has four words; t is its place among the four lanes of a row.
template <int G>
struct Row {
    static constexpr int KC = G ? 128 : 32;                // k of a chunk
    static constexpr int GROUPS = G ? 128 / (G ? G : 1) : 1;   // of a chunk
    static constexpr int IN_GROUP = 4 / GROUPS;            // words of a lane in a group
    static constexpr int UNITS = G ? 4 : 1;                // 16-byte pieces of x for a lane, column and chunk
    // Of x's piece of 8 values from 8 p on in a chunk: the word whose codes it meets, and the lane.
    __device__ static __forceinline__ int word_of(int p) { return G == 128 ? p % 4 : G == 64 ? p / 8 * 2 + p % 2 : p / 4; }
    __device__ static __forceinline__ int lane_of(int p) { return G == 128 ? p / 4 : G == 64 ? p % 8 / 2 : p % 4; }
    // A lane's words of chunk `half` of a staged row: its 16-byte pieces are where TMA's
    // swizzle put them.
    __device__ static __forceinline__ void words(const uint8_t *stage, int row, int half, int t, uint32_t (&w)[4]) {
        const uint8_t *at = stage + row * 128;
        auto piece = [&](int c) { return at + 16 * ((4 * half + c) ^ (row & 7)); };
        if (G == 0 || G == 128) {
            const uint4 q = *reinterpret_cast<const uint4 *>(piece(t));
            w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
        } else if (G == 64) {
            const uint2 a = *reinterpret_cast<const uint2 *>(piece(t / 2) + 8 * (t & 1));
            const uint2 b = *reinterpret_cast<const uint2 *>(piece(2 + t / 2) + 8 * (t & 1));
            w[0] = a.x; w[1] = a.y; w[2] = b.x; w[3] = b.y;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint32_t *>(piece(i) + 4 * t);
        }
    }
};

__device__ __forceinline__ float4 load_rank(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile("{\n\t.reg .u32 a;\n\t"
                 "mapa.shared::cluster.u32 a, %4, %5;\n\t"
                 "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr), "r"(rank) : "memory");
    return v;
}
__device__ __forceinline__ void add4(float4 &a, const float4 &b) {
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
}

// Eight values of a row of x from k on (zero from K on): bf16 as they are, in pairs, or as fp32.
// What does not start on 16 bytes, or ends inside them, goes element by element, in a
// function of its own: laying out x runs through its code once, so code counts.
static __device__ __noinline__ uint4 slow_bf16(const Params &p, int m, int k) {
    const uint16_t *from = static_cast<const uint16_t *>(p.x) + m * p.ldx + k;
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = (k + 2 * e < p.K ? (uint32_t)from[2 * e] : 0u) | (k + 2 * e + 1 < p.K ? (uint32_t)from[2 * e + 1] << 16 : 0u);
    return make_uint4(v[0], v[1], v[2], v[3]);
}
static __device__ __noinline__ uint4 slow_f32(const Params &p, int m, int k) {
    const uint32_t *from = static_cast<const uint32_t *>(p.x) + m * p.ldx + k;
    return make_uint4(k < p.K ? from[0] : 0u, k + 1 < p.K ? from[1] : 0u, k + 2 < p.K ? from[2] : 0u, k + 3 < p.K ? from[3] : 0u);
}
__device__ __forceinline__ uint4 load_bf16(const Params &p, int m, int k) {
    if (p.x_vec && k + 8 <= p.K)
        return *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + m * p.ldx + k);
    return slow_bf16(p, m, k);
}
template <bool F32>
struct Eight {                                 // values, as they are stored
    uint4 a, b;
    __device__ __forceinline__ void load(const Params &p, int m, int k) {
        if (!F32) {
            a = load_bf16(p, m, k);
        } else if (p.x_vec && k + 8 <= p.K) {
            const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const float *>(p.x) + m * p.ldx + k);
            a = from[0];
            b = from[1];
        } else {
            a = slow_f32(p, m, k);
            b = slow_f32(p, m, k + 4);
        }
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = __uint_as_float(F32 ? w[e] : e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
};

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return max(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
template <int G, bool ZEROS, int NT>
__global__ void __launch_bounds__(THREADS, NT <= 2 ? 2 : 1)
    few_kernel(const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1, const Params p) {
    using R = Row<G>;
    constexpr int KC = R::KC, U = R::UNITS, GROUPS = 2 * R::GROUPS;       // groups of a stage
    constexpr int PAD = G ? 1 : 0;                         // 16 bytes: so that a quad's writes meet in no bank
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[WARPS][kFewRing];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint4 *xs = reinterpret_cast<uint4 *>(smem + p.ring * WARPS * STAGE);  // [chunk][piece][column][t]
    float *red = reinterpret_cast<float *>(smem);          // [warp][column][RED], after the products
    const int lane = threadIdx.x & 31, warp = warp_index(), t = lane & 3;
    const int rank = p.ks > 1 ? (int)cluster_rank() : 0;
    const int kw = warp % p.wk, rw = warp / p.wk;
    const int per_warp = p.gated ? 16 : 32, per_cta = per_warp * (WARPS / p.wk);
    const int block_row = (int)blockIdx.x / p.ks * per_cta, row0 = block_row + rw * per_warp;
    const int m0 = (int)blockIdx.y * p.per_block;
    const int parts = G && p.x_f32 ? 2 : 1;
    const int rows = min(p.per_block, p.M - m0), cols = rows * parts;
    // (4 bits) of each chunk, the power of two that each column is to be multiplied by
    const int unit_step = 4 * cols + PAD;                  // from piece to piece
    float *units = reinterpret_cast<float *>(xs + 2 * p.depth * U * unit_step);
    // this CTA's stages, and this warp's among them: kw, kw + wk, ..
    const int s_begin = (int)((int64_t)p.stages * rank / p.ks), s_end = (int)((int64_t)p.stages * (rank + 1) / p.ks);
    const int mine = max(0, (s_end - s_begin - kw + p.wk - 1) / p.wk);
    uint8_t *ring = smem + warp * p.ring * STAGE;
    const uint32_t ring0 = smem_u32(ring), bar0 = smem_u32(&bars[warp][0]);

    auto issue = [&](int i, int slot) {                    // the warp's i-th stage
        if (elect_one()) {
            const uint32_t to = ring0 + (uint32_t)(slot * STAGE), bar = bar0 + 8u * slot;
            const int at = (s_begin + kw + i * p.wk) * 128;
            mbar_expect_tx(bar, STAGE);
            tma_load_2d(to, &map0, bar, at, row0);
            if (p.gated) tma_load_2d(to + STAGE / 2, &map1, bar, at, row0);
        }
        __syncwarp();
    };
    if (lane == 0) {
        for (int i = 0; i < p.ring; ++i) mbar_init(bar0 + 8u * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&map0);
        if (p.gated) prefetch_map(&map1);
    }
    __syncwarp();
    int issued = 0;
    auto fill = [&]() {
        for (; issued < min(p.ring, mine); ++issued) issue(issued, issued);
    };
    if (p.early) fill();                                   // (the kernel before writes no weights)

    // scales and zero codes of a stage: lane l has those of the warp's row l (by plain loads: the kernel
    // before may still be writing them when this one starts, so they are no constants of it)
    const int which = p.gated ? lane >> 4 : 0;
    const uint32_t n = (uint32_t)min(row0 + (p.gated ? lane & 15 : lane), p.N - 1);     // (rows past N: any valid one)
    float scale[G ? GROUPS : 1];
    uint32_t zero[G ? GROUPS : 1];             // (as loaded: what is made of them here would wait for them)
    auto fetch = [&](int i) {
        if constexpr (G != 0) {
            if (i >= mine) return;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                const int group = (s_begin + kw + i * p.wk) * GROUPS + g;
                const uint32_t at = (uint32_t)group * p.lds + n;
                const bool there = group < p.groups;
                scale[g] = there ? p.s[which][at] : 0.0f;
                if (ZEROS) zero[g] = there ? p.z[which][at] : 0u;
            }
        }
    };
    if (p.early) fetch(0);

    // (lanes of columns past the last read the last: their sums reach nothing)
    int column[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) column[j] = min(8 * j + lane / 4, cols - 1) * 4 + t;
    float acc[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][j][k] = 0.0f;

    pdl_wait();                                            // x may be written by the kernel before
    pdl_trigger();
    if (!p.early) {
        fill();
        fetch(0);
    }
    bool ok = true;
    int done = 0, slot = 0;
    uint32_t phase = 0;
    for (int s0 = s_begin; s0 < s_end; s0 += p.depth) {
        const int s1 = min(s0 + p.depth, s_end);
        if (s0 != s_begin) __syncthreads();                // x is no longer read
        // x into the order of the fragments: 64 quads of threads, each at (row, chunk) in turn
        const int chunks = 2 * (s1 - s0), quad = (int)threadIdx.x >> 2;
        int m = quad % rows, chunk = quad / rows;
        const int step_m = (THREADS / 4) % rows, step = (THREADS / 4) / rows;
        auto next = [&]() {
            m += step_m;
            chunk += step;
            if (m >= rows) {
                m -= rows;
                ++chunk;
            }
        };
        if (G == 0) {
            while (chunk < chunks) {
                constexpr int BATCH = 4;                   // loads under way
                int at[BATCH];
                uint4 v[BATCH];
#pragma unroll
                for (int b = 0; b < BATCH; ++b) {
                    at[b] = chunk < chunks ? chunk * unit_step + 4 * m + t : -1;
                    if (chunk < chunks) v[b] = load_bf16(p, m0 + m, (2 * s0 + chunk) * KC + 8 * t);
                    next();
                }
#pragma unroll
                for (int b = 0; b < BATCH; ++b)
                    if (at[b] >= 0) xs[at[b]] = v[b];
            }
        } else {
            auto lay_out = [&](auto f32) {
                constexpr bool F32 = decltype(f32)::value != 0;
                constexpr int PARTS = F32 ? 2 : 1;
                constexpr bool AHEAD = !F32 && NT >= 4;
                Eight<F32> there[4];
                auto load = [&]() {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (chunk < chunks) there[i].load(p, m0 + m, (2 * s0 + chunk) * KC + 8 * (4 * i + t));
                        else there[i].a = there[i].b = make_uint4(0, 0, 0, 0);
                    }
                };
                if (AHEAD) load();
#pragma unroll 1
                while (__any_sync(0xffffffffu, chunk < chunks)) {
                    // a chunk of 128 of a row for each quad: pieces next to each other by lanes
                    // next to each other, 32 bytes a lane in 128 of a row (by the lane that
                    // reads them, 4 lines for each quad's load, it took a third of 16 x 4096 x 8192);
                    // AHEAD: the next one's loads are under way meanwhile (bf16 32 x 4096 x 8192 18.3 us, not
                    // 23.4; 64 x 8192 x 4096 29.8, not 34.3; with 16 rows, whose quads have half as much to do, 15.0, not 13.5, and
                    // fp32 values take too many registers: 32 x 4096 x 8192 40.5 us, not 34.8)
                    const int row = m, to_chunk = chunk;
                    const bool live = chunk < chunks;
                    if (!AHEAD) load();
                    float v[4][8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) there[i].values(v[i]);
                    next();
                    if (AHEAD) load();
                    uint32_t most = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(v[i][e]) & 0x7fffffffu);
                    most = quad_max(most);
                    const bool odd = most >= 0x7f800000u;          // not all finite: the largest that is
                    if (__any_sync(0xffffffffu, odd)) {
                        uint32_t finite = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const uint32_t bits = __float_as_uint(v[i][e]) & 0x7fffffffu;
                                finite = max(finite, bits < 0x7f800000u ? bits : 0u);
                            }
                        most = quad_max(finite);
                    }
                    // (blocks below 2^-101 as if their largest were that: the factors stay normal)
                    const int exponent = max((int)(most >> 23), 26);
                    const float power = __uint_as_float((uint32_t)(268 - exponent) << 23);
                    if (live) {
#pragma unroll
                        for (int part = 0; part < PARTS; ++part) {
                            const int col = row * PARTS + part;
                            uint4 *to = xs + to_chunk * U * unit_step + 4 * col;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                // codes leave a word as (0, 4), (1, 5), (2, 6), (3, 7), the odd ones 16 times larger
                                uint32_t w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    float &lower = v[i][e], &upper = v[i][e + 4];
                                    if (part == 0) {
                                        lower *= e % 2 ? power * 0.0625f : power;
                                        upper *= e % 2 ? power * 0.0625f : power;
                                    }
                                    const __half2 h = __floats2half2_rn(lower, upper);
                                    w[e] = *reinterpret_cast<const uint32_t *>(&h);
                                    if (part + 1 < PARTS) {
                                        // what a second part holds: nothing of what is not finite
                                        const float2 back = __half22float2(h);
                                        lower = odd && !(fabsf(back.x) < __int_as_float(0x7f800000)) ? 0.0f : (lower - back.x) * 2048.0f;
                                        upper = odd && !(fabsf(back.y) < __int_as_float(0x7f800000)) ? 0.0f : (upper - back.y) * 2048.0f;
                                    }
                                }
                                to[R::word_of(4 * i + t) * unit_step + R::lane_of(4 * i + t)] = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                            // (2^11 smaller than they are: see ACC)
                            if (t == 0)
                                units[to_chunk * (8 * NT) + col] = __uint_as_float((uint32_t)(exponent - 14 - 11 * part) << 23) * (1.0f / ACC);
                        }
                    }
                }
            };
            if (p.x_f32) lay_out(act::Constant<1>());
            else lay_out(act::Constant<0>());
        }
        __syncthreads();

        for (; ok && done < mine && s_begin + kw + done * p.wk < s1; ++done) {
            float sc[G ? GROUPS : 1];
            uint32_t ze[(GROUPS + 3) / 4];                 // four groups' zero codes in a word
#pragma unroll
            for (int g = 0; g < (G ? GROUPS : 1); ++g) {
                sc[g] = scale[g];
                if (ZEROS) ze[g / 4] = (g % 4 ? ze[g / 4] : 0u) | zero[g] << (g % 4 * 8);
            }
            fetch(done + 1);
            ok = __all_sync(0xffffffffu, mbar_wait_for(bar0 + 8u * slot, phase, p.wait_ns, p.error));
            if (!ok) break;
            const uint8_t *stage = ring + slot * STAGE;
            const uint4 *xc = xs + (s_begin + kw + done * p.wk - s0) * (2 * U) * unit_step;
#pragma unroll
            for (int half = 0; half < 2; ++half, xc += U * unit_step) {
                uint32_t w[2][2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) R::words(stage, 16 * i + 8 * j + lane / 4, half, t, w[i][j]);
                if (G == 0) {
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const uint4 b = xc[column[j]];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            mma<false>(acc[i][j], w[i][0][0], w[i][1][0], w[i][0][1], w[i][1][1], b.x, b.y);
                            mma<false>(acc[i][j], w[i][0][2], w[i][1][2], w[i][0][3], w[i][1][3], b.z, b.w);
                        }
                    }
                } else {
                    const int chunk = 2 * (s_begin + kw + done * p.wk - s0) + half;
                    const float *unit = units + chunk * (8 * NT) + 2 * t;
                    uint32_t packed[2][2];                 // of the chunk's first group on
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (ZEROS) packed[i][j] = __shfl_sync(0xffffffffu, ze[half * R::GROUPS / 4], 16 * i + 8 * j + lane / 4);
#pragma unroll
                    for (int g = 0; g < R::GROUPS; ++g) {
                        const int byte = (half * R::GROUPS + g) % 4;
                        float s[2][2];
                        uint32_t z[2][2], z16[2][2];       // zero codes as the codes are: pairs of fp16 numbers
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int from = 16 * i + 8 * j + lane / 4;
                                s[i][j] = __shfl_sync(0xffffffffu, sc[half * R::GROUPS + g], from);
                                const uint32_t pick = 0x4040u | (uint32_t)byte << 8 | (uint32_t)byte;
                                z[i][j] = ZEROS ? __byte_perm(packed[i][j], 0x64u, pick) : 0x64086408u;
                                z16[i][j] = ZEROS ? __byte_perm(packed[i][j] << 4, 0x64u, pick) : 0x64806480u;
                            }
                        float sum[2][NT][4];
#pragma unroll
                        for (int k = 0; k < R::IN_GROUP; ++k) {
                            const int word = g * R::IN_GROUP + k;
                            uint32_t a[2][2][4];           // pairs (0, 4), (1, 5), (2, 6), (3, 7) of a word
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const uint32_t first = w[i][j][word], second = first >> 8;
                                    a[i][j][0] = subtract(codes_of(first, 0x000f000fu), z[i][j]);
                                    a[i][j][1] = subtract(codes_of(first, 0x00f000f0u), z16[i][j]);
                                    a[i][j][2] = subtract(codes_of(second, 0x000f000fu), z[i][j]);
                                    a[i][j][3] = subtract(codes_of(second, 0x00f000f0u), z16[i][j]);
                                }
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                const uint4 b = xc[word * unit_step + column[j]];
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    if (k == 0) mma_first(sum[i][j], a[i][0][0], a[i][1][0], a[i][0][1], a[i][1][1], b.x, b.y);
                                    else mma<true>(sum[i][j], a[i][0][0], a[i][1][0], a[i][0][1], a[i][1][1], b.x, b.y);
                                    mma<true>(sum[i][j], a[i][0][2], a[i][1][2], a[i][0][3], a[i][1][3], b.z, b.w);
                                }
                            }
                        }
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const float2 d = *reinterpret_cast<const float2 *>(unit + 8 * j);
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    acc[i][j][k] = __fmaf_rn(__fmul_rn(sum[i][j][k], k % 2 ? d.y : d.x), s[i][k / 2], acc[i][j][k]);
                        }
                    }
                }
            }
            __syncwarp();                                  // the slot is read
            if (issued < mine) {
                issue(issued, slot);
                ++issued;
            }
            if (++slot == p.ring) { slot = 0; phase ^= 1; }
        }
    }
    // a warp that gave up: what it has under way lands before its memory is used again
    for (; done < issued; ++done) {
        mbar_wait_for(bar0 + 8u * slot, phase, kDrainNs, p.error);
        if (++slot == p.ring) { slot = 0; phase ^= 1; }
    }

    // Partial sums, a column's 32 rows next to each other; then the CTA's for each output, and
    // the cluster's.  Outputs next to each other in a row of C by neighbours in a warp.
    __syncthreads();
    float *to = red + warp * (NT * 8 * RED);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                to[(8 * j + 2 * t + k % 2) * RED + 16 * i + lane / 4 + 8 * (k / 2)] = G ? acc[i][j][k] * ACC : acc[i][j][k];
    __syncthreads();
    // (a CTA's rows are a power of two; four of them, next to each other in red and in a row
    // of C, at a time)
    const int log_rows = 31 - __clz(per_cta), log_warp = p.gated ? 4 : 5, all = rows << log_rows;
    const int outs = min(per_cta, p.N - block_row);
    float *own = red + WARPS * NT * 8 * RED;               // [matrix][row of x][row of W]
    auto finish = [&](int o, float4 g, float4 u) {
        const int r = o & (per_cta - 1), m = o >> log_rows;
        float v[4] = {g.x, g.y, g.z, g.w};
        if (p.gated) {
            const float w[4] = {u.x, u.y, u.z, u.w};
            act::with(p.act, [&](auto a) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = act::value<a.value>(v[i]) * w[i];
            });
        }
        const int64_t place = (int64_t)(m0 + m) * p.ldc + block_row + r;
        if (p.c_f32) {
            float *c = static_cast<float *>(p.c) + place;
            if (p.c_vec && r + 4 <= outs) {
                *reinterpret_cast<float4 *>(c) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (r + i < outs) c[i] = v[i];
            }
        } else {
            __nv_bfloat16 *c = static_cast<__nv_bfloat16 *>(p.c) + place;
            const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
            if (p.c_vec && r + 4 <= outs) {
                *reinterpret_cast<uint2 *>(c) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
            } else {
                if (r < outs) c[0] = a.x;
                if (r + 1 < outs) c[1] = a.y;
                if (r + 2 < outs) c[2] = b.x;
                if (r + 3 < outs) c[3] = b.y;
            }
        }
    };
    for (int o = 4 * threadIdx.x; o < all; o += 4 * THREADS) {
        const int r = o & (per_cta - 1), m = o >> log_rows;
        const float *from = red + ((r >> log_warp) * p.wk) * (NT * 8 * RED) + m * parts * RED + (r & (per_warp - 1));
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f), u = v;
        for (int w = 0; w < p.wk; ++w, from += NT * 8 * RED)
            for (int part = parts - 1; part >= 0; --part) {
                add4(v, *reinterpret_cast<const float4 *>(from + part * RED));
                if (p.gated) add4(u, *reinterpret_cast<const float4 *>(from + part * RED + 16));
            }
        if (p.ks == 1) {
            finish(o, v, u);
        } else {
            *reinterpret_cast<float4 *>(own + o) = v;
            if (p.gated) *reinterpret_cast<float4 *>(own + all + o) = u;
        }
    }
    if (p.ks == 1) return;
    cluster_sync_all();
    const uint32_t own0 = smem_u32(own);
    for (int o = 4 * (rank * THREADS + threadIdx.x); o < all; o += 4 * p.ks * THREADS) {
        const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float4 v[8], u = none;                             // (every CTA's under way together)
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = q < p.ks ? load_rank(own0 + 4u * o, (uint32_t)q) : none;
        if (p.gated)
            for (int q = 0; q < p.ks; ++q) add4(u, load_rank(own0 + 4u * (all + o), (uint32_t)q));
#pragma unroll
        for (int q = 1; q < 8; ++q) add4(v[0], v[q]);
        finish(o, v[0], u);
    }
    cluster_sync_all();                                    // no CTA leaves while a peer reads its sums
}

}  // namespace few

struct FewLaunch {
    CUtensorMap map[2];
    few::Params p;
    int nt, grid_x, grid_y, smem;
};

template <int G, bool ZEROS, int NT>
int launch_kernel(const FewLaunch &l, cudaStream_t s) {
    static uint64_t done = 0;
    auto kern = few::few_kernel<G, ZEROS, NT>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SGEMM_ERR_CUDA;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (!bit || !(__atomic_load_n(&done, __ATOMIC_ACQUIRE) & bit)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 225 * 1024) != cudaSuccess)
            return launch_status();
        __atomic_fetch_or(&done, bit, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)l.grid_x, (unsigned)l.grid_y);
    cfg.blockDim = dim3((unsigned)few::THREADS);
    cfg.dynamicSmemBytes = (size_t)l.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (l.p.ks > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)l.p.ks;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    // (every kernel of this path waits for the one before it, whoever's that is, before it
    // touches memory; what comes before the wait overlaps with that one's end)
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = n;
    timing_mark(s, true);
    count_launch();
    cudaLaunchKernelEx(&cfg, kern, l.map[0], l.map[1], l.p);
    timing_mark(s, false);
    return launch_status();
}

// One group's kernels, by the columns' tiles (instantiated in a file of its own).
template <int G>
int launch_few(const FewLaunch &l, cudaStream_t s);

template <int G, bool ZEROS>
int launch_tiles(const FewLaunch &l, cudaStream_t s) {
    switch (l.nt) {
    case 1: return launch_kernel<G, ZEROS, 1>(l, s);
    case 2: return launch_kernel<G, ZEROS, 2>(l, s);
    case 4: return launch_kernel<G, ZEROS, 4>(l, s);
    default: return launch_kernel<G, ZEROS, 8>(l, s);
    }
}

}  // namespace sgemm_gb300
