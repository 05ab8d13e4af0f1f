// Few rows of x (decode) against a matrix that is read once from memory: bf16 weights of a
// feed-forward block, or 4-bit weights with group scales.
//
//   c(m,n) = sum over groups b of s(n,b) (sum_{k in b} x(m,k) (code(n,k) - zero(n,b)))
//
// Bound by the weights' stream, so the kernel is built around it.  A warp holds 32
// rows of W (or 16 of each of two matrices) and walks chunks of 64 bytes of each row, several
// chunks' 16-byte loads under way in registers (no staging: nothing else
// reads them).  The products are mma.sync.m16n8k16 (bf16, exact; fp32 sums): W's rows
// are the MMA's 16 rows, x's rows its 8 columns.  Which k an MMA calls its first is
// free as long as both operands agree, so a lane's 16 neighbouring bytes are its share of the
// fragments as they lie; x is laid out once in shared memory in the order in
// which lanes read it.
//   4 bits: the codes of a word come out in four pairs, a code in each half, by a shift and
//   one logic operation that also sets the exponent of 128: 128 + code, exact in bf16;
//   128 + zero is subtracted (exact), so that nothing cancels and infinities in x keep
//   their meaning: 11 instructions for 8 codes.  An MMA never spans two groups; a
//   group's sum is scaled into the fp32 accumulator.
//   x in fp32: three bf16 parts that add up to it exactly, in columns of their own.
// The sum is cut over the warps of a CTA (which take chunks in turn, so that neighbours in
// memory are read together) and over a cluster of CTAs; the partial sums meet
// through (distributed) shared memory in a fixed order: no workspace, no atomics.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "act.cuh"
#include "few.h"
#include "plan.h"
#include "ptx_util.cuh"
#include "tc_gemm.h"

namespace sgemm_gb300 {
namespace few {

constexpr int WARPS = kFewWarps;
constexpr int THREADS = 32 * WARPS;
constexpr int RED = 36;                        // floats of a column of 32 partial sums: no bank twice

struct Params {
    const void *x;
    int64_t ldx;
    const uint8_t *w[2];                       // the warp's two tiles of 16 rows: of one matrix or of two
    int64_t ldw;
    const float *s[2];
    const uint8_t *z[2];
    int64_t lds;
    void *c;
    int64_t ldc;
    int M, N, K;
    int gated, act, c_f32, x_f32, x_vec;
    int per_block;                             // rows of x in a block of columns
    int wk, ks, chunks, depth;
};

__device__ __forceinline__ uint4 stream16(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 stream8(const void *p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t stream4(const void *p) {
    uint32_t v;
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t subtract(uint32_t a, uint32_t b) {
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// G: 0 bf16, else the group.  A lane's words of a row's 64 bytes: word i holds the values from
// k_of(i, t) on, 2 of bf16 or 8 codes, t the lane's place among the four of a row.
template <int G>
struct Row {
    static constexpr int KC = G ? 128 : 32;                // k of a chunk
    static constexpr int WORDS = 4;
    static constexpr int GROUPS = G ? 128 / (G ? G : 1) : 1;   // of a chunk
    static constexpr int IN_GROUP = WORDS / GROUPS;        // words of a lane in a group
    static constexpr int UNITS = G ? 4 : 1;                // 16-byte pieces of x for a lane and column
    // the first k of piece i of x (8 values): a word of codes, or all of a lane's bf16
    __device__ static __forceinline__ int k_of(int i, int t) {
        return G ? i / IN_GROUP * G + t * (G / 4) + 8 * (i % IN_GROUP) : 8 * t;
    }
};

// A lane's weights of one chunk: two tiles, rows lane / 4 and lane / 4 + 8 of each.
template <int G, bool ZEROS>
struct Chunk {
    using R = Row<G>;
    uint32_t w[2][2][4];
    float s[2][2][R::GROUPS];
    uint32_t z[2][2][R::GROUPS];

    // at: byte of the chunk in a row; bytes: of a row
    __device__ __forceinline__ void load(const Params &p, const uint32_t (&row)[2][2], const int (&n)[2][2], int chunk) {
        const int t = threadIdx.x & 3;
        const int at = chunk * 64, bytes = G ? (p.K + 1) / 2 : 2 * p.K;
        const bool whole = at + 64 <= bytes;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t(&v)[4] = w[i][j];
                const uint8_t *from = p.w[i] + (uint64_t)row[i][j] * 16 + at;
                if (whole) {
                    if (G == 0 || G == 128) {
                        const uint4 q = stream16(from + 16 * t);
                        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
                    } else if (G == 64) {
                        const uint2 a = stream8(from + 8 * t), b = stream8(from + 32 + 8 * t);
                        v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = stream4(from + 16 * k + 4 * t);
                    }
                } else {
                    // the row ends in this chunk: what lies behind it is not read, and zero
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int b0 = G == 0 || G == 128 ? 16 * t + 4 * k : G == 64 ? k / 2 * 32 + 8 * t + 4 * (k % 2)
                                                                                     : 16 * k + 4 * t;
                        v[k] = 0;
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (at + b0 + b < bytes) v[k] |= (uint32_t)from[b0 + b] << (8 * b);
                    }
                }
                if (G) {
#pragma unroll
                    for (int g = 0; g < R::GROUPS; ++g) {
                        const int64_t group = (int64_t)chunk * R::GROUPS + g;
                        const bool there = group * G < p.K;
                        s[i][j][g] = there ? __ldg(p.s[i] + group * p.lds + n[i][j]) : 0.0f;
                        if (ZEROS) z[i][j][g] = there ? __ldg(p.z[i] + group * p.lds + n[i][j]) : 0u;
                    }
                }
            }
        }
    }
};

// Parts of an fp32 value: bf16 values of 8 bits that add up to it; one that is not finite is its
// own first part.
__device__ __forceinline__ uint32_t part_of(float v, int part) {
    const uint32_t bits = __float_as_uint(v);
    if ((bits & 0x7f800000u) == 0x7f800000u)
        return part ? 0u : (bits >> 16) | ((bits & 0x7fffffu) ? 0x40u : 0u);
    float r = v;
    for (int i = 0; i < part; ++i) r -= __uint_as_float(__float_as_uint(r) & 0xffff0000u);
    return __float_as_uint(r) >> 16;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float load_rank(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile("{\n\t.reg .u32 a;\n\t"
                 "mapa.shared::cluster.u32 a, %1, %2;\n\t"
                 "ld.shared::cluster.f32 %0, [a];\n\t}" : "=f"(v) : "r"(addr), "r"(rank) : "memory");
    return v;
}

// Chunks of weights under way: what two blocks' registers hold with few columns, one block's with more.
constexpr int ahead(int g, int nt) { return nt > 4 ? 2 : g == 0 ? 4 : g == 128 ? 3 : 2; }

template <int G, bool ZEROS, int NT>
__global__ void __launch_bounds__(THREADS, NT <= 2 ? 2 : 1) few_kernel(const Params p) {
    using R = Row<G>;
    constexpr int KC = R::KC, AHEAD = ahead(G, NT);
    extern __shared__ uint4 xs[];                          // [chunk][piece][tile of 8 columns][lane]
    float *red = reinterpret_cast<float *>(xs);            // [warp][column][RED], after the products
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 3;
    const int rank = p.ks > 1 ? (int)cluster_rank() : 0;
    const int kw = warp % p.wk, rw = warp / p.wk;
    const int per_warp = p.gated ? 16 : 32, per_cta = per_warp * (WARPS / p.wk);
    const int block_row = (int)blockIdx.x / p.ks * per_cta, row0 = block_row + rw * per_warp;
    const int m0 = (int)blockIdx.y * p.per_block;
    const int parts = p.x_f32 ? 3 : 1;
    const int cols = min(p.per_block, p.M - m0) * parts;
    // this CTA's chunks, and this warp's among them: kw, kw + wk, ..
    const int c_begin = (int)((int64_t)p.chunks * rank / p.ks), c_end = (int)((int64_t)p.chunks * (rank + 1) / p.ks);

    int n[2][2];
    uint32_t row[2][2];                                    // in 16 bytes from w
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            n[i][j] = min(row0 + lane / 4 + 8 * j + (p.gated ? 0 : 16 * i), p.N - 1);    // (rows past N: any valid one)
            row[i][j] = (uint32_t)(n[i][j] * (p.ldw / 16));
        }

    float acc[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][j][k] = 0.0f;

    Chunk<G, ZEROS> ring[AHEAD];
    for (int c0 = c_begin; c0 < c_end; c0 += p.depth) {
        const int c1 = min(c0 + p.depth, c_end);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (c0 + kw + u * p.wk < c1) ring[u].load(p, row, n, c0 + kw + u * p.wk);
        if (c0 == c_begin) {
            pdl_wait();                                    // x may be written by the kernel before
            pdl_trigger();
        } else {
            __syncthreads();                               // (x is still read)
        }
        // x into the order of the fragments.  Columns past the last hold what was there: they
        // reach nothing but their own sums, which no one reads.
        const int pieces = (c1 - c0) * R::UNITS * NT * 32;
        for (int i = threadIdx.x; i < pieces; i += THREADS) {
            const int l = i & 31, unit = i >> 5, j = unit % NT, piece = unit / NT;
            const int col = 8 * j + l / 4;
            if (col >= cols) continue;
            const int k = (c0 + piece / R::UNITS) * KC + R::k_of(piece % R::UNITS, l & 3);
            uint32_t v[4];
            if (p.x_f32) {
                const float *from = static_cast<const float *>(p.x) + (int64_t)(m0 + col / 3) * p.ldx + k;
                float f[8];
                if (p.x_vec && k + 8 <= p.K) {
                    const float4 a = *reinterpret_cast<const float4 *>(from), b = *reinterpret_cast<const float4 *>(from + 4);
                    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
                    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = k + e < p.K ? from[e] : 0.0f;
                }
                const int part = col % 3;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = part_of(f[2 * e], part) | (part_of(f[2 * e + 1], part) << 16);
            } else {
                const uint16_t *from = static_cast<const uint16_t *>(p.x) + (int64_t)(m0 + col) * p.ldx + k;
                if (p.x_vec && k + 8 <= p.K) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(from);
                    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = (k + 2 * e < p.K ? (uint32_t)from[2 * e] : 0u) |
                               (k + 2 * e + 1 < p.K ? (uint32_t)from[2 * e + 1] << 16 : 0u);
                }
            }
            // codes leave a word as (0, 4), (1, 5), (2, 6), (3, 7)
            xs[i] = G ? make_uint4(__byte_perm(v[0], v[2], 0x5410), __byte_perm(v[0], v[2], 0x7632),
                                   __byte_perm(v[1], v[3], 0x5410), __byte_perm(v[1], v[3], 0x7632))
                      : make_uint4(v[0], v[1], v[2], v[3]);
        }
        __syncthreads();

        for (int c = c0 + kw; c < c1; c += AHEAD * p.wk) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int at = c + u * p.wk;
                if (at >= c1) break;
                Chunk<G, ZEROS> &q = ring[u];
                const uint4 *xc = xs + (int64_t)(at - c0) * R::UNITS * NT * 32 + lane;
                if (G == 0) {
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const uint4 b = xc[j * 32];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            mma(acc[i][j], q.w[i][0][0], q.w[i][1][0], q.w[i][0][1], q.w[i][1][1], b.x, b.y);
                            mma(acc[i][j], q.w[i][0][2], q.w[i][1][2], q.w[i][0][3], q.w[i][1][3], b.z, b.w);
                        }
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < R::GROUPS; ++g) {
                        float sum[2][NT][4];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int j = 0; j < NT; ++j)
#pragma unroll
                                for (int k = 0; k < 4; ++k) sum[i][j][k] = 0.0f;
#pragma unroll
                        for (int k = 0; k < R::IN_GROUP; ++k) {
                            uint32_t a[2][2][4];           // pairs (0, 4), (1, 5), (2, 6), (3, 7) of a word
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const uint32_t word = q.w[i][j][g * R::IN_GROUP + k];
                                    const uint32_t zero = ZEROS ? 0x43004300u + q.z[i][j][g] * 0x10001u : 0x43084308u;
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        a[i][j][e] = subtract(((word >> (4 * e)) & 0x000f000fu) | 0x43004300u, zero);
                                }
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                const uint4 b = xc[((g * R::IN_GROUP + k) * NT + j) * 32];
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    mma(sum[i][j], a[i][0][0], a[i][1][0], a[i][0][1], a[i][1][1], b.x, b.y);
                                    mma(sum[i][j], a[i][0][2], a[i][1][2], a[i][0][3], a[i][1][3], b.z, b.w);
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int j = 0; j < NT; ++j)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    acc[i][j][k] = __fmaf_rn(sum[i][j][k], q.s[i][k / 2][g], acc[i][j][k]);
                    }
                }
                if (at + AHEAD * p.wk < c1) q.load(p, row, n, at + AHEAD * p.wk);
            }
        }
    }

    // partial sums, a column's 32 rows next to each other
    __syncthreads();
    float *mine = red + warp * (NT * 8 * RED);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) mine[(8 * j + 2 * t + k % 2) * RED + 16 * i + lane / 4 + 8 * (k / 2)] = acc[i][j][k];
    if (p.ks > 1) cluster_sync_all();
    else __syncthreads();
    // each output by one thread, neighbours in a row of C by neighbours in a warp
    const int rows = min(per_cta, p.N - block_row), tokens = cols / parts;
    const uint32_t red0 = smem_u32(red);
    for (int o = rank * THREADS + threadIdx.x; o < per_cta * tokens; o += p.ks * THREADS) {
        const int r = o % per_cta, m = o / per_cta;
        if (r >= rows) continue;
        const int at = (r / per_warp * p.wk) * (NT * 8 * RED) + m * parts * RED + r % per_warp;
        auto total = [&](int place0) {
            float v = 0.0f;
            for (int q = 0; q < p.ks; ++q)
                for (int w = 0; w < p.wk; ++w)
                    for (int part = parts - 1; part >= 0; --part) {
                        const int place = place0 + w * (NT * 8 * RED) + part * RED;
                        v += p.ks > 1 ? load_rank(red0 + 4u * place, (uint32_t)q) : red[place];
                    }
            return v;
        };
        float out = total(at);
        if (p.gated) {
            const float u = total(at + 16);
            act::with(p.act, [&](auto a) { out = act::value<a.value>(out) * u; });
        }
        const int64_t to = (int64_t)(m0 + m) * p.ldc + block_row + r;
        if (p.c_f32) static_cast<float *>(p.c)[to] = out;
        else static_cast<__nv_bfloat16 *>(p.c)[to] = __float2bfloat16_rn(out);
    }
    if (p.ks > 1) cluster_sync_all();                      // no CTA leaves while a peer reads its sums
}

}  // namespace few

template <int G, bool ZEROS, int NT>
int launch_kernel(const few::Params &p, int grid_x, int grid_y, int smem, cudaStream_t s, bool dep) {
    static uint64_t done = 0;
    auto kern = few::few_kernel<G, ZEROS, NT>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SGEMM_ERR_CUDA;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (!bit || !(__atomic_load_n(&done, __ATOMIC_ACQUIRE) & bit)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 163840) != cudaSuccess)
            return launch_status();
        __atomic_fetch_or(&done, bit, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid_x, (unsigned)grid_y);
    cfg.blockDim = dim3((unsigned)few::THREADS);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (p.ks > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)p.ks;
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
    cudaLaunchKernelEx(&cfg, kern, p);
    timing_mark(s, false);
    return launch_status();
}

// One group's kernels, by the columns' tiles (instantiated in a file of its own).
template <int G>
int launch_few(int nt, const few::Params &p, int grid_x, int grid_y, int smem, cudaStream_t s, bool dep);

template <int G, bool ZEROS>
int launch_tiles(int nt, const few::Params &p, int grid_x, int grid_y, int smem, cudaStream_t s, bool dep) {
    switch (nt) {
    case 1: return launch_kernel<G, ZEROS, 1>(p, grid_x, grid_y, smem, s, dep);
    case 2: return launch_kernel<G, ZEROS, 2>(p, grid_x, grid_y, smem, s, dep);
    case 4: return launch_kernel<G, ZEROS, 4>(p, grid_x, grid_y, smem, s, dep);
    case 6: return launch_kernel<G, ZEROS, 6>(p, grid_x, grid_y, smem, s, dep);
    default: return launch_kernel<G, ZEROS, 8>(p, grid_x, grid_y, smem, s, dep);
    }
}

}  // namespace sgemm_gb300
