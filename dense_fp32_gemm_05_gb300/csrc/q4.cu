// Matrices of 4-bit codes: the quantiser, and the entry point of products with few rows of x
// (the kernel is few_kernel.cuh's).
//
// Quantiser: bound by memory for fp32, by instructions for bf16 (77 % of the issue slots).  A
// thread takes 8 neighbours of a row (a word of codes), so a group of 32, 64 or 128 is 4, 8 or
// 16 lanes, and a warp 256 columns of ROWS rows, whose loads are under way together; the
// group's extremes meet by shuffles, and its scales for the rows are stored together.  Rows
// that do not start on a thread's pieces go through shared memory, so that a warp still
// moves neighbours together.  Each step is one rounded fp32 operation, so the result is
// defined bit for bit.
//   8192 x 4096 fp32, groups of 128, with values: 45.5 us among other calls, 6.3 TB/s (0.93 of the
// measured copy).  1537 x 4095 bf16, groups of 32 with zero codes, values in fp32: 14.4 us
// (2.9 TB/s; 29 where each thread moved its own elements).  16384 x 8192 bf16, groups of 128
// with zero codes: 124 us (173 with a check of each value for infinity and NaN, 4 rows
// a warp and a 64-bit division a tile).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "act.cuh"
#include "few.h"
#include "fp8.cuh"
#include "plan.h"
#include "ptx_util.cuh"
#include "tc_gemm.h"

namespace sgemm_gb300 {
namespace q4 {

constexpr int THREADS = 256;
// Rows of a warp, and CTAs an SM (40 registers a thread; the symmetric kernels spill 44 bytes of
// theirs).  1537 x 4095 with values and 16384 x 8192
// bf16, us: 1 row and 8 CTAs 15.7, 128.7; 2 and 6 14.4, 123.9; 2 and 5 16.5, 129.3; 4 and 4 18.5, 139.3.
constexpr int ROWS = 2;
constexpr int CTAS = 6;
constexpr int COLS = 256;

struct Params {
    const void *X;
    int64_t ldx;
    uint8_t *Q;
    int64_t ldq;
    float *S;
    uint8_t *Z;
    int64_t lds;
    void *V;
    int64_t ldv;
    int rows, cols, tiles_r, tiles_c, step_r, step_c;
    int x_vec, q_vec, v_vec, v_bf16;
};

__device__ __forceinline__ void load8(const float *from, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(from)[0], b = reinterpret_cast<const float4 *>(from)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *from, float (&v)[8]) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(from));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ float load1(const float *from) { return *from; }
__device__ __forceinline__ float load1(const __nv_bfloat16 *from) { return __bfloat162float(*from); }

template <typename T, int G, bool ZEROS>
__global__ void __launch_bounds__(THREADS, CTAS) quantize_kernel(const Params p) {
    constexpr int LANES = G / 8;               // of a group
    constexpr float INF = __builtin_huge_valf();
    __shared__ __align__(16) float rows_of[THREADS / 32][ROWS * COLS];      // a warp's
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *own = rows_of[warp];
    // tiles in rows of tiles_c; the next one of this warp is step_r rows and step_c tiles on
    // (a division for each tile was a quarter of the instructions)
    const uint32_t first = blockIdx.x * (THREADS / 32) + warp;
    int tile_r = (int)(first / (uint32_t)p.tiles_c), tile_c = (int)(first % (uint32_t)p.tiles_c);
    for (; tile_r < p.tiles_r; tile_r += p.step_r, tile_c += p.step_c) {
        if (tile_c >= p.tiles_c) {
            tile_c -= p.tiles_c;
            if (++tile_r >= p.tiles_r) break;
        }
        const int col0 = tile_c * COLS, col = col0 + 8 * lane, row0 = tile_r * ROWS;
        const bool whole = col + 8 <= p.cols;
        float v[ROWS][8];
        if (p.x_vec) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const T *from = static_cast<const T *>(p.X) + row0 * p.ldx + col + r * p.ldx;
                if (row0 + r < p.rows && whole) {
                    load8(from, v[r]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[r][i] = row0 + r < p.rows && col + i < p.cols ? load1(from + i) : 0.0f;
                }
            }
        } else {
            float e[ROWS][8];
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c = col0 + 32 * i + lane;
                    e[r][i] = row0 + r < p.rows && c < p.cols ? load1(static_cast<const T *>(p.X) + row0 * p.ldx + c + r * p.ldx) : 0.0f;
                }
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i) own[r * COLS + 32 * i + lane] = e[r][i];
            __syncwarp();
#pragma unroll
            for (int r = 0; r < ROWS; ++r) load8(own + r * COLS + 8 * lane, v[r]);
            __syncwarp();
        }
        float scale[ROWS], zero[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            // (0 x is NaN for an infinity or NaN: one operation a value finds a warp's rare rows of them)
            float test = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) test = __fmaf_rn(v[r][i], 0.0f, test);
            const bool odd = __any_sync(0xffffffffu, !(test == 0.0f));
            float high = 0.0f, low = 0.0f;     // (symmetric: high is the largest finite |value|)
            if (!odd) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    high = fmaxf(high, ZEROS ? v[r][i] : fabsf(v[r][i]));
                    if (ZEROS) low = fminf(low, v[r][i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = fabsf(v[r][i]) < INF ? v[r][i] : 0.0f;
                    high = fmaxf(high, ZEROS ? x : fabsf(x));
                    if (ZEROS) low = fminf(low, x);
                }
            }
#pragma unroll
            for (int k = 1; k < LANES; k *= 2) {
                high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, k));
                if (ZEROS) low = fminf(low, __shfl_xor_sync(0xffffffffu, low, k));
            }
            const float s = ZEROS ? __fsub_rn(__fdiv_rn(high, 15.0f), __fdiv_rn(low, 15.0f)) : __fdiv_rn(high, 7.0f);
            scale[r] = fmaxf(s, 1.17549435e-38f);
            const float inverse = __frcp_rn(scale[r]);
            zero[r] = ZEROS ? fminf(rintf(__fmul_rn(-low, inverse)), 15.0f) : 8.0f;
            // Numbers are rint(x inverse), by adding and taking off 1.5 2^23.  Finite ones are
            // -zero or more and, symmetric, 7 or less, but for roundings to half a step: with zero
            // codes both ends may round away from 0, to 16 steps.
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float n = __fsub_rn(__fadd_rn(__fmul_rn(v[r][i], inverse), 12582912.0f), 12582912.0f);
                if (odd) n = fmaxf(v[r][i] == v[r][i] ? n : 0.0f, -zero[r]);
                if (odd || ZEROS) n = fminf(n, 15.0f - zero[r]);
                v[r][i] = n;
            }
            // four codes, exactly, in a number's low 16 bits
            uint32_t half[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float *n = v[r] + 4 * i;
                const float sum = __fmaf_rn(n[3], 4096.0f, __fmaf_rn(n[2], 256.0f, __fmaf_rn(n[1], 16.0f, n[0])));
                half[i] = __float_as_uint(__fadd_rn(sum, __fmaf_rn(zero[r], 4369.0f, 12582912.0f)));
            }
            uint32_t word = __byte_perm(half[0], half[1], 0x5410);
            if (p.V) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[r][i] = __fmul_rn(v[r][i], scale[r]);
            }
            if (row0 + r >= p.rows) continue;
            uint8_t *q = p.Q + row0 * p.ldq + col / 2 + r * p.ldq;
            if (whole && p.q_vec) {
                *reinterpret_cast<uint32_t *>(q) = word;
            } else {
                if (col + 8 > p.cols) word &= p.cols > col ? 0xffffffffu >> (4 * (col + 8 - p.cols)) : 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (col + 2 * i < p.cols) q[i] = (uint8_t)(word >> (8 * i));
            }
            if (p.V && p.v_vec) {
                const int64_t at = row0 * p.ldv + col + r * p.ldv;
                if (whole && !p.v_bf16) {
                    float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(p.V) + at);
                    __stcs(to, make_float4(v[r][0], v[r][1], v[r][2], v[r][3]));
                    __stcs(to + 1, make_float4(v[r][4], v[r][5], v[r][6], v[r][7]));
                } else if (whole) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(v[r][2 * i], v[r][2 * i + 1]);
                        w[i] = *reinterpret_cast<const uint32_t *>(&b);
                    }
                    __stcs(reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.V) + at), make_uint4(w[0], w[1], w[2], w[3]));
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (col + i >= p.cols) continue;
                        if (p.v_bf16) static_cast<__nv_bfloat16 *>(p.V)[at + i] = __float2bfloat16_rn(v[r][i]);
                        else static_cast<float *>(p.V)[at + i] = v[r][i];
                    }
                }
            }
        }
        if (p.V && !p.v_vec) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                float4 *to = reinterpret_cast<float4 *>(own + r * COLS + 8 * lane);
                to[0] = make_float4(v[r][0], v[r][1], v[r][2], v[r][3]);
                to[1] = make_float4(v[r][4], v[r][5], v[r][6], v[r][7]);
            }
            __syncwarp();
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c = col0 + 32 * i + lane;
                    if (row0 + r >= p.rows || c >= p.cols) continue;
                    const float x = own[r * COLS + 32 * i + lane];
                    const int64_t at = row0 * p.ldv + c + r * p.ldv;
                    if (p.v_bf16) static_cast<__nv_bfloat16 *>(p.V)[at] = __float2bfloat16_rn(x);
                    else static_cast<float *>(p.V)[at] = x;
                }
            __syncwarp();
        }
        // a group's lanes store its rows' scales, a row each (there are 4 lanes at least)
        if (col / G * G < p.cols) {
            const int r = lane % LANES;
            float s = scale[0], z = zero[0];
#pragma unroll
            for (int i = 1; i < ROWS; ++i)
                if (r == i) {
                    s = scale[i];
                    z = zero[i];
                }
            if (r < ROWS && row0 + r < p.rows) {
                const int64_t at = (int64_t)(col / G) * p.lds + row0 + r;
                p.S[at] = s;
                if (ZEROS) p.Z[at] = (uint8_t)z;
            }
        }
    }
}

template <typename T, int G>
int launch(const Params &p, int grid, cudaStream_t s) {
    if (p.Z) {
        count_launch();
        quantize_kernel<T, G, true><<<grid, THREADS, 0, s>>>(p);
    } else {
        count_launch();
        quantize_kernel<T, G, false><<<grid, THREADS, 0, s>>>(p);
    }
    return launch_status();
}

template <typename T>
int launch(const Params &p, int group, int grid, cudaStream_t s) {
    return group == 128 ? launch<T, 128>(p, grid, s) : group == 64 ? launch<T, 64>(p, grid, s) : launch<T, 32>(p, grid, s);
}

constexpr int64_t kMost = INT32_MAX - 255;
bool is_group(int g) { return g == 32 || g == 64 || g == 128; }
bool aligned(const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace q4
}  // namespace sgemm_gb300

using namespace sgemm_gb300;

extern "C" int sgemm_q4_quantize(int64_t rows, int64_t cols, const void *X, int x_type, int64_t ldx, int group, void *Q,
                                 int64_t ldq, float *S, uint8_t *Z, int64_t lds, void *V, int v_type, int64_t ldv,
                                 sgemm_stream_t stream) {
    if (rows < 0 || rows > q4::kMost) return -1;
    if (cols < 0 || cols > q4::kMost) return -2;
    const bool some = rows > 0 && cols > 0, f32 = x_type == SGEMM_TYPE_F32;
    if (some && (X == nullptr || !q4::aligned(X, f32 ? 4 : 2))) return -3;
    if (!fp8::is_float_type(x_type)) return -4;
    if (ldx < std::max<int64_t>(1, cols)) return -5;
    if (!q4::is_group(group)) return -6;
    if (some && Q == nullptr) return -7;
    if (ldq < std::max<int64_t>(1, (cols + 1) / 2)) return -8;
    if (some && (S == nullptr || !q4::aligned(S, 4))) return -9;
    if (lds < std::max<int64_t>(1, rows)) return -11;
    if (V != nullptr && !fp8::is_float_type(v_type)) return -13;
    if (V != nullptr && !q4::aligned(V, v_type == SGEMM_TYPE_F32 ? 4 : 2)) return -12;
    if (V != nullptr && ldv < std::max<int64_t>(1, cols)) return -14;
    if (!some) return SGEMM_OK;
    int sms = 0;
    const int st = usable_device(&sms);
    if (st != SGEMM_OK) return st;
    q4::Params p{};
    p.X = X; p.ldx = ldx;
    p.Q = static_cast<uint8_t *>(Q); p.ldq = ldq;
    p.S = S; p.Z = Z; p.lds = lds;
    p.V = V; p.ldv = ldv;
    p.rows = (int)rows; p.cols = (int)cols;
    p.tiles_c = (int)((cols + q4::COLS - 1) / q4::COLS);
    p.tiles_r = (int)((rows + q4::ROWS - 1) / q4::ROWS);
    p.x_vec = aligned16(X) && ldx % (f32 ? 4 : 8) == 0;
    p.q_vec = q4::aligned(Q, 4) && ldq % 4 == 0;
    p.v_bf16 = v_type == SGEMM_TYPE_BF16;
    p.v_vec = aligned16(V) && ldv % (p.v_bf16 ? 8 : 4) == 0;
    const int warps = q4::THREADS / 32;
    const int64_t tiles = (int64_t)p.tiles_r * p.tiles_c;
    const int grid = (int)std::min<int64_t>((tiles + warps - 1) / warps, (int64_t)sms * 64);
    p.step_r = grid * warps / p.tiles_c;
    p.step_c = grid * warps % p.tiles_c;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return f32 ? q4::launch<float>(p, group, grid, s) : q4::launch<__nv_bfloat16>(p, group, grid, s);
}

extern "C" int sgemm_q4(int64_t M, int64_t N, int64_t K, const void *X, int x_type, int64_t ldx, const void *Q, const float *S,
                        const uint8_t *Z, const void *Q2, const float *S2, const uint8_t *Z2, int64_t ldq, int64_t lds, int group,
                        int activation, void *C, int c_type, int64_t ldc, sgemm_stream_t stream) {
    if (M < 0 || M > q4::kMost) return -1;
    if (N < 0 || N > q4::kMost) return -2;
    if (K < 0 || K > q4::kMost) return -3;
    const bool out = M > 0 && N > 0, all = out && K > 0, gated = Q2 != nullptr;
    if (all && (X == nullptr || !q4::aligned(X, x_type == SGEMM_TYPE_F32 ? 4 : 2))) return -4;
    if (!fp8::is_float_type(x_type)) return -5;
    if (ldx < std::max<int64_t>(1, K)) return -6;
    if (all && Q == nullptr) return -7;
    if (all && (S == nullptr || !q4::aligned(S, 4))) return -8;
    if (all && gated && (S2 == nullptr || !q4::aligned(S2, 4))) return -11;
    if (all && gated && (Z2 == nullptr) != (Z == nullptr)) return -12;
    if (ldq < std::max<int64_t>(1, (K + 1) / 2)) return -13;
    if (lds < std::max<int64_t>(1, N)) return -14;
    if (!q4::is_group(group)) return -15;
    // (a second matrix without elements may have no address: then there is nothing to activate)
    if (!act::is_activation(activation) || (all && !gated && activation != SGEMM_ACT_NONE)) return -16;
    if (!fp8::is_float_type(c_type)) return -18;
    const bool c_f32 = c_type == SGEMM_TYPE_F32;
    if (out && (C == nullptr || !q4::aligned(C, c_f32 ? 4 : 2))) return -17;
    if (ldc < std::max<int64_t>(1, N)) return -19;
    if (!out) return SGEMM_OK;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (K == 0) {
        const size_t size = c_f32 ? 4 : 2;
        return cudaMemset2DAsync(C, (size_t)ldc * size, 0, (size_t)N * size, (size_t)M, s) == cudaSuccess ? SGEMM_OK
                                                                                                        : SGEMM_ERR_CUDA;
    }
    if (!aligned16(Q) || !aligned16(Q2) || (ldq % 16 != 0 && N > 1)) return SGEMM_ERR_UNSUPPORTED;
    int sms = 0;
    const int st = usable_device(&sms);
    if (st != SGEMM_OK) return st;
    FewCall c{};
    c.M = M; c.N = N; c.K = K;
    c.x = X; c.x_f32 = x_type == SGEMM_TYPE_F32; c.ldx = ldx;
    c.w = Q; c.w2 = Q2; c.ldw = (ldq + 15) / 16 * 16;
    c.group = group;
    c.s = S; c.s2 = S2; c.z = Z; c.z2 = Z2; c.lds = lds;
    c.act = activation;
    c.c = C; c.c_f32 = c_f32; c.ldc = ldc;
    return run_few(c, s, false);
}
