// Quantisation to 8-bit floating point with a scale for each group of 128.
//
//   amax  = the largest |x| of the group's finite values
//   scale = max(amax / L, 2^-126), L the format's largest value (448, 57344)
//   code  = round(x * (1 / scale)), to nearest even
//
// Each step is one fp32 operation rounded to nearest (the quotient, the
// reciprocal, the product), so the result is defined bit for bit.  The floor
// 2^-126 keeps the reciprocal finite and a group of zeros at code 0.  NaN
// stays NaN; an infinity becomes infinity in E5M2 and NaN in E4M3, which has
// none; neither enters amax, so the group's other values survive.
//
// Memory bound: x is read once into registers (a tile of 32 or, of large matrices,
// 64 x 128 for row groups, 128 x 128 for the others), reduced, converted and stored.
// Measured on GB300: 16384 x 8192 fp32 in 128 x 128 blocks 104.8 us, 6.40 TB/s, 0.94 of
// the measured copy; three CTAs an SM (85 registers) and streaming stores took it
// there from 119 us with two and plain ones: a CTA loads its whole tile before it
// stores, so others have to load meanwhile.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp8.cuh"
#include "plan.h"
#include "ptx_util.cuh"
#include "tc_gemm.h"

namespace sgemm_gb300 {
namespace fp8q {

enum { ROWS = 0, COLS = 1, BLOCKS = 2 };   // group shape: 1 x 128, 128 x 1, 128 x 128
constexpr int tile_rows(int mode, bool tall) { return mode != ROWS ? 128 : tall ? 64 : 32; }
constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr uint32_t INF_BITS = 0x7f800000u;

struct Params {
    const void *X;
    uint8_t *Q;
    float *S;
    int64_t ldx, ldq, lds;
    int rows, cols, tiles_c;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Four elements as loaded (16 bytes of fp32, 8 of bf16), and their values.  They are
// held as loaded: converted at once, the compiler had few of a tile's bf16 loads
// under way (8192 x 8192 in blocks 103 us).
template <typename T> struct Quad;
template <> struct Quad<float> { using Raw = float4; };
template <> struct Quad<__nv_bfloat16> { using Raw = uint2; };
__device__ __forceinline__ void values(float4 t, float (&v)[4]) { v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w; }
__device__ __forceinline__ void values(uint2 t, float (&v)[4]) {
    v[0] = __uint_as_float(t.x << 16);
    v[1] = __uint_as_float(t.x & 0xffff0000u);
    v[2] = __uint_as_float(t.y << 16);
    v[3] = __uint_as_float(t.y & 0xffff0000u);
}
__device__ __forceinline__ float4 pack(float a, float b, float c, float d, const float *) { return make_float4(a, b, c, d); }
__device__ __forceinline__ uint2 pack(float a, float b, float c, float d, const __nv_bfloat16 *) {
    return make_uint2((__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xffff0000u),
                      (__float_as_uint(c) >> 16) | (__float_as_uint(d) & 0xffff0000u));
}

// One value that may be infinite or NaN.
template <bool E5M2>
__device__ __forceinline__ uint32_t code_any(float x, float inv) {
    const uint32_t b = __float_as_uint(x);
    if ((b & 0x7fffffffu) == INF_BITS) return (b >> 24 & 0x80u) | (E5M2 ? 0x7cu : 0x7fu);
    return fp8::codes2<E5M2>(__fmul_rn(x, inv), 0.0f) & 0xffu;
}

// A tile is RT rows (RT / 8 for each warp; TALL: more of them where there are many, so
// that more loads are under way) x 128 columns, four of them for
// each lane: neighbours with VEC (whole-quad loads and stores; every row of X
// and Q starts on a quad), else 32 apart (element loads, still coalesced).
template <typename T, bool E5M2, int MODE, bool VEC, bool TALL>
__global__ void __launch_bounds__(THREADS, !VEC ? 2 : MODE == ROWS ? 4 : 3) quantize_kernel(const Params p) {
    constexpr int RT = tile_rows(MODE, TALL);
    constexpr int R = RT / WARPS;
    constexpr float LARGEST = E5M2 ? 57344.0f : 448.0f;
    __shared__ uint32_t red[WARPS][fp8::GROUP];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tr = (int)(blockIdx.x / (unsigned)p.tiles_c), tcol = (int)(blockIdx.x % (unsigned)p.tiles_c);
    const int r0 = tr * RT + warp * R, c0 = tcol * fp8::GROUP;
    const T *__restrict__ X = static_cast<const T *>(p.X);
    auto col = [&](int j) { return VEC ? c0 + 4 * lane + j : c0 + 32 * j + lane; };
    const bool quad = VEC && c0 + 4 * lane + 3 < p.cols;

    typename Quad<T>::Raw raw[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = r0 + i;
        const T *src = X + (int64_t)r * p.ldx;
        if (r < p.rows && quad) {
            raw[i] = __ldcs(reinterpret_cast<const typename Quad<T>::Raw *>(src + c0 + 4 * lane));
        } else {
            float e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) e[j] = r < p.rows && col(j) < p.cols ? to_f32(src[col(j)]) : 0.0f;
            raw[i] = pack(e[0], e[1], e[2], e[3], X);
        }
    }
    // largest finite |x|, as bits (non-negative fp32 values order as integers)
    uint32_t m[MODE == ROWS ? R : 4];
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < (MODE == ROWS ? R : 4); ++i) m[i] = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float v[4];
        values(raw[i], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t b = __float_as_uint(v[j]) & 0x7fffffffu;
            uint32_t &to = m[MODE == ROWS ? i : j];
            any = max(any, b);
            to = max(to, b < INF_BITS ? b : 0u);
        }
    }
    float inv[MODE == ROWS ? R : (MODE == COLS ? 4 : 1)];
    if (MODE == ROWS) {
        // lane i < R holds row i's maximum: one division for each row
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const uint32_t g = __reduce_max_sync(0xffffffffu, m[i]);
            if (lane == i) mine = g;
        }
        const float s = fmaxf(__fdiv_rn(__uint_as_float(mine), LARGEST), 0x1p-126f);
        const float si = __fdiv_rn(1.0f, s);
        if (lane < R && r0 + lane < p.rows) p.S[(int64_t)tcol * p.lds + r0 + lane] = s;
#pragma unroll
        for (int i = 0; i < R; ++i) inv[i] = __shfl_sync(0xffffffffu, si, i);
    } else if (MODE == COLS) {
#pragma unroll
        for (int j = 0; j < 4; ++j) red[warp][VEC ? 4 * lane + j : 32 * j + lane] = m[j];
        __syncthreads();
        if (threadIdx.x < fp8::GROUP) {
            const int c = threadIdx.x;
            uint32_t g = 0;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) g = max(g, red[w][c]);
            const float s = fmaxf(__fdiv_rn(__uint_as_float(g), LARGEST), 0x1p-126f);
            if (c0 + c < p.cols) p.S[(int64_t)tr * p.lds + c0 + c] = s;
            red[0][c] = __float_as_uint(__fdiv_rn(1.0f, s));   // (only this thread reads column c)
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) inv[j] = __uint_as_float(red[0][VEC ? 4 * lane + j : 32 * j + lane]);
    } else {
        const uint32_t g = __reduce_max_sync(0xffffffffu, max(max(m[0], m[1]), max(m[2], m[3])));
        if (lane == 0) red[0][warp] = g;
        __syncthreads();
        uint32_t all = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) all = max(all, red[0][w]);
        const float s = fmaxf(__fdiv_rn(__uint_as_float(all), LARGEST), 0x1p-126f);
        if (threadIdx.x == 0) p.S[(int64_t)tr * p.lds + tcol] = s;
        inv[0] = __fdiv_rn(1.0f, s);
    }
    const bool odd = any >= INF_BITS;      // an infinity or NaN among this thread's values
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = r0 + i;
        if (r >= p.rows) break;
        uint8_t *dst = p.Q + (int64_t)r * p.ldq;
        uint32_t q;
        float f[4], v[4];
        values(raw[i], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = inv[MODE == ROWS ? i : (MODE == COLS ? j : 0)];
        if (!odd) {
            const float y[4] = {__fmul_rn(v[0], f[0]), __fmul_rn(v[1], f[1]),
                                __fmul_rn(v[2], f[2]), __fmul_rn(v[3], f[3])};
            q = fp8::codes4<E5M2>(y);
        } else {
            q = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) q |= code_any<E5M2>(v[j], f[j]) << (8 * j);
        }
        if (quad) {
            __stcs(reinterpret_cast<uint32_t *>(dst + c0 + 4 * lane), q);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (col(j) < p.cols) dst[col(j)] = (uint8_t)(q >> (8 * j));
        }
    }
}

}  // namespace fp8q

template <typename T, bool E5M2, int MODE, bool VEC, bool TALL>
static int launch_quantize_tiles(const fp8q::Params &p, cudaStream_t s) {
    const int rt = fp8q::tile_rows(MODE, TALL);
    const int64_t grid = (((int64_t)p.rows + rt - 1) / rt) * p.tiles_c;
    if (grid > INT32_MAX) return SGEMM_ERR_UNSUPPORTED;
    count_launch();
    fp8q::quantize_kernel<T, E5M2, MODE, VEC, TALL><<<(unsigned)grid, fp8q::THREADS, 0, s>>>(p);
    return launch_status();
}

template <typename T, bool E5M2, int MODE>
static int launch_quantize(const fp8q::Params &p, bool vec, cudaStream_t s) {
    if (!vec) return launch_quantize_tiles<T, E5M2, MODE, false, false>(p, s);
    // tall tiles once short ones would fill the SMs twice over (8 CTAs each)
    const bool tall = MODE == fp8q::ROWS && (int64_t)(p.rows / 32) * p.tiles_c >= 2400;
    return tall ? launch_quantize_tiles<T, E5M2, MODE, true, MODE == fp8q::ROWS>(p, s)
                : launch_quantize_tiles<T, E5M2, MODE, true, false>(p, s);
}

template <typename T, bool E5M2>
static int launch_quantize(const fp8q::Params &p, int mode, bool vec, cudaStream_t s) {
    return mode == fp8q::ROWS   ? launch_quantize<T, E5M2, fp8q::ROWS>(p, vec, s)
           : mode == fp8q::COLS ? launch_quantize<T, E5M2, fp8q::COLS>(p, vec, s)
                                : launch_quantize<T, E5M2, fp8q::BLOCKS>(p, vec, s);
}

}  // namespace sgemm_gb300

using namespace sgemm_gb300;

extern "C" int sgemm_fp8_quantize(int64_t rows, int64_t cols, const void *X, int x_type,
                                  int64_t ldx, int group_rows, int group_cols, void *Q,
                                  int q_type, int64_t ldq, float *S, int64_t lds,
                                  sgemm_stream_t stream) {
    const int64_t lim = INT32_MAX - fp8::GROUP;      // the kernel's rows and columns are ints
    if (rows < 0 || rows > lim) return -1;
    if (cols < 0 || cols > lim) return -2;
    const bool any = rows > 0 && cols > 0;
    if (any && X == nullptr) return -3;
    if (!fp8::is_float_type(x_type)) return -4;
    if (ldx < std::max<int64_t>(1, cols)) return -5;
    if (group_rows != 1 && group_rows != fp8::GROUP) return -6;
    if ((group_cols != 1 && group_cols != fp8::GROUP) || (group_rows == 1 && group_cols == 1)) return -7;
    if (any && Q == nullptr) return -8;
    if (!fp8::is_code_type(q_type)) return -9;
    if (ldq < std::max<int64_t>(1, cols)) return -10;
    if (any && S == nullptr) return -11;
    const int mode = group_rows == 1 ? fp8q::ROWS : group_cols == 1 ? fp8q::COLS : fp8q::BLOCKS;
    const int64_t s_row = mode == fp8q::ROWS ? rows : mode == fp8q::COLS ? cols : fp8::blocks_of(cols);
    if (lds < std::max<int64_t>(1, s_row)) return -12;
    const int esize = x_type == SGEMM_TYPE_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(X) % esize != 0) return -3;
    if (reinterpret_cast<uintptr_t>(S) % 4 != 0) return -11;
    if (!any) return SGEMM_OK;
    int sms = 0;
    int st = usable_device(&sms);
    if (st != SGEMM_OK) return st;
    const bool vec = reinterpret_cast<uintptr_t>(X) % (4 * esize) == 0 && ldx % 4 == 0 &&
                     reinterpret_cast<uintptr_t>(Q) % 4 == 0 && ldq % 4 == 0;
    fp8q::Params p{X, static_cast<uint8_t *>(Q), S, ldx, ldq, lds, (int)rows, (int)cols,
                   (int)fp8::blocks_of(cols)};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool e5 = q_type == SGEMM_TYPE_E5M2;
    if (x_type == SGEMM_TYPE_F32)
        return e5 ? launch_quantize<float, true>(p, mode, vec, s)
                  : launch_quantize<float, false>(p, mode, vec, s);
    return e5 ? launch_quantize<__nv_bfloat16, true>(p, mode, vec, s)
              : launch_quantize<__nv_bfloat16, false>(p, mode, vec, s);
}
