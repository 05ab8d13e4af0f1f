// A gated feed-forward block in bf16 on the tensor cores, and its backward pass:
//
//   forward   g = x Wg^T, u = x Wu^T, h = act(g) u        one kernel (GATED)
//             y = h Wd^T                                  one kernel (STORE)
//   backward  dh = dy Wd; dg = dh u act'(g), du = dh act(g), h = act(g) u   (SLOPE)
//             dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T h  one kernel (STORE)
//
// g and u are kept for the backward pass as bf16, or as E4M3 codes with a bf16 scale
// for each 128 neighbours of a row.
//
// Every product is the same kernel: tcgen05.mma kind::f16 (bf16 products, exact in fp32,
// added in fp32 in tensor memory over the whole sum), operands brought by TMA as they are
// stored, along the sum or across it (MN-major descriptors), so nothing is transposed or
// copied.  Persistent CTAs walk the tiles of up to four products (grouped raster).  A
// tile's sum may run over two pairs of operands (dx), and its columns may be two
// matrices' (gate and up): with SM pairs (256 x 256 tiles) the leader loads 128 rows of
// gate and its peer the same 128 of up, with single SMs each half of the tile's columns.
// A tensor-memory row then holds g and u of the same columns: act(g) u, and the codes of
// whole groups of 128, need nothing from another thread.
//
// 384 threads: warp 0 TMA, warp 1 MMAs and tensor memory, warps 4-7 and 8-11 the
// epilogue of one of two buffers of tensor memory while the MMAs fill the other; the two
// warpgroups share a tile's columns.  A thread holds one row; 32 columns at a time
// go through shared memory (swizzled) to rows of 16-byte pieces, or element by element
// where alignment or the edge asks for it.
//
// What bounds it (4096 tokens x 2048 x 8192, values kept as codes; alone, us, and the tensor
// pipe's busy cycles): GATED 150, 92 %; the down product 82, 89 %; SLOPE 118, 58 %: its epilogue reads two and writes three
// matrices through the shared memory and L2 that feed the MMAs (95 without its stores, 105
// without its loads, 111 without its arithmetic, 75 without it, in copies made to measure that); the
// gradients 353, 97 %.  Tiles on pairs
// take half the operand traffic of single SMs' for each MMA (4096 x 4096 x 8192 down 164 us,
// with 128 x 128 tiles 225, 128 x 64 350); small calls have too few of them (ffn_plan.h), and where
// one product has few tiles of any size its sum is cut over a cluster (SPLIT: 100 x 1001 x 2731
// 22.5 -> 18.3 us).  Odd sizes: rows that lie 2000 bytes apart straddle the lines that TMA
// reads, which halves its rate (777 x 1000 x 2501 backward: 57 us, 12 for its operations).
//
// Roundings: g, u (kept) and h, dg, du are rounded to bf16 (or codes) once, because the
// products that read them take bf16; sums, activations and derivatives are fp32.
//
// Every wait is bounded, as in the 8-bit product: on expiry the device error word is set,
// the roles stop, copies and MMAs under way are waited for (again bounded) and the CTA
// frees its tensor memory and exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "act.cuh"
#include "few.h"
#include "ffn_plan.h"
#include "fp8.cuh"
#include "plan.h"
#include "ptx_util.cuh"
#include "tc_gemm.h"
#include "tc_ptx.cuh"

namespace sgemm_gb300 {
namespace ffn {

using namespace tc;

constexpr int BK = 64;                         // k per stage: 128 bytes
constexpr int BM = 128;                        // rows of the result per CTA
constexpr int A_BYTES = BM * BK * 2;
constexpr int CHUNK = 64 * BK * 2;             // 64 rows or columns x 64 k
constexpr int CH = 32;                         // columns of the epilogue at a time
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (4 + EPI_WARPS);
constexpr int BLOCK = 32 * CH * 2;             // bytes of 32 rows x 32 bf16 columns
constexpr int STAGING = 2 * BLOCK;             // of an epilogue warp: two bf16 blocks, or one fp32
constexpr int REGS_ISSUE = 56, REGS_EPILOGUE = 224;      // 384 x 168 = 128 x 56 + 256 x 224
constexpr int SMEM_MAX = 232448;
constexpr int BAR_BYTES = 256;
constexpr int MAX_STAGES = 8;
constexpr int PRODUCTS = 4;
constexpr uint64_t kDrainNs = 1000000000ull;

__device__ unsigned int g_error;               // sticky device error word of this path

enum Epilogue { STORE, GATED, SLOPE };

struct Maps {
    CUtensorMap a[2], b[2];
};

struct Product {
    int M, N;                                  // of the result; GATED: N of each matrix
    int tiles_m, tiles_n, first;               // the first unit of this product
    int nk0, nk;                               // blocks of k of the first pair of operands, and of both
    int a_mn, b_mn;                            // operand stored across the sum
    uint32_t idesc;
    void *out;
    int64_t ld;
    int f32, add, width;                       // fp32 result; added to what is there; see put_rows
};

struct Params {
    Maps maps[PRODUCTS];
    Product product[PRODUCTS];
    int count, units;
    int first_units, extra;                    // see unit_of
    int ks;                                    // CTAs of a cluster that share a tile's sum
    int act;
    // kept values, GATED and SLOPE
    void *g, *u;
    __nv_bfloat16 *sg, *su;
    int64_t ld_kept, ld_scales;
    int kept_width;                            // see put_rows
    __nv_bfloat16 *h, *dg, *du;                // all with rows on 16 bytes
    int64_t ldh;
    unsigned long long wait_ns;
};

template <bool PAIR, int BN>
struct Tile {
    static constexpr int B_ROWS = PAIR ? BN / 2 : BN;        // of B that a CTA loads
    static constexpr int STAGE = A_BYTES + B_ROWS * BK * 2;
    static constexpr int FIXED = 1024 + EPI_WARPS * STAGING + BAR_BYTES;
    static constexpr int STAGES = (SMEM_MAX - FIXED) / STAGE < MAX_STAGES ? (SMEM_MAX - FIXED) / STAGE : MAX_STAGES;
    static constexpr int SMEM = FIXED + STAGES * STAGE;
    static constexpr int TMEM = 2 * BN;
    static constexpr int ROWS = PAIR ? 2 * BM : BM;
    static_assert(STAGES >= 3, "stages");
};

__device__ __forceinline__ uint32_t peer_addr(uint32_t local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ void store_cluster(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(addr), "r"(v) : "memory");
}

// Bounded wait by a converged warp: true when every lane's was.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit) {
    return __all_sync(0xffffffffu, mbar_wait_for(bar, parity, limit, &g_error));
}

// kind::f16 (bf16 operands, fp32 result).
template <bool PAIR>
__device__ __forceinline__ void umma_bf16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
    if (PAIR)
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The k-th tile of a lane (a CTA or pair, of `lanes`), or units: none.  The first
// product's tiles (dx: the longest sums) go round the lanes; what is left goes first
// to the lanes that got one fewer of them, `extra` tiles each, then round all of them, from the
// last lane down.  (Plain rounds gave some lanes a long tile and as many short ones
// as the others: 49 us, not 43, for the gradients of 777 x 1000 x 2501.)
__device__ __forceinline__ int unit_of(const Params &p, int k, int lane, int lanes) {
    const int mine = (p.first_units - lane + lanes - 1) / lanes;
    if (k < mine) return lane + k * lanes;
    const int more = p.first_units % lanes;        // lanes below have one more of the first
    int j = k - mine, unit = p.first_units;
    if (lane >= more) {
        if (j < p.extra) return min(unit + j * (lanes - more) + lane - more, p.units);
        j -= p.extra;
    }
    unit += p.extra * (lanes - more) + j * lanes + lanes - 1 - lane;
    return min(unit, p.units);
}

// Product and tile of unit `unit`: GROUP tile rows of the result at a time, so
// that the tiles in flight share operand panels in L2.
__device__ __forceinline__ int tile_of(const Params &p, int unit, int &tm, int &tn) {
    constexpr int GROUP = 16;
    int i = 0;
    while (i + 1 < p.count && unit >= p.product[i + 1].first) ++i;
    const Product &q = p.product[i];
    const int u = unit - q.first, per = GROUP * q.tiles_n;
    const int g = u / per, r = u - g * per;
    const int rows = min(GROUP, q.tiles_m - g * GROUP);
    tn = r / rows;
    tm = g * GROUP + (r - tn * rows);
    return i;
}

// ------------------------------------------------ 32 rows through shared memory
// A block of 32 rows of BYTES (32, 64 or 128) each, in 16-byte pieces; a row's pieces
// are permuted so that neither a lane writing its row nor lanes moving whole rows
// meet in a bank.
template <int BYTES>
__device__ __forceinline__ int piece(int row, int c) {
    return BYTES == 128 ? c ^ (row & 7) : BYTES == 64 ? c ^ ((row >> 1) & 3) : c ^ ((row >> 2) & 1);
}
template <int BYTES>
__device__ __forceinline__ uint4 *piece_at(uint8_t *block, int row, int c) {
    return reinterpret_cast<uint4 *>(block + row * BYTES + 16 * piece<BYTES>(row, c));
}

// Word `k` of a row of a block.
template <int BYTES>
__device__ __forceinline__ uint32_t *word_at(uint8_t *block, int row, int k) {
    return reinterpret_cast<uint32_t *>(piece_at<BYTES>(block, row, k / 4)) + k % 4;
}

// `rows` x `cols` elements of E of the block to `out` (its first element), rows `ld`
// elements apart, in units of `width` bytes: 16 or 4, where every row's elements
// start on them, else one element (and at the matrix's edge).
template <typename E>
__device__ __forceinline__ void put_rows(uint8_t *block, E *out, int64_t ld, int rows, int cols, int width) {
    constexpr int BYTES = CH * sizeof(E), PER = BYTES / 16, STEP = 32 / PER, WORDS = BYTES / 4, ROWS = 32 / WORDS;
    const int lane = threadIdx.x & 31;
    if (width == 16 && cols >= CH) {
        const int c = lane % PER;
        E *at = out + (lane / PER) * ld + c * (16 / (int)sizeof(E));
#pragma unroll
        for (int i = 0; i < 32; i += STEP, at += STEP * ld) {
            const int r = i + lane / PER;
            if (r < rows) *reinterpret_cast<uint4 *>(at) = *piece_at<BYTES>(block, r, c);
        }
    } else if (width >= 4 && cols >= CH) {
        const int k = lane % WORDS;
        E *at = out + (lane / WORDS) * ld + k * (4 / (int)sizeof(E));
#pragma unroll 8
        for (int i = 0; i < 32; i += ROWS, at += ROWS * ld) {
            const int r = i + lane / WORDS;
            if (r < rows) *reinterpret_cast<uint32_t *>(at) = *word_at<BYTES>(block, r, k);
        }
    } else if (lane < cols) {
        E *at = out + lane;
        const int byte = lane * (int)sizeof(E);
#pragma unroll 4
        for (int r = 0; r < min(rows, 32); ++r, at += ld)
            *at = *reinterpret_cast<const E *>(reinterpret_cast<uint8_t *>(piece_at<BYTES>(block, r, byte / 16)) + byte % 16);
    }
}

// The reverse in two steps: fetched into registers (a lane's pieces or words of rows, or its
// column's elements; what lies outside is zero), and put into the block.
template <typename E>
struct Fetched {
    static constexpr int WORDS = CH * (int)sizeof(E) / 4;
    static constexpr int BYTES = CH * (int)sizeof(E), PER = BYTES / 16, STEP = 32 / PER;
    using Bits = typename std::conditional<sizeof(E) == 1, uint8_t,
                                           typename std::conditional<sizeof(E) == 2, uint16_t, uint32_t>::type>::type;
    static constexpr int IN_WORD = 4 / (int)sizeof(E);
    uint32_t w[WORDS];

    __device__ __forceinline__ void fetch(const void *from, int64_t at, int64_t ld, int rows, int cols, int width) {
        const int lane = threadIdx.x & 31;
        if (width == 16 && cols >= CH) {
            const E *in = static_cast<const E *>(from) + at + (lane / PER) * ld + lane % PER * (16 / (int)sizeof(E));
#pragma unroll
            for (int i = 0; i < PER; ++i, in += STEP * ld) {
                const uint4 v = i * STEP + lane / PER < rows ? *reinterpret_cast<const uint4 *>(in) : make_uint4(0, 0, 0, 0);
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        } else if (width >= 4 && cols >= CH) {
            const E *in = static_cast<const E *>(from) + at + (lane / WORDS) * ld + lane % WORDS * IN_WORD;
#pragma unroll
            for (int i = 0; i < WORDS; ++i, in += 32 / WORDS * ld)
                w[i] = i * (32 / WORDS) + lane / WORDS < rows ? *reinterpret_cast<const uint32_t *>(in) : 0u;
        } else {
            const Bits *in = static_cast<const Bits *>(from) + at + lane;
#pragma unroll
            for (int i = 0; i < WORDS; ++i) w[i] = 0;
#pragma unroll
            for (int r = 0; r < 32; ++r, in += ld)
                if (lane < cols && r < rows) w[r / IN_WORD] |= (uint32_t)*in << (r % IN_WORD * 8 * (int)sizeof(E));
        }
    }

    __device__ __forceinline__ void stash(uint8_t *block, int cols, int width) const {
        const int lane = threadIdx.x & 31;
        if (width == 16 && cols >= CH) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                *piece_at<BYTES>(block, i * STEP + lane / PER, lane % PER) =
                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else if (width >= 4 && cols >= CH) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) *word_at<BYTES>(block, i * (32 / WORDS) + lane / WORDS, lane % WORDS) = w[i];
        } else {
            const int byte = lane * (int)sizeof(E);
#pragma unroll
            for (int r = 0; r < 32; ++r)
                *reinterpret_cast<Bits *>(reinterpret_cast<uint8_t *>(piece_at<BYTES>(block, r, byte / 16)) + byte % 16) =
                    (Bits)(w[r / IN_WORD] >> (r % IN_WORD * 8 * (int)sizeof(E)));
        }
    }
};

template <typename E>
__device__ __forceinline__ void get_rows(uint8_t *block, const E *in, int64_t ld, int rows, int cols, int width) {
    Fetched<E> f;
    f.fetch(in, 0, ld, rows, cols, width);
    f.stash(block, cols, width);
}

// A thread's row of 32 bf16 values into its block.
__device__ __forceinline__ void put_bf16(uint8_t *block, const float (&v)[CH]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < CH / 8; ++i)
        *piece_at<2 * CH>(block, lane, i) = make_uint4(pack2(v[8 * i], v[8 * i + 1]), pack2(v[8 * i + 2], v[8 * i + 3]),
                                                       pack2(v[8 * i + 4], v[8 * i + 5]), pack2(v[8 * i + 6], v[8 * i + 7]));
}

// ------------------------------------------------ kept values in 8 bits
// The largest finite |v|.
__device__ __forceinline__ float larger(float m, float v) {
    const float a = fabsf(v);
    return a < __int_as_float(0x7f800000) ? fmaxf(m, a) : m;
}
// A group's scale: rounded to bf16, so that it costs a 64th of the codes; a value may then
// be past 448 scales by 2^-8 of that (449.75), where it still rounds to 448.
__device__ __forceinline__ float kept_scale(float amax) {
    return __bfloat162float(__float2bfloat16_rn(fmaxf(__fdiv_rn(amax, 448.0f), 1.17549435e-38f)));
}
// Codes of a thread's 32 values.  x inv + x 0: one rounding; NaN for an infinity,
// which the format lacks.
__device__ __forceinline__ void put_codes(uint8_t *block, const float (&v)[CH], float inv) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < CH / 16; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float t[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float x = v[16 * i + 4 * j + k];
                t[k] = __fmaf_rn(x, inv, __fmul_rn(x, 0.0f));
            }
            w[j] = fp8::codes4<false>(t);
        }
        *piece_at<CH>(block, lane, i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
__device__ __forceinline__ float2 code_values(uint32_t pair) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// 32 kept values of this thread's row, from rows fetched into `block`.
template <bool CODES>
__device__ __forceinline__ void kept_values(uint8_t *block, float scale, float (&v)[CH]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < CH * (CODES ? 1 : 2) / 16; ++i) {
        const uint4 q = *piece_at<CODES ? CH : 2 * CH>(block, lane, i);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (CODES) {
                const float2 a = code_values(w[j] & 0xffffu), b = code_values(w[j] >> 16);
                v[16 * i + 4 * j] = __fmul_rn(a.x, scale);
                v[16 * i + 4 * j + 1] = __fmul_rn(a.y, scale);
                v[16 * i + 4 * j + 2] = __fmul_rn(b.x, scale);
                v[16 * i + 4 * j + 3] = __fmul_rn(b.y, scale);
            } else {
                v[8 * i + 2 * j] = low(w[j]);
                v[8 * i + 2 * j + 1] = high(w[j]);
            }
        }
    }
}

// ------------------------------------------------ epilogues of one warp
// Its 32 rows start at m0 of the result; the accumulators at tmem (lane quadrant and
// buffer included).  `block`: the warp's STAGING bytes.

// A warpgroup's chunks: CHUNK columns, every other one.
template <int BN>
constexpr int store_chunk() { return BN >= 128 ? 2 * CH : CH; }

template <int BN>
__device__ __forceinline__ void store_tile(const Product &q, uint32_t tmem, uint8_t *block, int m0, int n0, int c0) {
    constexpr int WIDE = store_chunk<BN>();
    const int lane = threadIdx.x & 31, rows = q.M - m0, N = q.N;
    const int64_t ld = q.ld;
    const int width = q.width;
#pragma unroll 1
    for (int c = c0; c < BN && n0 + c < N; c += 2 * WIDE) {
        if (WIDE == 2 * CH && !q.f32 && !q.add) {
            // both halves' reads of tensor memory, and whole lines of bf16, under way together
            uint32_t r[2][CH];
            tmem_ld_async(tmem + c, r[0]);
            tmem_ld_async(tmem + c + CH, r[1]);
            tmem_ld_wait(r[0]);
            tmem_ld_wait(r[1]);
            if (rows <= 0) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[CH];
#pragma unroll
                for (int i = 0; i < CH; ++i) v[i] = __uint_as_float(r[h][i]);
                put_bf16(block + h * BLOCK, v);
            }
            __syncwarp();
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(q.out) + (int64_t)m0 * ld + n0 + c;
            put_rows(block, out, ld, rows, N - n0 - c, width);
            put_rows(block + BLOCK, out + CH, ld, rows, N - n0 - c - CH, width);
            __syncwarp();
            continue;
        }
#pragma unroll 1
        for (int d = c; d < c + WIDE && n0 + d < N; d += CH) {
            uint32_t r[CH];
            tmem_ld32(tmem + d, r);
            if (rows <= 0) continue;
            const int cols = N - n0 - d;
            float v[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) v[i] = __uint_as_float(r[i]);
            if (q.f32) {
                float *out = static_cast<float *>(q.out) + (int64_t)m0 * ld + n0 + d;
                if (q.add) {
                    get_rows(block, out, ld, rows, cols, width);
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < CH / 4; ++i) {
                    uint4 *at = piece_at<4 * CH>(block, lane, i);
                    if (q.add) {
                        const uint4 o = *at;
                        v[4 * i] += __uint_as_float(o.x);
                        v[4 * i + 1] += __uint_as_float(o.y);
                        v[4 * i + 2] += __uint_as_float(o.z);
                        v[4 * i + 3] += __uint_as_float(o.w);
                    }
                    *at = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                                     __float_as_uint(v[4 * i + 3]));
                }
                __syncwarp();
                put_rows(block, out, ld, rows, cols, width);
            } else {
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(q.out) + (int64_t)m0 * ld + n0 + d;
                if (q.add) {
                    get_rows(block, out, ld, rows, cols, width);
                    __syncwarp();
                    float o[CH];
                    kept_values<false>(block, 1.0f, o);
#pragma unroll
                    for (int i = 0; i < CH; ++i) v[i] += o[i];
                }
                put_bf16(block, v);
                __syncwarp();
                put_rows(block, out, ld, rows, cols, width);
            }
            __syncwarp();
        }
    }
}

// KEEP: 0 nothing, 1 bf16, 2 codes (tiles with 128 columns of each matrix).
template <int BN, int KEEP>
__device__ __forceinline__ void gated_tile(const Params &p, const Product &q, uint32_t tmem, uint8_t *block, int m0, int n0,
                                           int c0) {
    constexpr int HALF = BN / 2;
    const int lane = threadIdx.x & 31, rows = q.M - m0;
    float ig = 0.0f, iu = 0.0f;
    if (KEEP == 2) {
        // the group's scales first, by each warpgroup for itself: reading tensor memory twice
        // costs less than holding 256 values, or than an exchange between warps
        float mg = 0.0f, mu = 0.0f;
#pragma unroll 1
        for (int c = 0; c < HALF && n0 + c < q.N; c += CH) {     // (columns past N are zeros)
            uint32_t r[CH];
            tmem_ld32(tmem + c, r);
#pragma unroll
            for (int i = 0; i < CH; ++i) mg = larger(mg, __uint_as_float(r[i]));
            tmem_ld32(tmem + HALF + c, r);
#pragma unroll
            for (int i = 0; i < CH; ++i) mu = larger(mu, __uint_as_float(r[i]));
        }
        const float a = kept_scale(mg), b = kept_scale(mu);
        ig = __fdiv_rn(1.0f, a);
        iu = __fdiv_rn(1.0f, b);
        if (c0 == 0 && lane < rows) {
            const int64_t at = (int64_t)(n0 / 128) * p.ld_scales + m0 + lane;
            p.sg[at] = __float2bfloat16_rn(a);
            p.su[at] = __float2bfloat16_rn(b);
        }
    }
#pragma unroll 1
    for (int c = c0; c < HALF && n0 + c < q.N; c += 2 * CH) {
        uint32_t r[CH];
        float g[CH], u[CH];
        tmem_ld32(tmem + c, r);
#pragma unroll
        for (int i = 0; i < CH; ++i) g[i] = __uint_as_float(r[i]);
        tmem_ld32(tmem + HALF + c, r);
#pragma unroll
        for (int i = 0; i < CH; ++i) u[i] = __uint_as_float(r[i]);
        if (rows <= 0) continue;
        const int cols = q.N - n0 - c;
        const int64_t row = m0, col = n0 + c;
        uint8_t *other = block + BLOCK;
        const int64_t at = row * p.ld_kept + col;
        if (KEEP == 1) {
            put_bf16(block, g);
            put_bf16(other, u);
            __syncwarp();
            put_rows(block, static_cast<__nv_bfloat16 *>(p.g) + at, p.ld_kept, rows, cols, p.kept_width);
            put_rows(other, static_cast<__nv_bfloat16 *>(p.u) + at, p.ld_kept, rows, cols, p.kept_width);
        } else if (KEEP == 2) {
            put_codes(block, g, ig);
            put_codes(other, u, iu);
            __syncwarp();
            put_rows(block, static_cast<uint8_t *>(p.g) + at, p.ld_kept, rows, cols, p.kept_width);
            put_rows(other, static_cast<uint8_t *>(p.u) + at, p.ld_kept, rows, cols, p.kept_width);
        }
        act::with(p.act, [&](auto a) {
#pragma unroll
            for (int i = 0; i < CH; ++i) g[i] = act::value<a.value>(g[i]) * u[i];
        });
        __syncwarp();
        put_bf16(block, g);
        __syncwarp();
        put_rows(block, p.h + row * p.ldh + col, p.ldh, rows, cols, 16);
        __syncwarp();
    }
}

// The kept values of a chunk of columns: fetched a chunk ahead of the one that is
// computed, across tiles.
template <bool CODES>
struct Kept {
    using E = typename std::conditional<CODES, uint8_t, __nv_bfloat16>::type;
    Fetched<E> g, u;
    __nv_bfloat16 sg, su;

    __device__ __forceinline__ void fetch(const Params &p, int row, int rows, int col, int cols) {
        if (rows <= 0 || cols <= 0) return;
        const int64_t at = row * p.ld_kept + col;
        g.fetch(p.g, at, p.ld_kept, rows, cols, p.kept_width);
        u.fetch(p.u, at, p.ld_kept, rows, cols, p.kept_width);
        if (CODES) {
            const int64_t scale = (col / 128) * p.ld_scales + row + min((int)(threadIdx.x & 31), rows - 1);
            sg = p.sg[scale];
            su = p.su[scale];
        }
    }
};

// fetch_next(): the kept values of the first chunk of this warp's next tile.
template <int BN, bool CODES, typename Next>
__device__ __forceinline__ void slope_tile(const Params &p, const Product &q, uint32_t tmem, uint8_t *block, int m0, int n0,
                                           int c0, Kept<CODES> &kept, Next fetch_next) {
    const int rows = q.M - m0;
    uint8_t *bg = block, *bu = block + BLOCK;
#pragma unroll 1
    for (int c = c0; c < BN && n0 + c < q.N; c += 2 * CH) {
        const int cols = q.N - n0 - c;
        const int64_t at = m0 * p.ldh + n0 + c;
        uint32_t r[CH];
        tmem_ld32(tmem + c, r);
        const bool last = c + 2 * CH >= BN || cols <= 2 * CH;
        if (rows <= 0) {
            if (last) fetch_next();
            continue;
        }
        kept.g.stash(bg, cols, p.kept_width);
        kept.u.stash(bu, cols, p.kept_width);
        const float sg = CODES ? __bfloat162float(kept.sg) : 1.0f, su = CODES ? __bfloat162float(kept.su) : 1.0f;
        __syncwarp();
        if (last) fetch_next();
        else kept.fetch(p, m0, rows, n0 + c + 2 * CH, cols - 2 * CH);
        float g[CH], u[CH], h[CH];
        kept_values<CODES>(bg, sg, g);
        kept_values<CODES>(bu, su, u);
        if (CODES) __syncwarp();               // (rows of codes are shorter than the ones that replace them)
        act::with(p.act, [&](auto a) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const float dh = __uint_as_float(r[i]);
                float slope;
                const float v = act::value_slope<a.value>(g[i], slope);
                h[i] = v * u[i];
                g[i] = dh * u[i] * slope;
                u[i] = dh * v;
            }
        });
        put_bf16(bg, g);
        put_bf16(bu, u);
        __syncwarp();
        put_rows(bg, p.dg + at, p.ldh, rows, cols, 16);
        put_rows(bu, p.du + at, p.ldh, rows, cols, 16);
        __syncwarp();
        put_bf16(bg, h);
        __syncwarp();
        put_rows(bg, p.h + at, p.ldh, rows, cols, 16);
        __syncwarp();
    }
}

// SPLIT: this CTA's share of a tile's rows, the cluster's sums added in ascending order.
template <int BN>
__device__ __forceinline__ void add_parts(const Params &p, uint32_t sums, int unit, int part) {
    int tm, tn;
    const Product &q = p.product[tile_of(p, unit, tm, tn)];
    const int first = BM * part / p.ks, rows = BM * (part + 1) / p.ks - first;
    for (int i = (int)threadIdx.x - 128; i < rows * (BN / 4); i += 32 * EPI_WARPS) {
        const int r = first + i / (BN / 4), c = i % (BN / 4) * 4, m = tm * BM + r, n = tn * BN + c;
        if (m >= q.M || n >= q.N) continue;
        float4 v[8];                               // (all under way together)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (k < p.ks)
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(v[k].x), "=f"(v[k].y), "=f"(v[k].z), "=f"(v[k].w)
                             : "r"(peer_addr(sums + 4u * (r * (BN + 4) + c), (uint32_t)k)) : "memory");
        }
#pragma unroll
        for (int k = 1; k < 8; ++k) {
            v[0].x += v[k].x;
            v[0].y += v[k].y;
            v[0].z += v[k].z;
            v[0].w += v[k].w;
        }
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(q.out) + (int64_t)m * q.ld + n;
        if (q.width == 16 && n + 4 <= q.N) {
            *reinterpret_cast<uint2 *>(out) = make_uint2(pack2(v[0].x, v[0].y), pack2(v[0].z, v[0].w));
        } else {
            const float e[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (n + k < q.N) out[k] = __float2bfloat16_rn(e[k]);
        }
    }
}

// ------------------------------------------------ the kernel
// KEEP: GATED and SLOPE, as in the epilogues.  SPLIT (STORE on single SMs): the CTAs of a
// cluster each sum a range of a tile's blocks, and add up a share of its rows through
// distributed shared memory, in ascending order.
template <bool PAIR, int BN, int EPI, int KEEP, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1) ffn_kernel(const __grid_constant__ Params p) {
    using T_ = Tile<PAIR, BN>;
    constexpr int S = T_::STAGES;
    constexpr int B_ROWS = T_::B_ROWS;
    constexpr int WIDTH = EPI == GATED ? BN / 2 : BN;        // columns of a matrix per tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t smem0 = smem_u32(smem);
    uint8_t *staging = smem + S * T_::STAGE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(staging + EPI_WARPS * STAGING);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * S + 4);
    uint32_t *counts = tmem_slot + 1;              // stages filled by either CTA, stages multiplied
    static_assert((2 * S + 4) * 8 + 16 <= BAR_BYTES, "barriers");
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };
    auto tfull = [&](int b) { return bar0 + 8u * (2 * S + b); };
    auto tempty = [&](int b) { return bar0 + 8u * (2 * S + 2 + b); };

    const int warp = warp_index(), lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_rank() : 0u;
    const int part = SPLIT ? (int)cluster_rank() : 0;
    const int self = PAIR ? (int)blockIdx.x >> 1 : SPLIT ? (int)blockIdx.x / p.ks : (int)blockIdx.x;
    const int lanes = PAIR ? (int)gridDim.x >> 1 : (int)gridDim.x;
    auto unit_at = [&](int k) { return SPLIT ? (k == 0 ? self : p.units) : unit_of(p, k, self, lanes); };
    // the blocks of a product's sum that this CTA adds
    auto block_from = [&](const Product &q) { return SPLIT ? (int)((int64_t)q.nk * part / p.ks) : 0; };
    auto block_to = [&](const Product &q) { return SPLIT ? (int)((int64_t)q.nk * (part + 1) / p.ks) : q.nk; };
    const uint64_t lim = p.wait_ns;
    auto publish = [&](int which, int n) {         // to both CTAs
        if (lane == 0) {
            counts[which] = (uint32_t)n;
            if (PAIR) store_cluster(peer_addr(smem_u32(counts + which), rank ^ 1u), (uint32_t)n);
        }
    };
    auto sync_all = [&]() {
        if (PAIR || SPLIT) cluster_sync_all();
        else __syncthreads();
    };

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tempty(b), (PAIR ? 2 : 1) * EPI_WARPS);    // of both CTAs, on the leader's
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int i = 0; i < p.count; ++i) {
            prefetch_map(&p.maps[i].a[0]);
            prefetch_map(&p.maps[i].b[0]);
        }
    }
    if (warp == 1) tmem_alloc<PAIR>(smem_u32(tmem_slot), T_::TMEM);
    tc_fence_before();
    sync_all();                                    // the peer's barriers exist before anything arrives on them
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();                                    // the kernel before may write what is read here
    pdl_trigger();                                 // (the next one waits for this one's end all the same)

    // The epilogues hold 32 rows' values of three matrices and those under way: registers
    // that the first warpgroup does not need.
    bool ok = true;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(REGS_ISSUE));
        if (warp == 0) {
            // ------------------------------------------------ TMA producer
            int s = 0, filled = 0;
            uint32_t ph = 1;
            int unit;
            for (int k = 0; ok && (unit = unit_at(k)) < p.units; ++k) {
                int tm, tn;
                const int i = tile_of(p, unit, tm, tn);
                const Product &q = p.product[i];
                const Maps &maps = p.maps[i];
                const int m = tm * T_::ROWS + (int)rank * BM;
                // GATED: gate and up on the pair's CTAs, or one after the other
                const int n = tn * WIDTH + (PAIR && EPI != GATED ? (int)rank * B_ROWS : 0);
                const int nk0 = q.nk0, to = block_to(q);
                const bool a_mn = q.a_mn != 0, b_mn = q.b_mn != 0;
                for (int kb = block_from(q); kb < to; ++kb) {
                    if (!warp_wait(empty(s), ph, lim)) { ok = false; break; }
                    const bool second = kb >= nk0;
                    const int at = (second ? kb - nk0 : kb) * BK;
                    const uint32_t a = smem0 + (uint32_t)(s * T_::STAGE), b = a + A_BYTES;
                    const uint32_t bar = PAIR ? leader_addr(full(s)) : full(s);
                    const CUtensorMap *ma = &maps.a[second], *mb = &maps.b[EPI == GATED ? (int)rank : (int)second];
                    auto load = [&](uint32_t to, const CUtensorMap *map, int c0, int c1) {
                        if (PAIR) tma_load_2d_pair(to, map, bar, c0, c1);
                        else tma_load_2d(to, map, bar, c0, c1);
                    };
                    if (elect_one()) {
                        if (rank == 0) mbar_expect_tx(full(s), (PAIR ? 2 : 1) * T_::STAGE);
                        if (a_mn) {
                            load(a, ma, m, at);
                            load(a + CHUNK, ma, m + 64, at);
                        } else {
                            load(a, ma, at, m);
                        }
                        if (EPI == GATED) {
                            load(b, mb, at, n);
                            if (!PAIR) load(b + B_ROWS * BK, &maps.b[1], at, n);
                        } else if (b_mn) {
#pragma unroll
                            for (int j = 0; j < B_ROWS; j += 64) load(b + (uint32_t)(j / 64 * CHUNK), mb, n + j, at);
                        } else {
                            load(b, mb, at, n);
                        }
                    }
                    __syncwarp();
                    ++filled;
                    if (++s == S) { s = 0; ph ^= 1; }
                }
            }
            publish((int)rank, filled);
        } else if (warp == 1) {
            // ------------------------------------------------ MMA issuer (the leader's)
            if (rank == 0) {
                int s = 0, b = 0, issued = 0;
                uint32_t ph = 0, bph = 1;
                int unit;
                for (int k = 0; ok && (unit = unit_at(k)) < p.units; ++k) {
                    int tm, tn;
                    const Product &q = p.product[tile_of(p, unit, tm, tn)];
                    const uint32_t a_step = q.a_mn ? 2048u >> 4 : 32u >> 4, b_step = q.b_mn ? 2048u >> 4 : 32u >> 4;
                    const uint32_t idesc = q.idesc, d = tmem + (uint32_t)(b * BN);
                    const int nk = block_to(q) - block_from(q);
                    if (!warp_wait(tempty(b), bph, lim)) { ok = false; break; }
                    for (int kb = 0; kb < nk; ++kb) {
                        if (!warp_wait(full(s), ph, lim)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t a = smem0 + (uint32_t)(s * T_::STAGE);
                        const uint64_t da = smem_desc_8bit(a, CHUNK), db = smem_desc_8bit(a + A_BYTES, CHUNK);
                        if (elect_one()) {
#pragma unroll
                            for (int i = 0; i < BK / 16; ++i)
                                umma_bf16<PAIR>(d, da + i * a_step, db + i * b_step, idesc, kb > 0 || i > 0);
                            if (PAIR) umma_commit_pair(empty(s));
                            else umma_commit(empty(s));
                            if (kb + 1 == nk) {
                                if (PAIR) umma_commit_pair(tfull(b));
                                else umma_commit(tfull(b));
                            }
                        }
                        __syncwarp();
                        ++issued;
                        if (++s == S) { s = 0; ph ^= 1; }
                    }
                    if (++b == 2) { b = 0; bph ^= 1; }
                }
                publish(2, issued);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(REGS_EPILOGUE));
        // ------------------------------------------------ epilogues
        // Chunks of 32 columns alternate between the two warpgroups, and the first
        // changes sides from tile to tile (a narrow GATED tile is a single chunk).
        const int quad = warp & 3, group = (warp - 4) >> 2;
        const uint32_t tmem_rows = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t lead_tempty0 = PAIR ? leader_addr(tempty(0)) : tempty(0);
        uint8_t *block = staging + (warp - 4) * STAGING;
        int b = 0, side = group;
        uint32_t ph = 0;
        Kept<KEEP == 2> kept;
        auto fetch_first = [&](int unit, int s) {
            if (EPI != SLOPE || unit >= p.units) return;
            int tm, tn;
            const Product &q = p.product[tile_of(p, unit, tm, tn)];
            const int m0 = tm * T_::ROWS + (int)rank * BM + quad * 32, c = tn * WIDTH + s * CH;
            kept.fetch(p, m0, q.M - m0, c, q.N - c);
        };
        fetch_first(unit_at(0), side);
        int unit;
        for (int k = 0; (unit = unit_at(k)) < p.units; ++k) {
            int tm, tn;
            const Product &q = p.product[tile_of(p, unit, tm, tn)];
            const int m0 = tm * T_::ROWS + (int)rank * BM + quad * 32, n0 = tn * WIDTH;
            const int c0 = side * (EPI == STORE && !SPLIT ? store_chunk<BN>() : CH);
            const uint32_t at = tmem_rows + (uint32_t)(b * BN);
            if (!warp_wait(tfull(b), ph, lim)) break;
            tc_fence_after();
            if (SPLIT) {
                // (the ring is free: every stage of this CTA is multiplied)
                float *sums = reinterpret_cast<float *>(smem) + (quad * 32 + lane) * (BN + 4);
#pragma unroll 1
                for (int c = c0; c < BN; c += 2 * CH) {
                    uint32_t r[CH];
                    tmem_ld32(at + c, r);
#pragma unroll
                    for (int i = 0; i < CH; i += 4)
                        *reinterpret_cast<uint4 *>(sums + c + i) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
                }
            } else if (EPI == STORE) store_tile<BN>(q, at, block, m0, n0, c0);
            else if (EPI == GATED) gated_tile<BN, KEEP>(p, q, at, block, m0, n0, c0);
            else {
                auto next = [&]() { fetch_first(unit_at(k + 1), side ^ 1); };
                // (a tile without a chunk for this warp: past the last column)
                if (n0 + c0 >= q.N) next();
                else slope_tile<BN, KEEP == 2>(p, q, at, block, m0, n0, c0, kept, next);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                // (nothing but tensor-memory reads, which are complete, is ordered by it: a
                // release would wait for this warp's stores)
                if (PAIR) remote_arrive_relaxed(lead_tempty0 + 8u * b);
                else mbar_arrive(lead_tempty0 + 8u * b);
            }
            side ^= 1;
            if (++b == 2) { b = 0; ph ^= 1; }
        }
    }
    __syncwarp();

    tc_fence_before();
    sync_all();
    // Nothing of this CTA's is under way when it leaves: the commits of the last stages
    // have arrived (and so the MMAs are done), and where a role gave up, stages that were
    // filled and never multiplied have landed.  A stage is complete with both CTAs'
    // copies (counted on the leader's barrier), so the CTA that filled fewer fills the
    // missing ones, which are free, since the other was let into them.
    if (warp == 0) {
        const int f0 = (int)counts[0], f1 = PAIR ? (int)counts[1] : f0, multiplied = (int)counts[2];
        for (int i = max(multiplied - S, 0); i < multiplied; ++i)
            mbar_wait_for(empty(i % S), (uint32_t)(i / S) & 1u, kDrainNs, &g_error);
        __syncwarp();
        const int most = max(f0, f1);
        for (int i = rank == 0 ? f0 : f1; PAIR && i < most; ++i) {
            const uint32_t a = smem0 + (uint32_t)(i % S * T_::STAGE);
            if (elect_one()) {
                if (rank == 0) mbar_expect_tx(full(i % S), 2 * T_::STAGE);
                // (as many bytes as the stage: pieces of the same boxes)
                const Product &q = p.product[0];
                for (int j = 0; j < (q.a_mn ? 2 : 1); ++j)
                    tma_load_2d_pair(a + j * CHUNK, &p.maps[0].a[0], leader_addr(full(i % S)), 0, 0);
                for (int j = 0; j < (EPI != GATED && q.b_mn ? B_ROWS / 64 : 1); ++j)
                    tma_load_2d_pair(a + A_BYTES + j * CHUNK, &p.maps[0].b[0], leader_addr(full(i % S)), 0, 0);
            }
            __syncwarp();
        }
        for (int i = max(most - S, multiplied); rank == 0 && i < most; ++i)
            mbar_wait_for(full(i % S), (uint32_t)(i / S) & 1u, kDrainNs, &g_error);
    }
    __syncwarp();
    if (SPLIT && warp >= 4 && self < p.units) add_parts<BN>(p, smem_u32(smem), self, part);
    sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_free<PAIR>(tmem, T_::TMEM);
    }
}

}  // namespace ffn

// ---------------------------------------------------------------- host side
int ffn_take_device_error() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, ffn::g_error, sizeof(v)) != cudaSuccess) return SGEMM_ERR_CUDA;
    if (v != 0 && cudaMemcpyToSymbol(ffn::g_error, &zero, sizeof(zero)) != cudaSuccess) return SGEMM_ERR_CUDA;
    return v == 0 ? SGEMM_OK : (int)v;
}

namespace {

// A row-major bf16 matrix as a product reads it: across: its rows run along the sum's k.
struct Operand {
    const void *p;
    int64_t rows, cols, ld;
    bool across;
};

// Boxes of 64 columns (128 bytes, swizzled) x box_rows; outside reads as zeros.
bool bf16_map(CUtensorMap *m, const Operand &o, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows};
    cuuint64_t strides[1] = {(cuuint64_t)o.ld * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(o.p), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t k_blocks(int64_t k) { return (k + ffn::BK - 1) / ffn::BK; }

// Collects the products of one launch.
struct Launch {
    ffn::Params p{};
    int variant, epi;
    int64_t units = 0;
    bool ok = true;

    Launch(const FfnCut &cut, int epi_) : variant(cut.variant), epi(epi_) { p.ks = cut.ks; }

    // M x N result of a0 b0 (+ a1 b1), sums k0 (and k1) long; GATED: b0 is gate, b1 up.
    ffn::Product &add(int64_t M, int64_t N, int64_t k0, int64_t k1, const Operand &a0, const Operand &b0, const Operand &a1,
                      const Operand &b1) {
        const FfnTile &t = kFfnTiles[variant];
        const bool gated = epi == ffn::GATED;
        const int width = gated ? t.cols / 2 : t.cols;
        ffn::Maps &maps = p.maps[p.count];
        ffn::Product &q = p.product[p.count++];
        q.M = (int)M;
        q.N = (int)N;
        const int64_t tm = (M + t.rows - 1) / t.rows, tn = (N + width - 1) / width;
        q.tiles_m = (int)tm;
        q.tiles_n = (int)tn;
        q.first = (int)units;
        q.nk0 = (int)k_blocks(k0);
        q.nk = q.nk0 + (int)k_blocks(k1);
        q.a_mn = a0.across;
        q.b_mn = b0.across;
        q.idesc = tc::idesc_8bit(1, 1, q.a_mn, q.b_mn, t.rows, t.cols);      // (both types bf16: 1)
        units += tm * tn;
        const int b_rows = t.ctas == 2 ? t.cols / 2 : t.cols;                // of B per CTA
        const int box_a = a0.across ? 64 : 128;
        const int box_b = b0.across ? 64 : gated && t.ctas == 1 ? b_rows / 2 : b_rows;
        map(maps.a[0], a0, box_a);
        map(maps.b[0], b0, box_b);
        map(maps.a[1], a1, box_a);
        map(maps.b[1], b1, box_b);
        return q;
    }

  private:
    struct Made {
        Operand o;
        int box;
        const CUtensorMap *map;
    };
    Made made[4 * ffn::PRODUCTS];
    int count = 0;

    // (a map takes the host half a microsecond: those of this launch are copied)
    void map(CUtensorMap &to, const Operand &o, int box) {
        for (int i = 0; i < count; ++i)
            if (made[i].o.p == o.p && made[i].o.rows == o.rows && made[i].o.cols == o.cols && made[i].o.ld == o.ld &&
                made[i].box == box) {
                to = *made[i].map;
                return;
            }
        ok = ok && bf16_map(&to, o, box);
        made[count++] = Made{o, box, &to};
    }
};

template <bool PAIR, int BN, int EPI, int KEEP, bool SPLIT = false>
int launch_tiles(const ffn::Params &p, int sms, cudaStream_t s) {
    using T_ = ffn::Tile<PAIR, BN>;
    static uint64_t done = 0;
    auto kern = ffn::ffn_kernel<PAIR, BN, EPI, KEEP, SPLIT>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SGEMM_ERR_CUDA;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (!bit || !(__atomic_load_n(&done, __ATOMIC_ACQUIRE) & bit)) {
        // (a block launched with fewer registers than its warpgroups ask for would wait for ever)
        cudaFuncAttributes attr;
        if (cudaFuncGetAttributes(&attr, kern) != cudaSuccess) return launch_status();
        if (attr.numRegs * ffn::THREADS < 128 * ffn::REGS_ISSUE + 32 * ffn::EPI_WARPS * ffn::REGS_EPILOGUE)
            return SGEMM_ERR_UNSUPPORTED;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T_::SMEM) != cudaSuccess)
            return launch_status();
        __atomic_fetch_or(&done, bit, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(SPLIT ? p.units * p.ks : ffn_lanes(PAIR ? 2 : 1, p.units, sms) * (PAIR ? 2 : 1)));
    cfg.blockDim = dim3((unsigned)ffn::THREADS);
    cfg.dynamicSmemBytes = (size_t)T_::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (PAIR || SPLIT) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = PAIR ? 2 : (unsigned)p.ks;
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
    cudaLaunchKernelEx(&cfg, kern, p);
    timing_mark(s, false);
    return launch_status();
}

template <int EPI, int KEEP>
int launch_variant(int variant, const ffn::Params &p, int sms, cudaStream_t s) {
    if (variant == 0) return launch_tiles<true, 256, EPI, KEEP>(p, sms, s);
    if constexpr (!(EPI == ffn::GATED && KEEP == 2)) {       // (whole groups of 128 need the wide tiles)
        if (variant == 1) return launch_tiles<false, 128, EPI, KEEP>(p, sms, s);
        return launch_tiles<false, 64, EPI, KEEP>(p, sms, s);
    }
    return SGEMM_ERR_UNSUPPORTED;
}

int launch(Launch &l, int keep, int sms, cudaStream_t s) {
    if (!l.ok || l.units > INT32_MAX / 2) return SGEMM_ERR_UNSUPPORTED;
    l.p.units = (int)l.units;
    l.p.first_units = l.p.count == ffn::PRODUCTS ? l.p.product[1].first : l.p.units;
    l.p.extra = 0;
    if (l.p.count == ffn::PRODUCTS) {
        // the tiles of the others that take as long as one of the first
        const int lanes = ffn_lanes(kFfnTiles[l.variant].ctas, l.p.units, sms), less = lanes - l.p.first_units % lanes;
        const double ratio = ffn_tile_time(FFN_STORE, l.variant, l.p.product[0].nk) /
                             ffn_tile_time(FFN_STORE, l.variant, l.p.product[1].nk);
        if (less < lanes) l.p.extra = (int)std::min(ratio + 0.5, (double)((l.p.units - l.p.first_units) / less));
    }
    l.p.wait_ns = tc_wait_limit();
    if (l.epi == ffn::STORE && l.p.ks > 1)
        return l.variant == 1 ? launch_tiles<false, 128, ffn::STORE, 0, true>(l.p, sms, s)
                              : launch_tiles<false, 64, ffn::STORE, 0, true>(l.p, sms, s);
    if (l.epi == ffn::STORE) return launch_variant<ffn::STORE, 0>(l.variant, l.p, sms, s);
    if (l.epi == ffn::SLOPE)
        return keep == 2 ? launch_variant<ffn::SLOPE, 2>(l.variant, l.p, sms, s)
                         : launch_variant<ffn::SLOPE, 1>(l.variant, l.p, sms, s);
    return keep == 0   ? launch_variant<ffn::GATED, 0>(l.variant, l.p, sms, s)
           : keep == 1 ? launch_variant<ffn::GATED, 1>(l.variant, l.p, sms, s)
                       : launch_variant<ffn::GATED, 2>(l.variant, l.p, sms, s);
}

// Rows on 16 bytes, as TMA reads them (a single row may have any leading dimension).
bool tma_rows(const void *p, int64_t ld, int64_t rows) { return aligned16(p) && (ld % 8 == 0 || rows == 1); }
int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }

// The cuts of a block's launches.  apart: dx has a launch of its own, else it is in the
// weights' (whose tiles start while its longer sums run).
struct FfnPlan {
    FfnCut gated, down, slope, dx, weights;
    bool apart;
};
FfnPlan ffn_plan(int64_t T, int64_t D, int64_t F, bool codes, int sms) {
    FfnPlan pl;
    const FfnShape gated{T, 2 * F, k_blocks(D)}, down{T, D, k_blocks(F)}, slope{T, F, k_blocks(D)};
    const FfnShape grads[4] = {{T, D, 2 * k_blocks(F)}, {F, D, k_blocks(T)}, {F, D, k_blocks(T)}, {D, F, k_blocks(T)}};
    pl.gated = ffn_cut(FFN_GATED, &gated, 1, codes, false, sms);
    pl.down = ffn_cut(FFN_STORE, &down, 1, false, true, sms);
    pl.slope = ffn_cut(FFN_SLOPE, &slope, 1, false, false, sms);
    pl.dx = ffn_cut(FFN_STORE, &grads[0], 1, false, true, sms);
    const FfnCut together = ffn_cut(FFN_STORE, grads, 4, false, false, sms),
                 weights = ffn_cut(FFN_STORE, grads + 1, 3, false, false, sms);
    pl.apart = pl.dx.clocks + weights.clocks < together.clocks;
    pl.weights = pl.apart ? weights : together;
    if (!pl.apart) pl.dx = together;
    return pl;
}

// The units, 16 bytes, 4 or an element, on which every row starts.
int row_width(const void *p, int64_t ld, int size) {
    const uint64_t at = reinterpret_cast<uintptr_t>(p) | (uint64_t)ld * size;
    return at % 16 == 0 ? 16 : at % 4 == 0 ? 4 : size;
}

struct Block {
    int64_t T, D, F;
    Operand x, gate, up, down;                   // as stored
    int act, keep;                               // 0 nothing, 1 bf16, 2 codes
    void *g, *u, *sg, *su;
    int64_t ld_kept, ld_scales;
    void *h;
    int64_t ldh;

    void fill(ffn::Params &p) const {
        p.act = act;
        p.g = g;
        p.u = u;
        p.sg = static_cast<__nv_bfloat16 *>(sg);
        p.su = static_cast<__nv_bfloat16 *>(su);
        p.ld_kept = ld_kept;
        p.ld_scales = ld_scales;
        p.kept_width = std::min(row_width(g, ld_kept, keep == 2 ? 1 : 2), row_width(u, ld_kept, keep == 2 ? 1 : 2));
        p.h = static_cast<__nv_bfloat16 *>(h);
        p.ldh = ldh;
    }
};

void set_out(ffn::Product &q, void *out, int64_t ld, int type, int add) {
    q.out = out;
    q.ld = ld;
    q.f32 = type == SGEMM_TYPE_F32;
    q.add = add;
    q.width = row_width(out, ld, q.f32 ? 4 : 2);
}

int zero_rows(void *p, int64_t ld, int64_t rows, int64_t cols, int bytes, cudaStream_t s) {
    if (rows == 0 || cols == 0) return SGEMM_OK;
    return cudaMemset2DAsync(p, (size_t)ld * bytes, 0, (size_t)cols * bytes, (size_t)rows, s) == cudaSuccess ? SGEMM_OK
                                                                                                         : SGEMM_ERR_CUDA;
}

int run_forward(const Block &b, void *y, int64_t ldy, cudaStream_t s) {
    int sms = 0;
    int st = usable_device(&sms);
    if (st != SGEMM_OK) return st;
    if (b.keep == 0 && b.T <= kFfnFewTokens) {
        FewCall c{};
        c.M = b.T; c.N = b.F; c.K = b.D;
        c.x = b.x.p; c.ldx = b.x.ld;
        c.w = b.gate.p; c.w2 = b.up.p; c.ldw = 2 * b.gate.ld;
        c.act = b.act;
        c.c = b.h; c.ldc = b.ldh;
        st = run_few(c, s, false);
        if (st != SGEMM_OK) return st;
        c.N = b.D; c.K = b.F;
        c.x = b.h; c.ldx = b.ldh;
        c.w = b.down.p; c.w2 = nullptr; c.ldw = 2 * b.down.ld;
        c.c = y; c.ldc = ldy;
        return run_few(c, s, true);
    }
    const FfnPlan pl = ffn_plan(b.T, b.D, b.F, b.keep == 2, sms);
    Launch gated(pl.gated, ffn::GATED);
    b.fill(gated.p);
    gated.add(b.T, b.F, b.D, 0, b.x, b.gate, b.x, b.up);
    st = launch(gated, b.keep, sms, s);
    if (st != SGEMM_OK) return st;
    const Operand h{b.h, b.T, b.F, b.ldh, false};
    Launch down(pl.down, ffn::STORE);
    set_out(down.add(b.T, b.D, b.F, 0, h, b.down, h, b.down), y, ldy, SGEMM_TYPE_BF16, 0);
    return launch(down, 0, sms, s);
}

struct Gradients {
    void *dg, *du;                               // scratch, leading dimension Block::ldh
    void *dx;
    int64_t lddx;
    void *gate, *up;
    int64_t ld_in;
    void *down;
    int64_t ld_down;
    int type, add;
};

Operand across(Operand o) {
    o.across = true;
    return o;
}

int run_backward(const Block &b, const Operand &dy, const Gradients &d, cudaStream_t s) {
    int sms = 0;
    int st = usable_device(&sms);
    if (st != SGEMM_OK) return st;
    const FfnPlan pl = ffn_plan(b.T, b.D, b.F, false, sms);
    Launch slope(pl.slope, ffn::SLOPE);
    b.fill(slope.p);
    slope.p.dg = static_cast<__nv_bfloat16 *>(d.dg);
    slope.p.du = static_cast<__nv_bfloat16 *>(d.du);
    slope.add(b.T, b.F, b.D, 0, dy, across(b.down), dy, across(b.down));
    st = launch(slope, b.keep, sms, s);
    if (st != SGEMM_OK) return st;
    const Operand dg{d.dg, b.T, b.F, b.ldh, false}, du{d.du, b.T, b.F, b.ldh, false}, h{b.h, b.T, b.F, b.ldh, true};
    Launch grads(pl.weights, ffn::STORE), apart(pl.dx, ffn::STORE);
    Launch &first = pl.apart ? apart : grads;
    set_out(first.add(b.T, b.D, b.F, b.F, dg, across(b.gate), du, across(b.up)), d.dx, d.lddx, SGEMM_TYPE_BF16, 0);
    if (pl.apart) {
        st = launch(apart, 0, sms, s);
        if (st != SGEMM_OK) return st;
    }
    const Operand x = across(b.x), dgt = across(dg), dut = across(du), dyt = across(dy);
    set_out(grads.add(b.F, b.D, b.T, 0, dgt, x, dgt, x), d.gate, d.ld_in, d.type, d.add);
    set_out(grads.add(b.F, b.D, b.T, 0, dut, x, dut, x), d.up, d.ld_in, d.type, d.add);
    set_out(grads.add(b.D, b.F, b.T, 0, dyt, h, dyt, h), d.down, d.ld_down, d.type, d.add);
    return launch(grads, 0, sms, s);
}

bool aligned(const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

constexpr int64_t kMost = INT32_MAX - 255;       // tiles are rounded up in int

}  // namespace
}  // namespace sgemm_gb300

using namespace sgemm_gb300;

extern "C" int sgemm_ffn(int64_t T, int64_t D, int64_t F, const void *x, int64_t ldx, const void *gate, const void *up,
                         int64_t ld_in, const void *down, int64_t ld_down, int activation, int kept_type, void *g, void *u,
                         int64_t ld_kept, void *sg, void *su, int64_t ld_scales, void *h, int64_t ldh, void *y, int64_t ldy,
                         sgemm_stream_t stream) {
    if (T < 0 || T > kMost) return -1;
    if (D < 0 || D > kMost) return -2;
    if (F < 0 || F > kMost) return -3;
    const bool some = T > 0 && D > 0, all = some && F > 0;
    const bool keep = g != nullptr || u != nullptr, codes = kept_type == SGEMM_TYPE_E4M3;
    auto bad = [&](const void *p) { return p == nullptr || !aligned(p, 2); };
    if (all && bad(x)) return -4;
    if (ldx < std::max<int64_t>(1, D)) return -5;
    if (all && bad(gate)) return -6;
    if (all && bad(up)) return -7;
    if (ld_in < std::max<int64_t>(1, D)) return -8;
    if (all && bad(down)) return -9;
    if (ld_down < std::max<int64_t>(1, F)) return -10;
    if (!act::is_activation(activation)) return -11;
    if (keep && kept_type != SGEMM_TYPE_BF16 && !codes) return -12;
    if (keep && all && (g == nullptr || !aligned(g, codes ? 1 : 2))) return -13;
    if (keep && all && (u == nullptr || !aligned(u, codes ? 1 : 2))) return -14;
    if (keep && ld_kept < std::max<int64_t>(1, F)) return -15;
    if (keep && codes && all && bad(sg)) return -16;
    if (keep && codes && all && bad(su)) return -17;
    if (keep && codes && ld_scales < std::max<int64_t>(1, T)) return -18;
    if (all && bad(h)) return -19;
    if (ldh < std::max<int64_t>(1, F)) return -20;
    if (some && bad(y)) return -21;
    if (ldy < std::max<int64_t>(1, D)) return -22;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0 || D == 0) {
        // (no columns of x: g = u = 0, whose codes and bf16 values are bytes of zero; scales are not)
        if (T > 0 && F > 0 && keep) return SGEMM_ERR_UNSUPPORTED;
        return SGEMM_OK;
    }
    if (F == 0) return zero_rows(y, ldy, T, D, 2, s);
    if (!tma_rows(x, ldx, T) || !tma_rows(gate, ld_in, F) || !tma_rows(up, ld_in, F) || !tma_rows(down, ld_down, D) ||
        !tma_rows(h, ldh, T))
        return SGEMM_ERR_UNSUPPORTED;
    // (one buffer for two results: tiles that run together would write over each other)
    if (keep && u == g) return -14;
    if (keep && codes && su == sg) return -17;
    if (y == h) return -21;
    Block b{T, D, F};
    b.x = Operand{x, T, D, up8(ldx), false};
    b.gate = Operand{gate, F, D, up8(ld_in), false};
    b.up = Operand{up, F, D, up8(ld_in), false};
    b.down = Operand{down, D, F, up8(ld_down), false};
    b.act = activation;
    b.keep = !keep ? 0 : codes ? 2 : 1;
    b.g = g; b.u = u; b.sg = sg; b.su = su;
    b.ld_kept = ld_kept; b.ld_scales = ld_scales;
    b.h = h; b.ldh = up8(ldh);
    return run_forward(b, y, ldy, s);
}

extern "C" int sgemm_ffn_backward(int64_t T, int64_t D, int64_t F, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                  const void *gate, const void *up, int64_t ld_in, const void *down, int64_t ld_down,
                                  int activation, int kept_type, const void *g, const void *u, int64_t ld_kept, const void *sg,
                                  const void *su, int64_t ld_scales, void *dg, void *du, void *h, int64_t ldh, void *dx,
                                  int64_t lddx, int grad_type, int accumulate, void *dgate, void *dup, int64_t ld_din,
                                  void *ddown, int64_t ld_ddown, sgemm_stream_t stream) {
    if (T < 0 || T > kMost) return -1;
    if (D < 0 || D > kMost) return -2;
    if (F < 0 || F > kMost) return -3;
    const bool all = T > 0 && D > 0 && F > 0, codes = kept_type == SGEMM_TYPE_E4M3;
    const int grad = grad_type == SGEMM_TYPE_F32 ? 4 : 2;
    auto bad = [&](const void *p) { return p == nullptr || !aligned(p, 2); };
    if (all && bad(dy)) return -4;
    if (lddy < std::max<int64_t>(1, D)) return -5;
    if (all && bad(x)) return -6;
    if (ldx < std::max<int64_t>(1, D)) return -7;
    if (all && bad(gate)) return -8;
    if (all && bad(up)) return -9;
    if (ld_in < std::max<int64_t>(1, D)) return -10;
    if (all && bad(down)) return -11;
    if (ld_down < std::max<int64_t>(1, F)) return -12;
    if (!act::is_activation(activation)) return -13;
    if (kept_type != SGEMM_TYPE_BF16 && !codes) return -14;
    if (all && (g == nullptr || !aligned(g, codes ? 1 : 2))) return -15;
    if (all && (u == nullptr || !aligned(u, codes ? 1 : 2))) return -16;
    if (ld_kept < std::max<int64_t>(1, F)) return -17;
    if (codes && all && bad(sg)) return -18;
    if (codes && all && bad(su)) return -19;
    if (codes && ld_scales < std::max<int64_t>(1, T)) return -20;
    if (all && bad(dg)) return -21;
    if (all && bad(du)) return -22;
    if (all && bad(h)) return -23;
    if (ldh < std::max<int64_t>(1, F)) return -24;
    if (T > 0 && D > 0 && bad(dx)) return -25;
    if (lddx < std::max<int64_t>(1, D)) return -26;
    if (grad_type != SGEMM_TYPE_F32 && grad_type != SGEMM_TYPE_BF16) return -27;
    auto bad_grad = [&](const void *p) { return D > 0 && F > 0 && (p == nullptr || !aligned(p, grad)); };
    if (bad_grad(dgate)) return -29;
    if (bad_grad(dup)) return -30;
    if (ld_din < std::max<int64_t>(1, D)) return -31;
    if (bad_grad(ddown)) return -32;
    if (ld_ddown < std::max<int64_t>(1, F)) return -33;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!all) {
        // empty sums: gradients of zero, where they are not added to
        int st = zero_rows(dx, lddx, T, D, 2, s);
        if (accumulate || T > 0) return st;
        if (st == SGEMM_OK) st = zero_rows(dgate, ld_din, F, D, grad, s);
        if (st == SGEMM_OK) st = zero_rows(dup, ld_din, F, D, grad, s);
        if (st == SGEMM_OK) st = zero_rows(ddown, ld_ddown, D, F, grad, s);
        return st;
    }
    if (!tma_rows(dy, lddy, T) || !tma_rows(x, ldx, T) || !tma_rows(gate, ld_in, F) || !tma_rows(up, ld_in, F) ||
        !tma_rows(down, ld_down, D) || !tma_rows(dg, ldh, T) || !tma_rows(du, ldh, T) || !tma_rows(h, ldh, T))
        return SGEMM_ERR_UNSUPPORTED;
    // (one buffer for two results, such as two tied weights' gradients, which would both be added to at once)
    if (du == dg) return -22;
    if (h == dg || h == du) return -23;
    if (dup == dgate) return -30;
    if (ddown == dgate || ddown == dup) return -32;
    Block b{T, D, F};
    b.x = Operand{x, T, D, up8(ldx), false};
    b.gate = Operand{gate, F, D, up8(ld_in), false};
    b.up = Operand{up, F, D, up8(ld_in), false};
    b.down = Operand{down, D, F, up8(ld_down), false};
    b.act = activation;
    b.keep = codes ? 2 : 1;
    b.g = const_cast<void *>(g); b.u = const_cast<void *>(u);
    b.sg = const_cast<void *>(sg); b.su = const_cast<void *>(su);
    b.ld_kept = ld_kept; b.ld_scales = ld_scales;
    b.h = h; b.ldh = up8(ldh);
    return run_backward(b, Operand{dy, T, D, up8(lddy), false},
                        Gradients{dg, du, dx, lddx, dgate, dup, ld_din, ddown, ld_ddown, grad_type, accumulate != 0}, s);
}

extern "C" int sgemm_ffn_plan(int64_t T, int64_t D, int64_t F, int kept_type, int num_sms, int *out_rows, int *out_cols,
                              int *out_split) {
    if (T < 1 || T > kMost) return -1;
    if (D < 1 || D > kMost) return -2;
    if (F < 1 || F > kMost) return -3;
    if (num_sms <= 0) return -5;
    const FfnPlan pl = ffn_plan(T, D, F, kept_type == SGEMM_TYPE_E4M3, num_sms);
    const FfnCut *cuts[5] = {&pl.gated, &pl.down, &pl.slope, &pl.dx, &pl.weights};
    for (int i = 0; i < 5; ++i) {
        if (out_rows) out_rows[i] = kFfnTiles[cuts[i]->variant].rows;
        if (out_cols) out_cols[i] = kFfnTiles[cuts[i]->variant].cols;
        if (out_split) out_split[i] = i == 3 && !pl.apart ? 0 : cuts[i]->ks;
    }
    return SGEMM_OK;
}
