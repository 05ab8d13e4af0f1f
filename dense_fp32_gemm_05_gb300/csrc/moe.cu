// A mixture-of-experts layer for a few tokens in one kernel: the router, the
// top-k choice, the experts' gate, up and down products over 8-bit weights and
// the weighted sum of the experts' outputs.
//
// A few tokens use every weight a few times at most, so the layer is bound by
// reading the chosen experts' weights once, 3 D F bytes for each.  What the
// kernel is built for is therefore an HBM stream that never stops:
//   * weights go from HBM by TMA into shared memory and from there into the
//     tensor cores (tcgen05 kind::f8f6f4) as they are, 8-bit codes as the
//     MMA's 128 rows; no instruction converts a weight;
//   * activations are the MMA's columns.  They are wider than 8 bits, so each
//     block of 128 of a token is scaled by a power of two (largest value in
//     [128, 256)) and split into PARTS E4M3 numbers,
//       x = 2^-e (q_0 + q_1 / 32 + q_2 / 1024 + ...),
//     q_i the rounding of what the parts before left, times 32^i: each part adds
//     5 bits.  E4M3's smallest step is 2^-9, so what is small beside the block's
//     largest value keeps an absolute error.  bf16 takes 2 parts (exact but for
//     values below 2^-14 of the block's largest, and those to 2^-22 of it), fp32 and
//     h take 4 (to the larger of 2^-19 of the value and 2^-32 of the block's largest).
//     The parts are separate columns of one MMA: it costs the same
//     (few columns), and the products are exact;
//   * a block's sums come back from tensor memory, the parts are added and the
//     block's scales (weights' and token's) applied in fp32 registers;
//   * the work of a product, (expert, 128 rows, block of 128 k) after block, is
//     cut into equal contiguous ranges, one for each CTA.  A range's first and
//     last tile may be shared with the neighbours; partial sums go to a
//     workspace and are added in ascending order of k: no result depends on
//     timing.
//
// Phases, one CTA per SM, cooperative launch:
//   0  x in parts, to memory; router logits: 4 tokens x 2 experts x a slice of D for each warp of the grid
//      (fp32 FMAs); after a grid barrier softmax and top-k, a token each on
//      different CTAs; after another every CTA lists the experts' tokens for itself;
//   1  h = silu(gate x) * (up x): tiles of 64 gate rows and the same 64 up rows.
//      The last CTA to finish a shared tile adds its parts, here and in 2;
//   2  down h.  Only the warps that split h wait, for all tiles of the chunk's h:
//      the weights' stream goes on meanwhile, and a CTA waits for the few that
//      had the same experts, not for the slowest;
//   3  after a last grid barrier y = sum over a token's experts, all threads.
//
// Warps: 0 TMA producer; 1 tensor memory and MMA issue; 2-10 the MMA's column
// operand: x's parts as they are, h split into its; 11 publishes finished tiles; 12-15 promotion (128
// rows, one per thread).
// Every wait is bounded: a role that gives up sets the device error word and
// stops; every CTA still arrives at every grid barrier, so that the counters
// are whole again when the kernel ends.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <new>
#include <type_traits>

#include "fp8.cuh"
#include "plan.h"
#include "ptx_util.cuh"
#include "tc_gemm.h"
#include "tc_ptx.cuh"

namespace sgemm_gb300 {
namespace moe {

using namespace tc;

constexpr int BK = fp8::GROUP;
constexpr int ROWS = 128;                      // weight rows of a tile (64 gate + 64 up, or 128 down)
constexpr int A_BYTES = ROWS * BK;
constexpr int SPLITTERS = 9;                   // warps 2..10
constexpr int FINISHER = 2 + SPLITTERS;        // warp 11
constexpr int PROMOTER0 = FINISHER + 1;        // the first of the 4 promoting warps (a multiple of 4)
constexpr int THREADS = 32 * (PROMOTER0 + 4);
constexpr int MAX_T = 128, MAX_E = 512, MAX_TOPK = 16;
constexpr int MAX_SLOTS = MAX_T * MAX_TOPK;
constexpr int MAX_CHUNKS = 2 * MAX_E;          // (expert, up to NT of its tokens)
constexpr int LOGIT_SLICES = 32;               // slices of D for a group of logits, at most
constexpr int SMEM_MAX = 232448;               // shared memory per block, static and dynamic
constexpr uint64_t kDrainNs = 1000000000ull;

__device__ unsigned int g_error;               // sticky device error word of this path

// NT: tokens of one expert that a tile takes (columns for each part).
template <int NT>
struct Cfg {
    static constexpr int A_STAGES = NT <= 8 ? 10 : 8;   // 16 KB of weights each
    static constexpr int B_BYTES = 4 * NT * BK;
    static constexpr int B_STAGES = NT >= 64 ? 2 : NT >= 32 ? 4 : 8;
    static constexpr uint32_t COLS = 8 * NT;    // two buffers of 4 NT columns
    static constexpr int SMEM = 1024 + A_STAGES * A_BYTES + B_STAGES * B_BYTES;
    static_assert(COLS <= 512, "tensor memory");
    static_assert(B_STAGES * B_BYTES >= (2 * MAX_E + MAX_TOPK) * 4, "a row of logits, a token's choices");
    static_assert(SMEM + 34 * 1024 <= SMEM_MAX, "shared memory (the routing is static)");
};

struct Params {
    int T, D, F, E, topk;
    const void *x;
    int64_t ldx;
    int x_vec;                                 // whole-quad loads of x
    const float *router;
    float *logits;
    const float *s_gate, *s_up, *s_down;
    int renormalize;
    void *y;
    int64_t ldy;
    int32_t *indices;
    float *weights;
    int slices;                                // of D in phase 0
    int ldh, ldo;                              // multiples of 4
    unsigned int *sync;                        // grid barriers 0 .. 2, exits (3)
    // counters: CTAs done with a tile (phase 1's tiles, then phase 2's), then tiles of h done in a chunk
    unsigned int *arrivals;
    int n_arrivals;
    float *logit_parts;                        // [slices][T][E]
    uint32_t *x_parts;                         // [token][block][part][128 bytes]
    float *x_scales;                           // [token][block]
    float *h;                                  // [slot][ldh]
    float *parts;                              // [phase][CTA][first, last tile of its range][token][ROWS]
    float *out;                                // [slot][ldo]: down h
    unsigned long long wait_ns;
};

// Routing as every CTA holds it.  A slot is t * topk + j.
struct Routing {
    short expert[MAX_SLOTS];                   // of a slot
    short rank[MAX_SLOTS];                     // of a slot among its expert's
    short list[MAX_SLOTS];                     // slots by expert, ascending within one
    short token[MAX_SLOTS];                    // their tokens
    int count[MAX_E];                          // an expert's slots
    short first[MAX_E];                        // its first in `list`
    short c_expert[MAX_CHUNKS], c_first[MAX_CHUNKS], c_n[MAX_CHUNKS];
    int chunks;
};

__device__ __forceinline__ unsigned int load_acquire(const unsigned int *p) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Counter updates by one thread after a barrier of the threads whose writes they
// publish: release and acquire are cumulative, so no other thread needs a fence.
__device__ __forceinline__ void add_release(unsigned int *p) {
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" :: "l"(p) : "memory");
}
__device__ __forceinline__ unsigned int add_acq_rel(unsigned int *p) {
    unsigned int v;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ bool grid_wait(const unsigned int *counter, unsigned int n, uint64_t limit) {
    if (load_acquire(counter) >= n) return true;
    const uint64_t t0 = global_timer_ns();
    while (load_acquire(counter) < n) {
        if (global_timer_ns() - t0 > limit) {
            atomicExch(&g_error, (unsigned)SGEMM_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

// Bounded wait by a converged warp: true when every lane's was.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit) {
    return __all_sync(0xffffffffu, mbar_wait_for(bar, parity, limit, &g_error));
}

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ float4 quad(const float *p) { return __ldcg(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ float4 quad(const __nv_bfloat16 *p) {
    const uint2 t = __ldcg(reinterpret_cast<const uint2 *>(p));
    return make_float4(__uint_as_float(t.x << 16), __uint_as_float(t.x & 0xffff0000u),
                       __uint_as_float(t.y << 16), __uint_as_float(t.y & 0xffff0000u));
}

// Elements k .. k+3 of a row of n (zeros past it).  The element path is a call, so
// that the code around it stays short: each launch fetches it anew.
template <typename T>
__device__ __noinline__ float4 load_elements(const T *row, int k, int n) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (k < n) v.x = to_f32(__ldcg(row + k));
    if (k + 1 < n) v.y = to_f32(__ldcg(row + k + 1));
    if (k + 2 < n) v.z = to_f32(__ldcg(row + k + 2));
    if (k + 3 < n) v.w = to_f32(__ldcg(row + k + 3));
    return v;
}
template <typename T>
__device__ __forceinline__ float4 load_quad(const T *row, int k, int n, bool vec) {
    if (vec && k + 3 < n) return quad(row + k);
    return load_elements(row, k, n);
}

// ------------------------------------------------------------ phase 0: logits
// One warp: 4 tokens x 2 experts over a slice of D; each lane has 4 k of each chunk
// of 128, then the lanes are added in a fixed order.  Rows past the last token or
// expert repeat it; their sums are not stored.
constexpr int LOGIT_T = 4, LOGIT_E = 2;
template <typename XT>
__device__ void logits_task(const Params &p, int t0, int e0, int slice) {
    const int lane = threadIdx.x & 31;
    const int chunks = (p.D + BK - 1) / BK;
    const int c0 = chunks * slice / p.slices, c1 = chunks * (slice + 1) / p.slices;
    const XT *x = static_cast<const XT *>(p.x);
    const bool w_vec = p.D % 4 == 0 && (reinterpret_cast<uintptr_t>(p.router) & 15) == 0;
    float v[LOGIT_T * LOGIT_E];
#pragma unroll
    for (int i = 0; i < LOGIT_T * LOGIT_E; ++i) v[i] = 0.0f;
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
        const int k = c * BK + 4 * lane;
        float4 w[LOGIT_E], a[LOGIT_T];
#pragma unroll
        for (int e = 0; e < LOGIT_E; ++e) w[e] = load_quad(p.router + (int64_t)min(e0 + e, p.E - 1) * p.D, k, p.D, w_vec);
#pragma unroll
        for (int t = 0; t < LOGIT_T; ++t) a[t] = load_quad(x + (int64_t)min(t0 + t, p.T - 1) * p.ldx, k, p.D, p.x_vec != 0);
#pragma unroll
        for (int t = 0; t < LOGIT_T; ++t)
#pragma unroll
            for (int e = 0; e < LOGIT_E; ++e) {
                float &s = v[LOGIT_E * t + e];
                s = __fmaf_rn(a[t].w, w[e].w, __fmaf_rn(a[t].z, w[e].z, __fmaf_rn(a[t].y, w[e].y, __fmaf_rn(a[t].x, w[e].x, s))));
            }
    }
    // lane l ends with sum l / 4: three steps keep the half that a bit of the lane names
#pragma unroll
    for (int half = 4; half >= 1; half /= 2) {
        const bool up = (lane & 4 * half) != 0;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
            v[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, send, 4 * half));
        }
    }
    v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xffffffffu, v[0], 2));
    v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
    const int t = t0 + lane / 4 / LOGIT_E, e = e0 + lane / 4 % LOGIT_E;
    if (lane % 4 == 0 && t < p.T && e < p.E) p.logit_parts[((int64_t)slice * p.T + t) * p.E + e] = v[0];
}

// ------------------------------------------------------------ routing
// fp32 values in the order of unsigned integers; NaN lowest, -0 as +0
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 0u;
    const uint32_t b = __float_as_uint(__fadd_rn(v, 0.0f));
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A token's logits from their parts, by the whole CTA: 8 lanes for each expert.
__device__ void token_logits(const Params &p, int t, float *buf) {
    const int n = 8 * p.E, kg = threadIdx.x & 7;
#pragma unroll 1
    for (int i = threadIdx.x; i < (n + 31) / 32 * 32; i += THREADS) {
        const int e = min(i >> 3, p.E - 1);
        const float *src = p.logit_parts + (int64_t)t * p.E + e;
        float part[LOGIT_SLICES / 8];           // (loads under way together)
#pragma unroll
        for (int k = 0; k < LOGIT_SLICES / 8; ++k) {
            const int slice = kg * (LOGIT_SLICES / 8) + k;
            part[k] = slice < p.slices ? __ldcg(src + (int64_t)slice * p.T * p.E) : 0.0f;
        }
        float s = part[0];
#pragma unroll
        for (int k = 1; k < LOGIT_SLICES / 8; ++k) s = __fadd_rn(s, part[k]);
#pragma unroll
        for (int o = 1; o < 8; o *= 2) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
        if (kg == 0 && i < n) {
            buf[e] = s;
            p.logits[(int64_t)t * p.E + e] = s;
        }
    }
}

// One token's softmax and top-k by a warp; `buf`: its logits and room for 2 MAX_E
// floats in all, `chosen`: topk ints.  Loops are not unrolled: every launch runs
// this code once, from a cold instruction cache.
__device__ void route_token(const Params &p, int t, float *buf, int *chosen) {
    constexpr uint32_t TAKEN = 0xffffffffu;     // a NaN that no sum yields marks an expert taken
    const int lane = threadIdx.x & 31;
    float most = -INFINITY;
    bool nan = false;
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) {
        float s = p.router ? buf[e] : p.logits[(int64_t)t * p.E + e];
        if (s != s) {
            nan = true;
            s = __uint_as_float(0x7fffffffu);
        }
        buf[e] = s;
        most = fmaxf(most, s);
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (__any_sync(0xffffffffu, nan)) most = __uint_as_float(0x7fffffffu);   // every weight is NaN then
    float sum = 0.0f;
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) sum = __fadd_rn(sum, expf(__fsub_rn(buf[e], most)));
#pragma unroll
    for (int o = 16; o > 0; o /= 2) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
    float mine = 0.0f;                          // lane j: choice j's weight
    int mine_e = 0;
    __syncwarp();
    if (p.E <= 4 * 32) {
        // each expert's rank: how many come before it.  No round waits for the one
        // before; the work grows as E^2 / 32, so that many experts take rounds.
        uint32_t *keys = reinterpret_cast<uint32_t *>(buf + MAX_E);
        const int padded = (p.E + 3) / 4 * 4;
#pragma unroll 1
        for (int e = lane; e < padded; e += 32) keys[e] = e < p.E ? order_key(buf[e]) : 0u;   // (0 comes last)
        __syncwarp();
#pragma unroll 1
        for (int e = lane; e < p.E; e += 32) {
            const uint32_t key = keys[e];
            int rank = 0;
#pragma unroll 4
            for (int o = 0; o < padded; o += 4) {
                const uint4 k = *reinterpret_cast<const uint4 *>(keys + o);
                rank += (k.x > key || (k.x == key && o < e)) + (k.y > key || (k.y == key && o + 1 < e)) +
                        (k.z > key || (k.z == key && o + 2 < e)) + (k.w > key || (k.w == key && o + 3 < e));
            }
            if (rank < p.topk) chosen[rank] = e;
        }
        __syncwarp();
        if (lane < p.topk) mine_e = chosen[lane];
        mine = buf[mine_e];
    } else {
#pragma unroll 1
        for (int j = 0; j < p.topk; ++j) {
            uint32_t best = 0, at = 0xffffffffu;    // this lane's largest key and its lowest index
#pragma unroll 1
            for (int e = lane; e < p.E; e += 32) {
                const float v = buf[e];
                const uint32_t key = __float_as_uint(v) == TAKEN ? 0u : max(order_key(v), 1u);
                if (key > best) { best = key; at = (uint32_t)e; }
            }
            const uint32_t top = __reduce_max_sync(0xffffffffu, best);
            const int e = (int)__reduce_min_sync(0xffffffffu, best == top ? at : 0xffffffffu);
            if (lane == j) {
                mine = buf[e];
                mine_e = e;
            }
            __syncwarp();
            if ((e & 31) == lane) buf[e] = __uint_as_float(TAKEN);
            __syncwarp();
        }
    }
    mine = __fdiv_rn(expf(__fsub_rn(mine, most)), sum);
    if (p.renormalize) {
        float total = 0.0f;
#pragma unroll 1
        for (int j = 0; j < p.topk; ++j) total = __fadd_rn(total, __shfl_sync(0xffffffffu, mine, j));
        mine = __fdiv_rn(mine, total);
    }
    if (lane < p.topk) {
        p.weights[t * p.topk + lane] = mine;
        p.indices[t * p.topk + lane] = mine_e;
    }
}

// The experts' slot lists and their chunks of up to NT slots, by the whole CTA from
// the experts that the tokens chose.
template <int NT>
__device__ void route_lists(const Params &p, Routing &rt) {
    const int lane = threadIdx.x & 31, slots = p.T * p.topk;
    if (p.T == 1) {                             // its experts differ: a chunk for each
        if ((int)threadIdx.x < slots) {
            const int s = threadIdx.x;
            rt.c_expert[s] = (short)min((unsigned)__ldcg(p.indices + s), (unsigned)(p.E - 1));
            rt.c_first[s] = (short)s;
            rt.c_n[s] = 1;
            rt.list[s] = (short)s;
            rt.token[s] = 0;
        }
        if (threadIdx.x == 0) rt.chunks = slots;
        return;
    }
    for (int s = threadIdx.x; s < slots; s += THREADS) {
        // (an index out of range is left by a router that gave up: its error is reported)
        rt.expert[s] = (short)min((unsigned)__ldcg(p.indices + s), (unsigned)(p.E - 1));
    }
    for (int e = threadIdx.x; e < p.E; e += THREADS) rt.count[e] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        // a slot's place among its expert's, 32 slots at a time
#pragma unroll 1
        for (int s0 = 0; s0 < slots; s0 += 32) {
            const int s = s0 + lane;
            const int e = s < slots ? rt.expert[s] : -1;
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            const int r = (e >= 0 ? rt.count[e] : 0) + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (e >= 0) {
                rt.rank[s] = (short)r;
                if ((same >> lane) == 1u) rt.count[e] = r + 1;   // the last of them
            }
            __syncwarp();
        }
        int slot_base = 0, chunk_base = 0;
#pragma unroll 1
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < p.E ? rt.count[e] : 0;
            const int c = (n + NT - 1) / NT;
            int ns = n, cs = c;                 // inclusive prefix sums
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int a = __shfl_up_sync(0xffffffffu, ns, o), b = __shfl_up_sync(0xffffffffu, cs, o);
                if (lane >= o) { ns += a; cs += b; }
            }
            if (e < p.E) {
                rt.first[e] = (short)(slot_base + ns - n);
#pragma unroll 1
                for (int i = 0; i < c; ++i) {
                    const int at = chunk_base + cs - c + i;
                    rt.c_expert[at] = (short)e;
                    rt.c_first[at] = (short)(slot_base + ns - n + i * NT);
                    rt.c_n[at] = (short)min(NT, n - i * NT);
                }
            }
            slot_base += __shfl_sync(0xffffffffu, ns, 31);
            chunk_base += __shfl_sync(0xffffffffu, cs, 31);
        }
        if (lane == 0) rt.chunks = chunk_base;
    }
    __syncthreads();
    for (int s = threadIdx.x; s < slots; s += THREADS) {
        const int at = rt.first[rt.expert[s]] + rt.rank[s];
        rt.list[at] = (short)s;
        rt.token[at] = (short)(s / p.topk);
    }
}

// ------------------------------------------------------------ work ranges
// A product's blocks: tile after tile (chunk-major), kb blocks each, in equal
// contiguous ranges (the first `more` are one block longer).
struct Work {
    int tiles, kb;                              // tiles per chunk, blocks per tile
    int total;
    // CTAs with a range: none of these is empty, and a small product is not cut into
    // more parts than it takes time to add (T = 1, D = 1024, F = 512: 21.6 -> 19.2 us)
    int n;
    static constexpr int MIN_BLOCKS = 4;
    int each, more;
    __device__ Work(int chunks, int tiles_, int kb_)
        : tiles(tiles_), kb(kb_), total(chunks * tiles_ * kb_), n(max(1, min((int)gridDim.x, total / MIN_BLOCKS))),
          each(total / n), more(total - each * n) {}
    __device__ int begin(int c) const { return c >= n ? total : c * each + min(c, more); }
    __device__ int owner(int it) const {
        const int longer = more * (each + 1);
        return it < longer ? it / (each + 1) : more + (it - longer) / each;
    }
};

// A tile's partial sums: CTAs c0 .. c1 hold them, c0 in the place `part0` of its
// two (a range that begins at or inside the tile: the first), the others in the
// first of theirs.
struct Parts {
    int c0, c1, part0;
    __device__ Parts(const Work &w, int u)
        : c0(w.owner(u * w.kb)), c1(w.owner((u + 1) * w.kb - 1)), part0(w.begin(c0) >= u * w.kb ? 0 : 1) {}
    // values `at` .. + 3 of tokens c .. c + 7 (those below n), in ascending order of k
    __device__ void sum8(const float *parts, int64_t size, int at, int c, int n, float4 (&s)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
        for (int cta = c0; cta <= c1; ++cta) {
            const float *src = parts + (2 * (int64_t)cta + (cta == c0 ? part0 : 0)) * size + c * ROWS + at;
            float4 v[8];                        // (loads under way together)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = c + i < n ? __ldcg(reinterpret_cast<const float4 *>(src + i * ROWS)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s[i] = make_float4(__fadd_rn(s[i].x, v[i].x), __fadd_rn(s[i].y, v[i].y), __fadd_rn(s[i].z, v[i].z),
                                   __fadd_rn(s[i].w, v[i].w));
        }
    }
};

// Calls f(tile, first block, end block) for the pieces of this CTA's range;
// stops when f returns false.
template <typename Fn>
__device__ __forceinline__ bool for_pieces(const Work &w, Fn f) {
    int it = w.begin(blockIdx.x);
    const int end = w.begin(blockIdx.x + 1);
    while (it < end) {
        const int u = it / w.kb;
        const int kb0 = it - u * w.kb;
        const int kb1 = min(w.kb, kb0 + (end - it));
        if (!f(u, kb0, kb1)) return false;
        it += kb1 - kb0;
    }
    return true;
}

__device__ __forceinline__ float gated(float g, float up) {
    return __fmul_rn(__fdiv_rn(g, __fadd_rn(1.0f, expf(-g))), up);
}

// ------------------------------------------------------------ activations
// The larger of two magnitudes; NaN (as bits above every number) if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A lane's 4 values of a token's block -> its bytes of each part, and (lane 0) the
// block's scale.  These instructions, ~60 for a token's block, bound the layer when experts have
// 8 tokens and more, so they are packed pairs where they can be.
// `store` takes part i's 4 bytes.
template <int PARTS, typename Store>
__device__ __forceinline__ void split_block(float4 v, float *scale, int lane, Store store) {
    const float hi = max_nan(max_nan(fabsf(v.x), fabsf(v.y)), max_nan(fabsf(v.z), fabsf(v.w)));
    const uint32_t amax = __reduce_max_sync(0xffffffffu, __float_as_uint(hi));
    const int e = (int)(amax >> 23);
    if (e == 255) {
        // an infinity or NaN makes the token NaN
        const float q = __uint_as_float(0x7fffffffu);
        if ((__float_as_uint(v.x) & 0x7fffffffu) >= 0x7f800000u) v.x = q;
        if ((__float_as_uint(v.y) & 0x7fffffffu) >= 0x7f800000u) v.y = q;
        if ((__float_as_uint(v.z) & 0x7fffffffu) >= 0x7f800000u) v.z = q;
        if ((__float_as_uint(v.w) & 0x7fffffffu) >= 0x7f800000u) v.w = q;
    }
    // 2^(7 - floor(log2 amax)), within the powers whose reciprocal is a normal number
    const int ub = min(max(261 - e, 1), 253);
    const float up = __uint_as_float((uint32_t)ub << 23);
    if (lane == 0) *scale = __uint_as_float((uint32_t)(254 - ub) << 23);
    float2 y01 = __fmul2_rn(make_float2(v.x, v.y), make_float2(up, up));
    float2 y23 = __fmul2_rn(make_float2(v.z, v.w), make_float2(up, up));
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        const uint32_t q01 = fp8::codes2<false>(y01.x, y01.y), q23 = fp8::codes2<false>(y23.x, y23.y);
        store(i, q01 | (q23 << 16));
        if (i + 1 < PARTS) {
            // y = 32 (y - q), exact: 32 q is a half (at most 14336), and the multiply-add
            // has nothing to round
            uint32_t h01, h23;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h01) : "h"((uint16_t)q01));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h23) : "h"((uint16_t)q23));
            const __half2 m32 = __float2half2_rn(-32.0f);
            const float2 d01 = __half22float2(__hmul2(*reinterpret_cast<__half2 *>(&h01), m32));
            const float2 d23 = __half22float2(__hmul2(*reinterpret_cast<__half2 *>(&h23), m32));
            y01 = __ffma2_rn(y01, make_float2(32.0f, 32.0f), d01);
            y23 = __ffma2_rn(y23, make_float2(32.0f, 32.0f), d23);
        }
    }
}

// ------------------------------------------------------------ kernel
template <typename XT, int NT>
__global__ void __launch_bounds__(THREADS, 1)
    moe_kernel(const __grid_constant__ CUtensorMap tm_gate, const __grid_constant__ CUtensorMap tm_up,
               const __grid_constant__ CUtensorMap tm_down, const Params p) {
    using K_ = Cfg<NT>;
    constexpr int P1 = sizeof(XT) == 2 ? 2 : 4;   // parts of x
    // parts of h, for bf16 y too: with three (an error of 2^-14 of a value) 1.3 % of the outputs
    // at T = 4, D = 4096 were not the 64-bit result rounded to bf16, with four 0.07 % (in fp32
    // arithmetic 0.05 %), in the same time but for 2 % at T = 128 (203 -> 206 us)
    constexpr int P2 = 4;
    constexpr int SB = K_::B_STAGES, A_STAGES = K_::A_STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ Routing rt;
    __shared__ alignas(16) float b_scale[SB][NT];
    __shared__ uint64_t bars[2 * A_STAGES + 2 * SB + 6];
    __shared__ uint32_t tmem_slot;
    __shared__ unsigned int s_last;
    const uint32_t smem0 = smem_u32(smem), bar0 = smem_u32(bars);
    auto a_at = [&](int s) { return smem0 + (uint32_t)(s * A_BYTES); };
    auto b_at = [&](int s) { return smem0 + (uint32_t)(A_STAGES * A_BYTES + s * K_::B_BYTES); };
    auto a_full = [&](int s) { return bar0 + 8u * s; };
    auto a_empty = [&](int s) { return bar0 + 8u * (A_STAGES + s); };
    auto b_full = [&](int s) { return bar0 + 8u * (2 * A_STAGES + s); };
    auto b_empty = [&](int s) { return bar0 + 8u * (2 * A_STAGES + SB + s); };
    auto t_full = [&](int b) { return bar0 + 8u * (2 * A_STAGES + 2 * SB + b); };
    auto t_empty = [&](int b) { return bar0 + 8u * (2 * A_STAGES + 2 * SB + 2 + b); };
    const uint32_t tile_left = bar0 + 8u * (2 * A_STAGES + 2 * SB + 4), tile_taken = tile_left + 8u;

    const int warp = warp_index(), lane = threadIdx.x & 31;
    const unsigned int G = gridDim.x;
    const uint64_t lim = p.wait_ns;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < A_STAGES; ++s) {
            mbar_init(a_full(s), 1);
            mbar_init(a_empty(s), 1);
        }
        for (int s = 0; s < SB; ++s) {
            mbar_init(b_full(s), SPLITTERS);
            mbar_init(b_empty(s), 4);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(t_full(b), 1);
            mbar_init(t_empty(b), 4);
        }
        mbar_init(tile_left, 4);
        mbar_init(tile_taken, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&tm_gate);
        prefetch_map(&tm_up);
        prefetch_map(&tm_down);
    }
    if (warp == 1) tmem_alloc<false>(smem_u32(&tmem_slot), K_::COLS);

    // ---- phase 0: logits, and the shared tiles' arrival counters
    for (int i = blockIdx.x * THREADS + threadIdx.x; i < p.n_arrivals; i += G * THREADS) p.arrivals[i] = 0;
    if (p.router) {
        const int tt = (p.T + LOGIT_T - 1) / LOGIT_T, et = (p.E + LOGIT_E - 1) / LOGIT_E;
        for (int i = warp * (int)G + blockIdx.x; i < tt * et * p.slices; i += (THREADS / 32) * G) {
            const int slice = i % p.slices, tile = i / p.slices;
            logits_task<XT>(p, tile / et * LOGIT_T, tile % et * LOGIT_E, slice);
        }
    }
    // x in parts, once for all the tiles that read it
    {
        const int blocks = (p.D + BK - 1) / BK;
        const XT *x = static_cast<const XT *>(p.x);
        for (int i = warp * (int)G + blockIdx.x; i < p.T * blocks; i += (THREADS / 32) * G) {
            const int t = i / blocks, kb = i - t * blocks;
            const float4 v = load_quad(x + (int64_t)t * p.ldx, kb * BK + 4 * lane, p.D, p.x_vec != 0);
            uint32_t *to = p.x_parts + (int64_t)i * (P1 * BK / 4) + lane;
            split_block<P1>(v, p.x_scales + i, lane, [&](int part, uint32_t q) { to[part * (BK / 4)] = q; });
        }
    }
    bool ok = true;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    if (threadIdx.x == 0) {
        add_release(&p.sync[0]);
        s_last = grid_wait(&p.sync[0], G, lim);
    }
    __syncthreads();
    ok = s_last != 0;
    // each token is routed by one CTA, the result read by all after another barrier
    // (every CTA routing every token: 36 us of T = 64's 115); one token alone by every
    // CTA for itself (all write the same), which is shorter than the barrier
    const bool alone = p.T == 1;
    for (int t = alone ? 0 : (int)blockIdx.x; ok && t < p.T; t += G) {
        float *buf = reinterpret_cast<float *>(smem + A_STAGES * A_BYTES);   // (where activations go later)
        if (p.router) token_logits(p, t, buf);
        __syncthreads();
        if (warp == 0) route_token(p, t, buf, reinterpret_cast<int *>(buf + 2 * MAX_E));
        __syncthreads();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        if (!alone) add_release(&p.sync[1]);
        s_last = ok && (alone || grid_wait(&p.sync[1], G, lim));
    }
    __syncthreads();
    ok = s_last != 0;
    if (ok) route_lists<NT>(p, rt);
    else if (threadIdx.x == 0) rt.chunks = 0;
    __syncthreads();
    const int kb1 = (p.D + BK - 1) / BK, kb2 = (p.F + BK - 1) / BK;
    const Work w1(rt.chunks, (p.F + 63) / 64, kb1), w2(rt.chunks, (p.D + ROWS - 1) / ROWS, kb2);
    ok = ok && rt.chunks > 0;
    // (a CTA may be in phase 2 while another still adds phase 1's parts)
    const int64_t phase_parts = (int64_t)G * 2 * NT * ROWS;
    unsigned int *done = p.arrivals + rt.chunks * (w1.tiles + w2.tiles);   // tiles of h done, by chunk

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (ok) {
            int s = 0, filled = 0;
            uint32_t ph = 1;
            auto produce = [&](const Work &w, bool second) {
                return for_pieces(w, [&](int u, int k0, int k1) {
                    const int e = rt.c_expert[u / w.tiles], tile = u % w.tiles;
                    for (int kb = k0; kb < k1; ++kb) {
                        if (!warp_wait(a_empty(s), ph, lim)) return false;
                        if (elect_one()) {
                            mbar_expect_tx(a_full(s), A_BYTES);
                            if (second) {
                                tma_load_3d(a_at(s), &tm_down, a_full(s), kb * BK, tile * ROWS, e);
                            } else {
                                // 16 rows of gate and the same 16 of up for each promoting warp
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    tma_load_3d(a_at(s) + i * 32 * BK, &tm_gate, a_full(s), kb * BK, tile * 64 + 16 * i, e);
                                    tma_load_3d(a_at(s) + (i * 32 + 16) * BK, &tm_up, a_full(s), kb * BK, tile * 64 + 16 * i, e);
                                }
                            }
                        }
                        ++filled;
                        if (++s == A_STAGES) { s = 0; ph ^= 1; }
                    }
                    return true;
                });
            };
            if (produce(w1, false)) produce(w2, true);
            for (int i = 0; i < min(filled, A_STAGES); ++i) {   // copies in flight land before shared memory goes
                if (s == 0) { s = A_STAGES; ph ^= 1; }
                --s;
                mbar_wait_for(a_full(s), ph ^ 1u, kDrainNs, &g_error);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        if (ok) {
            int s = 0, bs = 0, b = 0, issued = 0;
            uint32_t ph = 0, bph = 0, tph = 1;
            const uint64_t da0 = smem_desc_8bit(a_at(0), A_BYTES), db0 = smem_desc_8bit(b_at(0), A_BYTES);
            auto multiply = [&](const Work &w, int parts) {
                return for_pieces(w, [&](int u, int k0, int k1) {
                    const int n8 = (rt.c_n[u / w.tiles] + 7) / 8 * 8;
                    const uint32_t idesc = idesc_8bit(0, 0, 0, 0, ROWS, (parts * n8 + 15) / 16 * 16);
                    for (int kb = k0; kb < k1; ++kb) {
                        // (the three tests overlap; what this role spends on a block is the
                        // least time a block can take: 730 clocks with waits and commits in turn)
                        const bool t0 = mbar_test(t_empty(b), tph), t1 = mbar_test(a_full(s), ph), t2 = mbar_test(b_full(bs), bph);
                        if (!__all_sync(0xffffffffu, t0 && t1 && t2) &&
                            (!warp_wait(t_empty(b), tph, lim) || !warp_wait(a_full(s), ph, lim) ||
                             !warp_wait(b_full(bs), bph, lim))) return false;
                        tc_fence_after();
                        const uint64_t da = da0 + (uint32_t)(s * (A_BYTES >> 4)), db = db0 + (uint32_t)(bs * (K_::B_BYTES >> 4));
                        if (elect_one()) {
#pragma unroll
                            for (int i = 0; i < BK / 32; ++i)
                                umma_8bit<false>(tmem + (uint32_t)(b * 4 * NT), da + i * 2, db + i * 2, idesc, i > 0);
                            umma_commit(t_full(b));
                        }
                        ++issued;
                        if (++s == A_STAGES) { s = 0; ph ^= 1; }
                        if (++bs == SB) { bs = 0; bph ^= 1; }
                        if (++b == 2) { b = 0; tph ^= 1; }
                    }
                    return true;
                });
            };
            if (multiply(w1, P1)) multiply(w2, P2);
            if (issued > 0)                      // MMAs retire before tensor memory is freed
                mbar_wait_for(t_full((issued - 1) & 1), (uint32_t)((issued - 1) >> 1) & 1u, kDrainNs, &g_error);
        }
        __syncwarp();
    } else if (warp < FINISHER) {
        // ------------------------------------------------ activations
        if (ok) {
            // The (block, token) pairs of a piece go round the warps, so that several
            // blocks are under way when an expert has few tokens.  Every warp still
            // waits for every block's stage and arrives on it: a parity tells
            // neighbouring uses of a stage apart and no more.
            const int me = warp - 2;
            int bs = 0;
            uint32_t bph = 1;
            auto split = [&](const Work &w, auto second_, auto parts) {
                constexpr bool SECOND = decltype(second_)::value;
                constexpr int PARTS = decltype(parts)::value;
                return for_pieces(w, [&](int u, int k0, int k1) {
                    const int ch = u / w.tiles, n = rt.c_n[ch], first = rt.c_first[ch];
                    const uint32_t part_bytes = (uint32_t)((n + 7) / 8 * 8 * BK);
                    if (SECOND) {                  // the chunk's h is whole?
                        bool go = true;
                        if (lane == 0) go = grid_wait(done + ch, (unsigned)w1.tiles, lim);
                        if (!__all_sync(0xffffffffu, go)) return false;
                    }
                    const int dk = SPLITTERS / n, di = SPLITTERS - dk * n;
                    int ik = k0 + me / n, i = me - me / n * n;     // this warp's next pair
                    int fk = ik, fi = i;                           // its next pair to load
                    auto advance = [&](int &k, int &c) {
                        k += dk;
                        c += di;
                        if (c >= n) { c -= n; ++k; }
                    };
                    // h: 4 values of a token's block; x: 16 bytes of its parts, and its scale
                    struct Loaded { float4 v; float scale; };
                    auto fetch = [&]() {
                        Loaded f{make_float4(0.0f, 0.0f, 0.0f, 0.0f), 0.0f};
                        if (fk < k1) {
                            if (SECOND) {
                                f.v = load_quad(p.h + (int64_t)rt.list[first + fi] * p.ldh, fk * BK + 4 * lane, p.F, true);
                            } else {
                                const int64_t at = (int64_t)rt.token[first + fi] * w.kb + fk;
                                if (lane < 8 * PARTS)
                                    f.v = __ldcg(reinterpret_cast<const float4 *>(p.x_parts + at * (PARTS * BK / 4)) + lane);
                                f.scale = __ldcg(p.x_scales + at);
                            }
                            advance(fk, fi);
                        }
                        return f;
                    };
                    Loaded v0 = fetch(), v1 = fetch();
                    for (int kb = k0; kb < k1; ++kb) {
                        if (!warp_wait(b_empty(bs), bph, lim)) return false;
                        if (ik == kb) {
                            do {
                                const Loaded l = v0;
                                v0 = v1;
                                v1 = fetch();
                                // part j of token i is row j n8 + i: 128 bytes, the 16-byte chunk
                                // index flipped by the row's low 3 bits (128-byte swizzle), i's
                                const uint32_t row = b_at(bs) + (uint32_t)(i * BK);
                                if (SECOND) {
                                    const uint32_t to = row + ((uint32_t)(((lane >> 2) ^ (i & 7)) << 4) | (uint32_t)(4 * (lane & 3)));
                                    split_block<PARTS>(l.v, &b_scale[bs][i], lane, [&](int j, uint32_t q) {
                                        asm volatile("st.shared.u32 [%0], %1;" :: "r"(to + j * part_bytes), "r"(q) : "memory");
                                    });
                                } else {
                                    const uint32_t to = row + (uint32_t)(lane >> 3) * part_bytes + (uint32_t)(((lane & 7) ^ (i & 7)) << 4);
                                    if (lane < 8 * PARTS)
                                        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};"
                                                     :: "r"(to), "f"(l.v.x), "f"(l.v.y), "f"(l.v.z), "f"(l.v.w) : "memory");
                                    if (lane == 0) b_scale[bs][i] = l.scale;
                                }
                                advance(ik, i);
                            } while (ik == kb);
                            // generic-proxy stores must be visible to the tensor core's reads
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                        }
                        if (lane == 0) mbar_arrive(b_full(bs));
                        if (++bs == SB) { bs = 0; bph ^= 1; }
                    }
                    return true;
                });
            };
            if (split(w1, std::false_type{}, std::integral_constant<int, P1>{}))
                split(w2, std::true_type{}, std::integral_constant<int, P2>{});
        }
    } else if (warp == FINISHER) {
        // ------------------------------------------------ finished tiles
        // What a tile's end needs beyond its sums waits for memory: publishing h,
        // counting the CTAs done with a shared tile, adding its parts.  This warp does
        // that while the promoters go on with the next tile.
        if (ok) {
            uint32_t ph = 0;
            auto finish = [&](const Work &w, bool second) {
                return for_pieces(w, [&](int u, int k0, int k1) {
                    if (!warp_wait(tile_left, ph, lim)) return false;
                    if (lane == 0) mbar_arrive(tile_taken);
                    ph ^= 1;
                    const int ch = u / w.tiles, tile = u - ch * w.tiles;
                    bool publish = !second;
                    if (k0 != 0 || k1 != w.kb) {
                        const Parts pt(w, u);
                        const float *parts = p.parts + (second ? phase_parts : 0);
                        bool last = false;
                        if (lane == 0)
                            last = add_acq_rel(&p.arrivals[second ? w1.tiles * rt.chunks + u : u]) == (unsigned)(pt.c1 - pt.c0);
                        last = __any_sync(0xffffffffu, last);
                        __syncwarp();
                        publish = publish && last;
                        if (last) {
                            const int n = rt.c_n[ch], first = rt.c_first[ch];
                            // 4 neighbouring rows for each lane
                            const int r0 = 4 * lane, f = tile * 64 + (r0 >> 5) * 16 + (r0 & 15);
#pragma unroll 1
                            for (int c = 0; c < n; c += 8) {
                                float4 s[8];
                                pt.sum8(parts, NT * ROWS, r0, c, n, s);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    if (c + i >= n) break;
                                    const int slot = rt.list[first + c + i];
                                    if (second) {
                                        if (tile * ROWS + r0 < p.ldo)
                                            __stcg(reinterpret_cast<float4 *>(p.out + (int64_t)slot * p.ldo + tile * ROWS + r0), s[i]);
                                    } else {
                                        // up's rows are 16 after gate's: four lanes on
                                        const float4 up = make_float4(__shfl_xor_sync(0xffffffffu, s[i].x, 4), __shfl_xor_sync(0xffffffffu, s[i].y, 4),
                                                                      __shfl_xor_sync(0xffffffffu, s[i].z, 4), __shfl_xor_sync(0xffffffffu, s[i].w, 4));
                                        if ((lane & 4) == 0 && f < p.ldh)
                                            __stcg(reinterpret_cast<float4 *>(p.h + (int64_t)slot * p.ldh + f),
                                                   make_float4(gated(s[i].x, up.x), gated(s[i].y, up.y), gated(s[i].z, up.z), gated(s[i].w, up.w)));
                                    }
                                }
                            }
                            __syncwarp();
                        }
                    }
                    if (publish && lane == 0) add_release(done + ch);
                    return true;
                });
            };
            if (finish(w1, false)) finish(w2, true);
        }
        __syncwarp();
        if (lane == 0) add_release(&p.sync[2]);
    } else {
        // ------------------------------------------------ promotion
        const int q = warp & 3, row = q * 32 + lane;
        int s = 0, b = 0, bs = 0;
        uint32_t tph = 0, fph = 1;
        auto promote = [&](const Work &w, bool second, auto parts_) {
            constexpr int PARTS = decltype(parts_)::value;
            return for_pieces(w, [&](int u, int k0, int k1) {
                const int ch = u / w.tiles, tile = u - ch * w.tiles;
                const int e = rt.c_expert[ch], n = rt.c_n[ch], n8 = (n + 7) / 8 * 8, first = rt.c_first[ch];
                // this row's weight scales, block after block
                const float *ws;
                if (second) {
                    ws = p.s_down + ((int64_t)e * ((p.D + 127) / 128) + tile) * w.kb;
                } else {
                    ws = (lane < 16 ? p.s_gate : p.s_up) + ((int64_t)e * ((p.F + 127) / 128) + tile / 2) * w.kb;
                }
                float acc[NT];
#pragma unroll
                for (int i = 0; i < NT; ++i) acc[i] = 0.0f;
                float ws_next = __ldg(ws + k0);
                for (int kb = k0; kb < k1; ++kb) {
                    const float sw = ws_next;
                    if (kb + 1 < k1) ws_next = __ldg(ws + kb + 1);
                    if (!warp_wait(t_full(b), tph, lim)) return false;
                    tc_fence_after();
                    // the block's MMAs are done with the weights' stage
                    if (q == 0 && lane == 0) mbar_arrive(a_empty(s));
                    if (++s == A_STAGES) s = 0;
                    const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * 4 * NT);
#pragma unroll
                    for (int i0 = 0; i0 < NT; i0 += 8) {
                        if (i0 >= n8) break;
                        uint32_t r[PARTS][8];
                        tmem_ld_parts(ta + (uint32_t)i0, (uint32_t)n8, r);
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            const float2 ts = *reinterpret_cast<const float2 *>(&b_scale[bs][i0 + j]);
                            float2 t = make_float2(__uint_as_float(r[PARTS - 1][j]), __uint_as_float(r[PARTS - 1][j + 1]));
#pragma unroll
                            for (int i = PARTS - 2; i >= 0; --i)
                                t = __ffma2_rn(t, make_float2(1.0f / 32.0f, 1.0f / 32.0f),
                                               make_float2(__uint_as_float(r[i][j]), __uint_as_float(r[i][j + 1])));
                            // (the weights' scale first: times a small token's, a power of two from 2^-126
                            // up, it could lose bits below the normal numbers that the result has)
                            const float2 a = __ffma2_rn(__fmul2_rn(t, make_float2(sw, sw)), ts, make_float2(acc[i0 + j], acc[i0 + j + 1]));
                            acc[i0 + j] = a.x;
                            acc[i0 + j + 1] = a.y;
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(t_empty(b));
                        mbar_arrive(b_empty(bs));   // (the block's MMAs are done too)
                    }
                    if (++b == 2) { b = 0; tph ^= 1; }
                    if (++bs == SB) bs = 0;
                }
                if (k0 != 0 || k1 != w.kb) {
                    // a share of the sum
                    const Parts pt(w, u);
                    float *dst = p.parts + (second ? phase_parts : 0) + ((int64_t)blockIdx.x * 2 + ((int)blockIdx.x == pt.c0 ? pt.part0 : 0)) * NT * ROWS + row;
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        if (i < n) __stcg(dst + i * ROWS, acc[i]);
                } else if (second) {
                    const int d = tile * ROWS + row;
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        if (i < n && d < p.D) __stcg(p.out + (int64_t)rt.list[first + i] * p.ldo + d, acc[i]);
                } else {
                    // gate in the lower 16 lanes, up in the upper ones: the lower take the
                    // even tokens, the upper the odd ones
                    const int f = tile * 64 + q * 16 + (lane & 15);
#pragma unroll
                    for (int i = 0; i < NT; i += 2) {
                        if (i >= n) break;
                        const bool low = lane < 16;
                        const float other = __shfl_xor_sync(0xffffffffu, low ? acc[i + 1] : acc[i], 16);
                        const int c = low ? i : i + 1;
                        if (c < n && f < p.F)
                            __stcg(p.h + (int64_t)rt.list[first + c] * p.ldh + f,
                                   gated(low ? acc[i] : other, low ? other : acc[i + 1]));
                    }
                }
                // the finisher has taken the tile before; this one is its now
                if (!warp_wait(tile_taken, fph, lim)) return false;
                fph ^= 1;
                __syncwarp();
                if (lane == 0) mbar_arrive(tile_left);
                return true;
            });
        };
        if (ok && promote(w1, false, std::integral_constant<int, P1>{}))
            promote(w2, true, std::integral_constant<int, P2>{});
    }
    // ---- phase 3: y
    if (threadIdx.x == THREADS - 1) s_last = grid_wait(&p.sync[2], G, lim);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free<false>(tmem, K_::COLS);
    }
    if (s_last && ok) {
        // 32 columns of a token per warp, neighbouring tasks on different CTAs
        const int across = (p.D + 31) / 32;
        for (int task = warp * (int)G + blockIdx.x; task < p.T * across; task += (THREADS / 32) * G) {
            const int t = task / across, d = (task - t * across) * 32 + lane;
            const float *src = p.out + (int64_t)t * p.topk * p.ldo + min(d, p.D - 1);
            float sum = 0.0f;
#pragma unroll 4
            for (int j = 0; j < p.topk; ++j)
                sum = __fmaf_rn(__ldcg(p.weights + t * p.topk + j), __ldcg(src + (int64_t)j * p.ldo), sum);
            if (d < p.D) {
                XT *y = static_cast<XT *>(p.y) + (int64_t)t * p.ldy + d;
                if (sizeof(XT) == 2) *reinterpret_cast<__nv_bfloat16 *>(y) = __float2bfloat16_rn(sum);
                else *reinterpret_cast<float *>(y) = sum;
            }
        }
    }
    __syncthreads();
    // the last CTA to leave clears the barriers for the next call
    if (threadIdx.x == 0 && add_acq_rel(&p.sync[3]) == G - 1)
        p.sync[0] = p.sync[1] = p.sync[2] = p.sync[3] = 0;
}

}  // namespace moe

// ---------------------------------------------------------------- host side
int moe_take_device_error() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, moe::g_error, sizeof(v)) != cudaSuccess) return SGEMM_ERR_CUDA;
    if (v != 0 && cudaMemcpyToSymbol(moe::g_error, &zero, sizeof(zero)) != cudaSuccess)
        return SGEMM_ERR_CUDA;
    return v == 0 ? SGEMM_OK : (int)v;
}

// E matrices of rows x cols bytes in boxes of box_rows x 128, 128-byte swizzle.
static bool experts_map(CUtensorMap *m, const void *base, int64_t E, int64_t rows, int64_t cols, int64_t ld,
                        int64_t stride, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)E};
    cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)stride};
    cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename XT, int NT>
static int launch_moe(const CUtensorMap *maps, const moe::Params &p, int sms, cudaStream_t s) {
    auto kern = moe::moe_kernel<XT, NT>;
    constexpr int smem = moe::Cfg<NT>::SMEM;
    static uint64_t attr_done = 0;   // bit d: the shared-memory opt-in is set on device d
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SGEMM_ERR_CUDA;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (!bit || !(__atomic_load_n(&attr_done, __ATOMIC_ACQUIRE) & bit)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return launch_status();
        __atomic_fetch_or(&attr_done, bit, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)sms);
    cfg.blockDim = dim3(moe::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    timing_mark(s, true);
    count_launch();
    cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], p);
    timing_mark(s, false);
    return launch_status();
}

template <typename XT>
static int launch_moe(const CUtensorMap *maps, const moe::Params &p, int nt, int sms, cudaStream_t s) {
    return nt == 8    ? launch_moe<XT, 8>(maps, p, sms, s)
           : nt == 16 ? launch_moe<XT, 16>(maps, p, sms, s)
           : nt == 32 ? launch_moe<XT, 32>(maps, p, sms, s)
                      : launch_moe<XT, 64>(maps, p, sms, s);
}

static int run_moe(moe::Params p, int x_type, const void *gate, const void *up, int64_t ld_in, int64_t stride_in,
                   const void *down, int64_t ld_down, int64_t stride_down, cudaStream_t s) {
    int sms = 0;
    int st = usable_device(&sms);
    if (st != SGEMM_OK) return st;
    const int64_t T = p.T, D = p.D, F = p.F, E = p.E, slots = T * p.topk;
    // Columns for twice the tokens that an expert has on average; one with more is
    // taken in several chunks, each of which reads its weights again.  Fewer columns
    // leave room for more stages: T = 64, 8 tokens an expert, 145 us with 64 columns.
    const int64_t want = std::min<int64_t>(T, (2 * slots + E - 1) / E);
    const int nt = want <= 8 ? 8 : want <= 16 ? 16 : want <= 32 ? 32 : 64;
    const int64_t logit_tasks = ((T + moe::LOGIT_T - 1) / moe::LOGIT_T) * ((E + moe::LOGIT_E - 1) / moe::LOGIT_E);   // a warp each
    p.slices = p.router ? (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(fp8::blocks_of(D), moe::LOGIT_SLICES),
                                                                      sms * (moe::THREADS / 32) / logit_tasks))
                        : 1;
    p.ldh = (int)((F + 3) / 4 * 4);
    p.ldo = (int)((D + 3) / 4 * 4);
    const int64_t chunks = std::min<int64_t>(slots, std::min(E, slots) + slots / nt);   // at most
    const int64_t arrivals = chunks * ((F + 63) / 64 + (D + 127) / 128 + 1);
    // blocks of 128 k and tasks are counted in int
    if (arrivals * fp8::blocks_of(std::max(D, F)) > INT32_MAX || T * D > INT32_MAX) return SGEMM_ERR_UNSUPPORTED;
    p.n_arrivals = (int)arrivals;
    auto up256 = [](size_t b) { return (b + 255) & ~size_t(255); };
    // the barriers keep a workspace of their own: they are zero between calls
    void *sync = nullptr, *ws = nullptr;
    st = workspace(s, 256, &sync, 3, true);
    if (st != SGEMM_OK) return st;
    const size_t b_arr = up256((size_t)arrivals * 4), b_log = up256((size_t)p.slices * T * E * 4),
                 b_xp = up256((size_t)T * fp8::blocks_of(D) * (x_type == SGEMM_TYPE_F32 ? 4 : 2) * moe::BK),
                 b_xs = up256((size_t)T * fp8::blocks_of(D) * 4), b_h = up256((size_t)slots * p.ldh * 4), b_parts = up256((size_t)2 * sms * 2 * nt * moe::ROWS * 4),
                 b_out = up256((size_t)slots * p.ldo * 4);
    st = workspace(s, b_arr + b_log + b_xp + b_xs + b_h + b_parts + b_out, &ws);
    if (st != SGEMM_OK) return st;
    char *w = static_cast<char *>(ws);
    p.sync = static_cast<unsigned int *>(sync);
    p.arrivals = reinterpret_cast<unsigned int *>(w);
    p.logit_parts = reinterpret_cast<float *>(w += b_arr);
    p.x_parts = reinterpret_cast<uint32_t *>(w += b_log);
    p.x_scales = reinterpret_cast<float *>(w += b_xp);
    p.h = reinterpret_cast<float *>(w += b_xs);
    p.parts = reinterpret_cast<float *>(w += b_h);
    p.out = reinterpret_cast<float *>(w += b_parts);
    p.wait_ns = tc_wait_limit();
    const int esize = x_type == SGEMM_TYPE_F32 ? 4 : 2;
    p.x_vec = reinterpret_cast<uintptr_t>(p.x) % (4 * esize) == 0 && p.ldx % 4 == 0;
    CUtensorMap maps[3];
    if (!experts_map(&maps[0], gate, E, F, D, ld_in, stride_in, 16) ||
        !experts_map(&maps[1], up, E, F, D, ld_in, stride_in, 16) ||
        !experts_map(&maps[2], down, E, D, F, ld_down, stride_down, 128))
        return SGEMM_ERR_UNSUPPORTED;
    return x_type == SGEMM_TYPE_F32 ? launch_moe<float>(maps, p, nt, sms, s)
                                    : launch_moe<__nv_bfloat16>(maps, p, nt, sms, s);
}

}  // namespace sgemm_gb300

using namespace sgemm_gb300;

extern "C" int sgemm_moe(int64_t T, int64_t D, int64_t F, int64_t E, int64_t topk, const void *x, int x_type,
                         int64_t ldx, const float *router, float *logits, const void *gate,
                         const float *s_gate, const void *up, const float *s_up, int64_t ld_in,
                         int64_t stride_in, const void *down, const float *s_down, int64_t ld_down,
                         int64_t stride_down, int renormalize, void *y, int64_t ldy, int32_t *indices,
                         float *weights, sgemm_stream_t stream) {
    const int64_t most = 1 << 20;                  // widths (tiles and blocks are ints)
    if (T < 0 || T > moe::MAX_T) return -1;
    if (D < 1 || D > most) return -2;
    if (F < 1 || F > most) return -3;
    if (E < 1 || E > moe::MAX_E) return -4;
    if (topk < 1 || topk > std::min<int64_t>(E, moe::MAX_TOPK)) return -5;
    if (!fp8::is_float_type(x_type)) return -7;
    auto bad = [](const void *q, int align) { return q == nullptr || reinterpret_cast<uintptr_t>(q) % align != 0; };
    const int esize = x_type == SGEMM_TYPE_F32 ? 4 : 2;
    if (T > 0 && bad(x, esize)) return -6;
    if (ldx < D) return -8;
    if (router != nullptr && bad(router, 4)) return -9;
    if (T > 0 && bad(logits, 4)) return -10;
    if (T > 0 && gate == nullptr) return -11;
    if (T > 0 && bad(s_gate, 4)) return -12;
    if (T > 0 && up == nullptr) return -13;
    if (T > 0 && bad(s_up, 4)) return -14;
    if (ld_in < D) return -15;
    if (stride_in < F * ld_in) return -16;
    if (T > 0 && down == nullptr) return -17;
    if (T > 0 && bad(s_down, 4)) return -18;
    if (ld_down < F) return -19;
    if (stride_down < D * ld_down) return -20;
    if (T > 0 && bad(y, esize)) return -22;
    if (ldy < D) return -23;
    if (T > 0 && bad(indices, 4)) return -24;
    if (T > 0 && bad(weights, 4)) return -25;
    if (!aligned16(gate) || !aligned16(up) || !aligned16(down) || ld_in % 16 || stride_in % 16 || ld_down % 16 ||
        stride_down % 16)
        return SGEMM_ERR_UNSUPPORTED;
    if (T == 0) return SGEMM_OK;
    moe::Params p{};
    p.T = (int)T; p.D = (int)D; p.F = (int)F; p.E = (int)E; p.topk = (int)topk;
    p.x = x; p.ldx = ldx; p.router = router; p.logits = logits;
    p.s_gate = s_gate; p.s_up = s_up; p.s_down = s_down;
    p.renormalize = renormalize;
    p.y = y; p.ldy = ldy; p.indices = indices; p.weights = weights;
    try {
        return run_moe(p, x_type, gate, up, ld_in, stride_in, down, ld_down, stride_down,
                       reinterpret_cast<cudaStream_t>(stream));
    } catch (const std::bad_alloc &) {
        return SGEMM_ERR_NOMEM;
    }
}
