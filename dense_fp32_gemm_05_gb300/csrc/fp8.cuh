// 8-bit floating point: types, group geometry and conversions shared by the
// quantiser, the block-scaled product and the mixture-of-experts layer.
//
// A quantised matrix is codes (E4M3 or E5M2) and fp32 scales, one for each
// group of 128 along the dimension a product sums over (1 x 128 or 128 x 1),
// or for each block of 128 x 128; the value is code * scale.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/sgemm_gb300.h"

namespace sgemm_gb300 {
namespace fp8 {

constexpr int GROUP = 128;

inline int64_t blocks_of(int64_t n) { return (n + GROUP - 1) / GROUP; }
inline bool is_code_type(int t) { return t == SGEMM_TYPE_E4M3 || t == SGEMM_TYPE_E5M2; }
inline bool is_float_type(int t) { return t == SGEMM_TYPE_F32 || t == SGEMM_TYPE_BF16; }

// Two fp32 values to two codes (the first in the low byte): round to nearest
// even, values past the largest code to the largest code, NaN to NaN.
template <bool E5M2>
__device__ __forceinline__ uint32_t codes2(float a, float b) {
    uint16_t r;
    if (E5M2) asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    else asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Four values to four codes in ascending bytes.
template <bool E5M2>
__device__ __forceinline__ uint32_t codes4(const float (&v)[4]) {
    return codes2<E5M2>(v[0], v[1]) | (codes2<E5M2>(v[2], v[3]) << 16);
}

}  // namespace fp8
}  // namespace sgemm_gb300
