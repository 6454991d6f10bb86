// 8-bit floating point with scales, shared by the operators that write it.
//
// A block of 128 values y along a row (or of 128 x 128) has the scale
//   s = max(max |y|, 2^-96) / 448     (448: the largest e4m3 value)
// and the stored values q = e4m3(y * (448 / max)), rounded to nearest even.  The
// least value keeps 448 / max finite; a block of zeros is stored as zeros.  The
// largest value is found on the bits, where NaN lies above infinity and both
// above the rest, so a block that holds either gets the scale NaN or infinity
// and reads back as NaN throughout.
#pragma once

#include "row_ops.h"

namespace coc {

constexpr int kScaleBlock = 128;
constexpr float kTopFp8 = 448.0f;

struct Fp8Scale {
    float scale, inverse;
};
// `top`: the bits of the block's largest |y|.
__device__ __forceinline__ Fp8Scale fp8_scale(uint32_t top) {
    const float t = __uint_as_float(max(top, 0x0f800000u));   // 2^-96
    return {t / kTopFp8, kTopFp8 / t};
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Four values times `inverse` as four bytes.
__device__ __forceinline__ uint32_t pack_fp8(const float* y, float inverse) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * inverse, y[1] * inverse, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2] * inverse, y[3] * inverse, w, true);
}

// N (4 or 8) values to 8 bits at `at` (N-byte aligned).
template <int N>
__device__ __forceinline__ void store_fp8(uint8_t* at, const float* y, float inverse) {
    if constexpr (N == 4) {
        __builtin_nontemporal_store(pack_fp8(y, inverse), (uint32_t*)at);
    } else {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        __builtin_nontemporal_store(u32x2{pack_fp8(y, inverse), pack_fp8(y + 4, inverse)}, (u32x2*)at);
    }
}

}  // namespace coc
