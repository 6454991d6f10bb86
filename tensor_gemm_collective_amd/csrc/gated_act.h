// The activations of the gated feed-forward block, in binary32.
//
//   silu(g)  = g p,  p = 1 / (1 + exp(-g))
//   gelu(g)  = g p,  p = 1 / (1 + exp(-2 z)),  z = sqrt(2 / pi) (g + 0.044715 g^3)
//              (the tanh form: (1 + tanh z) / 2 = p)
// Both slopes are p + g p (1 - p) r with r = 1 for silu and 2 z' for gelu.
#pragma once

#include "row_ops.h"

namespace coc {

// exp2 and the reciprocal are the hardware's: relative errors of about 1e-7 each.  The
// exponent's own rounding adds some |z| 2^-24 where p is far below 1 (2e-6 at g = -20),
// nothing beside a rounding to 16 or 8 bits; binary32 results take act_fine.
__device__ __forceinline__ float logistic_of(float minus_log2) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(minus_log2));
}

template <int ACT>
__device__ __forceinline__ float act_p(float g) {
    constexpr float log2e = 1.44269504088896f, c2 = 1.59576912160573f;   // 2 sqrt(2 / pi)
    if constexpr (ACT == COC_ACT_SILU)
        return logistic_of(-log2e * g);
    else
        return logistic_of(-log2e * c2 * (g + 0.044715f * (g * g * g)));
}

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
    return g * act_p<ACT>(g);
}

// act(g) and its slope.  gelu's r is taken at g within [-20, 20]: past that p is 0 or 1
// to the last bit, and r of a large g would be infinite.
template <int ACT>
__device__ __forceinline__ void act_both(float g, float* value, float* slope) {
    const float p = act_p<ACT>(g), v = g * p;
    *value = v;
    if constexpr (ACT == COC_ACT_SILU) {
        *slope = p + v * (1.0f - p);
    } else {
        const float c = fminf(fmaxf(g, -20.0f), 20.0f);
        *slope = p + v * (1.0f - p) * (1.59576912160573f * (1.0f + 0.134145f * c * c));
    }
}

// For results in binary32: p and 1 - p by e = exp(-|z|), which neither loses where it is
// small.  The exponent is formed in binary64; exp2 takes its binary32 part and a
// multiply-add the rest.  Past |exponent| 1000 e is 0 all the same.  Memory bound like the
// 16-bit forms: 4096 x 3584 24.9 us for act(g) u, 41.2 for its gradient (24.7 and 41.0 with
// act_value and act_both).
template <int ACT>
__device__ __forceinline__ void act_fine(float g, float* value, float* slope) {
    constexpr double log2e = 1.4426950408889634, c2 = 1.5957691216057308;   // 2 sqrt(2 / pi)
    const double x = g;
    const double z = ACT == COC_ACT_SILU ? x * log2e : x * (c2 * log2e + (0.044715 * c2 * log2e) * (x * x));
    const double t = -fmin(fabs(z), 1000.0);
    const float hi = (float)t, lo = (float)(t - (double)hi) * 0.693147181f;
    const float e2 = __builtin_amdgcn_exp2f(hi), e = fmaf(e2, lo, e2);
    const float r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
    const float p = g < 0.0f ? er : r, rest = g < 0.0f ? r : er, v = g * p;
    *value = v;
    if constexpr (ACT == COC_ACT_SILU) {
        *slope = p + v * rest;
    } else {
        const float c = fminf(fmaxf(g, -20.0f), 20.0f);
        *slope = p + v * rest * (1.59576912160573f * (1.0f + 0.134145f * c * c));
    }
}

// By the type T of the rows.
template <class T, int ACT>
__device__ __forceinline__ float act_of(float g) {
    if constexpr (sizeof(T) == 4) {
        float value, slope;
        act_fine<ACT>(g, &value, &slope);
        return value;
    } else {
        return act_value<ACT>(g);
    }
}
template <class T, int ACT>
__device__ __forceinline__ void act_and_slope_of(float g, float* value, float* slope) {
    if constexpr (sizeof(T) == 4)
        act_fine<ACT>(g, value, slope);
    else
        act_both<ACT>(g, value, slope);
}

// f(integral constant of the activation).
template <class F>
__host__ __device__ __forceinline__ void by_act(coc_act act, F&& f) {
    if (act == COC_ACT_SILU)
        f(std::integral_constant<int, COC_ACT_SILU>());
    else
        f(std::integral_constant<int, COC_ACT_GELU>());
}

// Launches of gated_act.hip that gated_ffn.hip uses too; sizes and pointers are checked.
void launch_gated_act_backward(const void* dh, const void* gate_up, void* dgate_up, int64_t rows, int64_t f,
                               coc_act act, coc_dtype dt, hipStream_t stream);

}  // namespace coc
