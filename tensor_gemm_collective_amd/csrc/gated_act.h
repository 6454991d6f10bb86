// The activations of the gated feed-forward block, in binary32.
//
//   silu(g)  = g p,  p = 1 / (1 + exp(-g))
//   gelu(g)  = g p,  p = 1 / (1 + exp(-2 z)),  z = sqrt(2 / pi) (g + 0.044715 g^3)
//              (the tanh form: (1 + tanh z) / 2 = p)
// Both slopes are p + g p (1 - p) r with r = 1 for silu and 2 z' for gelu.
#pragma once

#include "row_ops.h"

namespace coc {

// exp2 and the reciprocal are the hardware's: relative errors of about 1e-7 each, and
// the exponent's own rounding |g| 2^-24 matters only where p is far below 1.
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
