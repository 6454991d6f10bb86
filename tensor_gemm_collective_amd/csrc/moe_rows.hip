// Row moves of a MoE layer: tokens into their send rows, the experts' rows
// summed by their gates, and the gradient of that sum.
#include "row_ops.h"

namespace coc {
namespace {

constexpr int kMaxTopk = 16;

// out[positions[t][j]] = x[t].  tpr threads a token; its row is read once.
template <class T>
__global__ __launch_bounds__(256) void permute_rows(const T* x, const int32_t* positions, T* out, int64_t tokens,
                                                    int64_t rows, int n, int topk, int tpr) {
    const int64_t t = (int64_t)blockIdx.x * (256 / tpr) + threadIdx.x / tpr;
    if (t >= tokens) return;
    for (int c = (int)(threadIdx.x % tpr) * kVec<T>; c < n; c += tpr * kVec<T>) {
        Packed<T> v;
        load_raw(x + t * n, c, n, &v);
        for (int j = 0; j < topk; ++j) {
            const int64_t r = positions[t * topk + j];
            if (r >= 0 && r < rows) store_raw(out + r * n, c, n, v);
        }
    }
}

// y[t] = sum_j gates[t][j] h[positions[t][j]], in order of j (gates NULL: 1).
template <class T>
__global__ __launch_bounds__(256) void combine_rows(const T* h, const int32_t* positions, const float* gates, T* y,
                                                    int64_t tokens, int64_t rows, int n, int topk, int tpr) {
    const int64_t t = (int64_t)blockIdx.x * (256 / tpr) + threadIdx.x / tpr;
    if (t >= tokens) return;
    for (int c = (int)(threadIdx.x % tpr) * kVec<T>; c < n; c += tpr * kVec<T>) {
        float s[kVec<T>];
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) s[i] = 0.0f;
        for (int j = 0; j < topk; ++j) {
            const int64_t r = positions[t * topk + j];
            if (r < 0 || r >= rows) continue;
            const float g = gates ? gates[t * topk + j] : 1.0f;
            float f[kVec<T>];
            load_vec(h + r * n, c, n, f);
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) s[i] += g * f[i];
        }
        store_vec(y + t * n, c, n, s);
    }
}

// dh[positions[t][j]] = gates[t][j] dy[t],  dgates[t][j] = <dy[t], h[positions[t][j]]>.
// A wave a (token, choice).
template <class T>
__global__ __launch_bounds__(256) void combine_backward(const T* dy, const T* h, const int32_t* positions,
                                                        const float* gates, T* dh, float* dgates, int64_t tokens,
                                                        int64_t rows, int n, int topk) {
    const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (i >= tokens * topk) return;
    const int lane = threadIdx.x & 63;
    const int64_t t = i / topk, r = positions[i];
    if (r < 0 || r >= rows) {
        if (lane == 0) dgates[i] = 0.0f;
        return;
    }
    const float g = gates[i];
    float s = 0.0f;
    for (int c = lane * kVec<T>; c < n; c += 64 * kVec<T>) {
        float d[kVec<T>], f[kVec<T>];
        load_vec(dy + t * n, c, n, d);
        load_vec(h + r * n, c, n, f);
#pragma unroll
        for (int q = 0; q < kVec<T>; ++q) {
            s += d[q] * f[q];
            d[q] = product(d[q], g);
        }
        store_vec(dh + r * n, c, n, d);
    }
    s = lanes_sum<64>(s);
    if (lane == 0) dgates[i] = s;
}

int threads_per_row(int64_t vecs) {
    int t = 8;
    while (t < 256 && t < vecs) t *= 2;
    return t;
}

template <class F>
void by_type(coc_dtype dt, F&& f) {
    if (dt == COC_F32)
        f(float());
    else if (dt == COC_F16)
        f(f16_t());
    else
        f(bf16_t());
}

coc_status check_rows(int64_t tokens, int64_t rows, int64_t n, int32_t topk, coc_dtype dt) {
    if (!dtype_valid(dt)) return fail(COC_ERR_DTYPE, "unknown dtype %d", (int)dt);
    if (n < 1) return fail(COC_ERR_SHAPE, "a row has at least one element (n=%lld)", (long long)n);
    if (topk < 1 || topk > kMaxTopk)
        return fail(COC_ERR_SHAPE, "topk must be in [1, %d] (got %d)", kMaxTopk, topk);
    coc_status s = check_matrix(tokens, n, "the tokens' matrix");
    if (s != COC_OK) return s;
    s = check_matrix(tokens * topk, 1, "positions");
    if (s != COC_OK) return s;
    return check_matrix(rows, n, "the rows' matrix");
}

}  // namespace
}  // namespace coc

extern "C" {

coc_status coc_moe_permute(const void* x, const int32_t* positions, void* out, int64_t tokens, int64_t rows,
                           int64_t n, int32_t topk, coc_dtype dt, hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_rows(tokens, rows, n, topk, dt);
    if (st != COC_OK) return st;
    if (tokens == 0 || rows == 0) return COC_OK;
    const int32_t es = (int32_t)elem_size(dt);
    const Arg args[] = {
        {x, tokens * n * es, es, false, "x"},
        {positions, tokens * topk * 4, 4, false, "positions"},
        {out, rows * n * es, es, true, "out"},
    };
    st = check_args(args, 3);
    if (st != COC_OK) return st;
    by_type(dt, [&](auto t) {
        using T = decltype(t);
        const int tpr = threads_per_row(ceil_div(n, kVec<T>));
        permute_rows<T><<<dim3((uint32_t)ceil_div(tokens, 256 / tpr)), dim3(256), 0, stream>>>(
            (const T*)x, positions, (T*)out, tokens, rows, (int)n, topk, tpr);
    });
    return launched("permute");
}

coc_status coc_moe_combine(const void* h, const int32_t* positions, const float* gates, void* y, int64_t tokens,
                           int64_t rows, int64_t n, int32_t topk, coc_dtype dt, hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_rows(tokens, rows, n, topk, dt);
    if (st != COC_OK) return st;
    if (tokens == 0) return COC_OK;
    const int32_t es = (int32_t)elem_size(dt);
    const Arg args[] = {
        {h, rows * n * es, es, false, "h"},
        {positions, tokens * topk * 4, 4, false, "positions"},
        {gates, gates ? tokens * topk * 4 : 0, 4, false, "gates"},
        {y, tokens * n * es, es, true, "y"},
    };
    st = check_args(args, 4);
    if (st != COC_OK) return st;
    by_type(dt, [&](auto t) {
        using T = decltype(t);
        const int tpr = threads_per_row(ceil_div(n, kVec<T>));
        combine_rows<T><<<dim3((uint32_t)ceil_div(tokens, 256 / tpr)), dim3(256), 0, stream>>>(
            (const T*)h, positions, gates, (T*)y, tokens, rows, (int)n, topk, tpr);
    });
    return launched("combine");
}

coc_status coc_moe_combine_backward(const void* dy, const void* h, const int32_t* positions, const float* gates,
                                    void* dh, float* dgates, int64_t tokens, int64_t rows, int64_t n, int32_t topk,
                                    coc_dtype dt, hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_rows(tokens, rows, n, topk, dt);
    if (st != COC_OK) return st;
    if (tokens == 0) return COC_OK;
    const int32_t es = (int32_t)elem_size(dt);
    const int64_t choices = tokens * topk * 4;
    const Arg args[] = {
        {dy, tokens * n * es, es, false, "dy"},
        {h, rows * n * es, es, false, "h"},
        {positions, choices, 4, false, "positions"},
        {gates, choices, 4, false, "gates"},
        {dh, rows * n * es, es, true, "dh"},
        {dgates, choices, 4, true, "dgates"},
    };
    st = check_args(args, 6);
    if (st != COC_OK) return st;
    by_type(dt, [&](auto t) {
        using T = decltype(t);
        combine_backward<T><<<dim3((uint32_t)ceil_div(tokens * topk, 4)), dim3(256), 0, stream>>>(
            (const T*)dy, (const T*)h, positions, gates, (T*)dh, dgates, tokens, rows, (int)n, topk);
    });
    return launched("combine backward");
}

}  // extern "C"
