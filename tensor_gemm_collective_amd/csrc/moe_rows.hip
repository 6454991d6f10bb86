// Row moves of a MoE layer: tokens into their send rows, the experts' rows
// summed by their gates, and the gradient of that sum.
#include "row_ops.h"

namespace coc {
namespace {

constexpr int kMaxTopk = 16;

// out[positions[t][j]] = x[t].  tpr threads a token; its row is read once.
template <class T, RowKind KIND>
__global__ __launch_bounds__(256) void permute_rows(const T* x, const int32_t* positions, T* out, int64_t tokens,
                                                    int64_t rows, int n, int topk, int tpr) {
    const int64_t t = (int64_t)blockIdx.x * (256 / tpr) + threadIdx.x / tpr;
    if (t >= tokens) return;
    for (int i = (int)(threadIdx.x % tpr); i * kVec<T> < n; i += tpr) {
        const Cols<T, KIND> col(i, n);
        Packed<T> v;
        col.load(x + t * n, n, &v);
        for (int j = 0; j < topk; ++j) {
            const int64_t r = positions[t * topk + j];
            if (r >= 0 && r < rows) col.store(out + r * n, n, v);
        }
    }
}

// y[t] = sum_j gates[t][j] h[positions[t][j]], in order of j (gates NULL: 1).
template <class T, RowKind KIND>
__global__ __launch_bounds__(256) void combine_rows(const T* h, const int32_t* positions, const float* gates, T* y,
                                                    int64_t tokens, int64_t rows, int n, int topk, int tpr) {
    const int64_t t = (int64_t)blockIdx.x * (256 / tpr) + threadIdx.x / tpr;
    if (t >= tokens) return;
    for (int v = (int)(threadIdx.x % tpr); v * kVec<T> < n; v += tpr) {
        const Cols<T, KIND> col(v, n);
        float s[kVec<T>];
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) s[i] = 0.0f;
        for (int j = 0; j < topk; ++j) {
            const int64_t r = positions[t * topk + j];
            if (r < 0 || r >= rows) continue;
            const float g = gates ? gates[t * topk + j] : 1.0f;
            Packed<T> f;
            col.load(h + r * n, n, &f);
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) s[i] += g * f.get(i);
        }
        Packed<T> o;
        o.set(s);
        col.store(y + t * n, n, o);
    }
}

// dh[positions[t][j]] = gates[t][j] dy[t],  dgates[t][j] = <dy[t], h[positions[t][j]]>.
// A wave a (token, choice).
template <class T, RowKind KIND>
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
    for (int v = lane; v * kVec<T> < n; v += 64) {
        const Cols<T, KIND> col(v, n);
        Packed<T> d, f, o;
        col.load(dy + t * n, n, &d);
        col.load(h + r * n, n, &f);
        float p[kVec<T>];
#pragma unroll
        for (int q = 0; q < kVec<T>; ++q) {
            s += col.has(q, n) ? d.get(q) * f.get(q) : 0.0f;
            p[q] = product(d.get(q), g);
        }
        o.set(p);
        col.store(dh + r * n, n, o);
    }
    s = lanes_sum<64>(s);
    if (lane == 0) dgates[i] = s;
}

int threads_per_row(int64_t vecs) {
    int t = 8;
    while (t < 256 && t < vecs) t *= 2;
    return t;
}

// f(T, kind of a row of n).
template <class F>
void by_type(coc_dtype dt, int64_t n, F&& f) {
    auto call = [&](auto t) {
        if (n < kVec<decltype(t)>)
            f(t, std::integral_constant<RowKind, kTiny>());
        else
            f(t, std::integral_constant<RowKind, kRagged>());
    };
    if (dt == COC_F32)
        call(float());
    else if (dt == COC_F16)
        call(f16_t());
    else
        call(bf16_t());
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
    by_type(dt, n, [&](auto t, auto kind) {
        using T = decltype(t);
        const int tpr = threads_per_row(ceil_div(n, kVec<T>));
        permute_rows<T, decltype(kind)::value><<<dim3((uint32_t)ceil_div(tokens, 256 / tpr)), dim3(256), 0, stream>>>(
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
    by_type(dt, n, [&](auto t, auto kind) {
        using T = decltype(t);
        const int tpr = threads_per_row(ceil_div(n, kVec<T>));
        combine_rows<T, decltype(kind)::value><<<dim3((uint32_t)ceil_div(tokens, 256 / tpr)), dim3(256), 0, stream>>>(
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
    by_type(dt, n, [&](auto t, auto kind) {
        using T = decltype(t);
        combine_backward<T, decltype(kind)::value><<<dim3((uint32_t)ceil_div(tokens * topk, 4)), dim3(256), 0, stream>>>(
            (const T*)dy, (const T*)h, positions, gates, (T*)dh, dgates, tokens, rows, (int)n, topk);
    });
    return launched("combine backward");
}

}  // extern "C"
