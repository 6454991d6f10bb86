// Row moves of a MoE layer: tokens into their send rows, the experts' rows
// summed by their gates, and the gradient of that sum.
#include "row_ops.h"

namespace coc {
namespace {

constexpr int kMaxTopk = 16;

// out[positions[t][j]] = x[t].  tpr threads a token; its row is read once.  Bound
// by memory: 8192 tokens x 12288 to two rows each (bf16, 604 MB) 112 us, 5.4 TB/s;
// 300 x 130 3.0 us, a launch.
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
// Bound by memory: 8192 x 12288 from two rows each (bf16, 604 MB) 109 us, 5.5 TB/s.
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
// TPT threads a token walk its columns, KB choices at a time: a vector of dy is
// read once for them and their rows of h are on their way together.  Bound by
// memory: 8192 x 12288 top 2 (bf16, 1.01 GB) 191 us, 5.3 TB/s; 30000 x 1001 top 8
// 238 us, 4.3 TB/s (a wave a choice: 202 and 275).
template <class T, RowKind KIND, int KB, int TPT>
__global__ __launch_bounds__(256) void combine_backward(const T* dy, const T* h, const int32_t* positions,
                                                        const float* gates, T* dh, float* dgates, int64_t tokens,
                                                        int64_t rows, int n, int topk) {
    __shared__ float sums[KB][4];
    const int64_t t = (int64_t)blockIdx.x * (256 / TPT) + threadIdx.x / TPT;
    if (t >= tokens) return;   // a whole wave, or with TPT 256 nobody
    const int lane = threadIdx.x % TPT;
    for (int j0 = 0; j0 < topk; j0 += KB) {
        int64_t r[KB];
        float g[KB], s[KB];
        bool ok[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const int64_t at = t * topk + min(j0 + j, topk - 1);
            r[j] = positions[at];
            g[j] = gates[at];
            const bool named = r[j] >= 0 && r[j] < rows;
            ok[j] = named && j0 + j < topk;
            if (!named) r[j] = 0;   // read and not used
            s[j] = 0.0f;
        }
        if (rows > 0)
            for (int v = lane; v * kVec<T> < n; v += TPT) {
                const Cols<T, KIND> col(v, n);
                Packed<T> d, f[KB];
                col.load(dy + t * n, n, &d);
#pragma unroll
                for (int j = 0; j < KB; ++j) col.load(h + r[j] * n, n, &f[j]);
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    float p[kVec<T>];
#pragma unroll
                    for (int q = 0; q < kVec<T>; ++q) {
                        s[j] += col.has(q, n) ? d.get(q) * f[j].get(q) : 0.0f;
                        p[q] = product(d.get(q), g[j]);
                    }
                    if (ok[j]) {
                        Packed<T> o;
                        o.set(p);
                        col.store(dh + r[j] * n, n, o);
                    }
                }
            }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            s[j] = lanes_sum<64>(s[j]);
            if constexpr (TPT > 64) {
                if ((threadIdx.x & 63) == 0) sums[j][threadIdx.x >> 6] = s[j];
            }
        }
        if constexpr (TPT > 64) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < KB; ++j) s[j] = sums[j][0] + sums[j][1] + sums[j][2] + sums[j][3];
            __syncthreads();
        }
        if (lane == 0) {
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (j0 + j < topk) dgates[t * topk + j0 + j] = ok[j] ? s[j] : 0.0f;
        }
    }
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
        else if (n % kVec<decltype(t)> == 0)
            f(t, std::integral_constant<RowKind, kWhole>());
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
    s = check_matrix(tokens, topk, "positions");
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
        auto go = [&](auto kb, auto tpt) {
            constexpr int TPT = decltype(tpt)::value;
            combine_backward<T, decltype(kind)::value, decltype(kb)::value, TPT>
                <<<dim3((uint32_t)ceil_div(tokens, 256 / TPT)), dim3(256), 0, stream>>>(
                    (const T*)dy, (const T*)h, positions, gates, (T*)dh, dgates, tokens, rows, (int)n, topk);
        };
        const std::integral_constant<int, 64> wave;
        const std::integral_constant<int, 256> group;
        const std::integral_constant<int, 2> two;
        const std::integral_constant<int, 4> four;
        const bool wide = ceil_div(n, kVec<T>) > 128;   // vectors enough for four waves
        if (topk <= 2)
            wide ? go(two, group) : go(two, wave);
        else
            wide ? go(four, group) : go(four, wave);
    });
    return launched("combine backward");
}

}  // extern "C"
