// Layer norm, forward and backward, with the residual sum joined in.
#include "row_ops.h"

namespace coc {
namespace {

// Forward.  TPR threads hold one row in registers, EPT elements each, so a row
// is read once: its mean, then the mean of its squared distances from it (two
// sums over registers, which lose nothing where the mean is far from zero),
// then the output.
template <class T, class W, int TPR, int EPT>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void ln_forward(
    const T* x, const T* residual, const W* gamma, const W* beta, T* y, T* sum_out, float* mean_out, float* rstd_out,
    int64_t rows, int n, float eps) {
    constexpr int VN = kVec<T>, V = EPT / VN;
    constexpr int RPB = TPR == 64 ? 4 : 1;   // rows per workgroup: several where a wave holds one
    __shared__ float buf[2][TPR / 64];
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (RPB > 1 && row >= rows) return;
    const T* xr = x + row * n;
    float h[V][VN];
#pragma unroll
    for (int v = 0; v < V; ++v) load_vec(xr, (v * TPR + t) * VN, n, h[v]);
    if (residual) {
        const T* rr = residual + row * n;
        T* sr = sum_out + row * n;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * TPR + t) * VN;
            float r[VN];
            load_vec(rr, c, n, r);
#pragma unroll
            for (int i = 0; i < VN; ++i) h[v][i] = (float)(T)(h[v][i] + r[i]);   // the sum as stored
            store_vec(sr, c, n, h[v]);
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < VN; ++i) s += h[v][i];
    const float mean = (TPR == 64 ? lanes_sum<64>(s) : group_sum<TPR>(s, buf[0])) / (float)n;
    float q = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const float d = (v * TPR + t) * VN + i < n ? h[v][i] - mean : 0.0f;
            h[v][i] = d;
            q += d * d;
        }
    const float var = (TPR == 64 ? lanes_sum<64>(q) : group_sum<TPR>(q, buf[1])) / (float)n;
    const float rstd = 1.0f / sqrtf(var + eps);
    if (t == 0) {
        mean_out[row] = mean;
        rstd_out[row] = rstd;
    }
    T* yr = y + row * n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * TPR + t) * VN;
        if (c >= n) break;
        float g[VN], b[VN];
        load_n<VN>(gamma, c, n, g);
        if (beta) {
            load_n<VN>(beta, c, n, b);
        } else {
#pragma unroll
            for (int i = 0; i < VN; ++i) b[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) h[v][i] = h[v][i] * rstd * g[i] + b[i];
        store_vec(yr, c, n, h[v]);
    }
}

// Backward.  xh = (x - mean) rstd, g = dy gamma:
//   dx = rstd (g - avg(g) - xh avg(g xh)) + dsum,  dgamma = sum dy xh,  dbeta = sum dy.
// Workgroup b takes rows b, b + grid, ..., a thread always the same columns,
// so the columns' sums stay in its registers over all its rows and go to the
// workspace once, as row b of `part` (grid x 2 x n); ln_backward_sum adds
// those rows in order.  The next row is on its way while this one is summed.
template <class T, class W, int TPR, int EPT>
__global__ __launch_bounds__(TPR) void ln_backward(
    const T* dy, const T* x, const W* gamma, const float* mean_in, const float* rstd_in, const T* dsum, T* dx,
    float* part, int64_t rows, int n) {
    constexpr int VN = kVec<T>, V = EPT / VN;
    constexpr bool AHEAD = EPT * (int)sizeof(T) * TPR <= 32768;   // what the registers of 1024 threads hold
    __shared__ float buf[2][2][TPR / 64];
    const int t = threadIdx.x;
    float dg[V][VN], db[V][VN];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < VN; ++i) dg[v][i] = db[v][i] = 0.0f;
    struct Row {
        Packed<T> x[V], d[V], s[V];
        float mean, rstd;
    };
    auto load = [&](int64_t row, Row* r) {
        r->mean = mean_in[row];
        r->rstd = rstd_in[row];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * TPR + t) * VN;
            load_raw(x + row * n, c, n, &r->x[v]);
            load_raw(dy + row * n, c, n, &r->d[v]);
            if (dsum) load_raw(dsum + row * n, c, n, &r->s[v]);
        }
    };
    Row now, next;
    int64_t row = blockIdx.x;
    load(row, &now);   // grid <= rows
    for (int flip = 0; row < rows; row += gridDim.x, flip ^= 1) {
        if (AHEAD && row + gridDim.x < rows) load(row + gridDim.x, &next);
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float g[VN];
            load_n<VN>(gamma, (v * TPR + t) * VN, n, g);
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                // past n dy and gamma are 0, and so is every term
                const float d = now.d[v].get(i), xh = (now.x[v].get(i) - now.mean) * now.rstd;
                dg[v][i] += d * xh;
                db[v][i] += d;
                s1 += d * g[i];
                s2 += d * g[i] * xh;
            }
        }
        s1 = lanes_sum<64>(s1);
        s2 = lanes_sum<64>(s2);
        if constexpr (TPR > 64) {
            // two buffers in turn: one barrier a row
            if ((t & 63) == 0) {
                buf[flip][0][t >> 6] = s1;
                buf[flip][1][t >> 6] = s2;
            }
            __syncthreads();
            s1 = buf[flip][0][0];
            s2 = buf[flip][1][0];
#pragma unroll
            for (int w = 1; w < TPR / 64; ++w) {
                s1 += buf[flip][0][w];
                s2 += buf[flip][1][w];
            }
        }
        s1 /= (float)n;
        s2 /= (float)n;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * TPR + t) * VN;
            if (c >= n) break;
            float g[VN], o[VN];
            load_n<VN>(gamma, c, n, g);
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                const float xh = (now.x[v].get(i) - now.mean) * now.rstd;
                o[i] = now.rstd * (now.d[v].get(i) * g[i] - s1 - xh * s2);
                if (dsum) o[i] += now.s[v].get(i);
            }
            store_vec(dx + row * n, c, n, o);
        }
        if (AHEAD)
            now = next;
        else if (row + gridDim.x < rows)
            load(row + gridDim.x, &now);
    }
    float* pr = part + (int64_t)blockIdx.x * 2 * n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * TPR + t) * VN;
        keep_n<VN>(pr, c, n, dg[v]);
        keep_n<VN>(pr + n, c, n, db[v]);
    }
}

// Sums the parts' columns: 64 columns a workgroup, its four waves a quarter of
// the parts each (in order), joined in order.  Columns [0, n) are dgamma's,
// [n, 2n) dbeta's.
template <class W>
__global__ __launch_bounds__(256) void ln_backward_sum(const float* part, int parts, int n, W* dgamma, W* dbeta) {
    __shared__ float buf[4][64];
    const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    const int w = threadIdx.x >> 6;
    const int64_t ld = 2 * (int64_t)n;
    const int p0 = (int)((int64_t)parts * w / 4), p1 = (int)((int64_t)parts * (w + 1) / 4);
    float s = 0.0f;
    if (c < ld) {
        int p = p0;
        for (; p + 8 <= p1; p += 8) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = part[(p + i) * ld + c];
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
        for (; p < p1; ++p) s += part[p * ld + c];
    }
    buf[w][threadIdx.x & 63] = s;
    __syncthreads();
    if (w == 0 && c < ld) {
        const int l = threadIdx.x;
        const float r = buf[0][l] + buf[1][l] + buf[2][l] + buf[3][l];
        if (c < n)
            dgamma[c] = (W)r;
        else if (dbeta)
            dbeta[c - n] = (W)r;
    }
}

#ifndef V_MOST
#define V_MOST (n <= 2048 ? 1024 : 256)
#endif
constexpr int64_t kMaxNorm = 32768;   // elements of a row: 1024 threads of 32

// Workgroups of the backward pass: one part each.
int64_t backward_parts(int64_t rows, int64_t n) {
    const int64_t most = V_MOST;
    return rows < most ? rows : most;
}

// f(threads of a row, elements of a thread).
template <class F>
void by_row_size(int64_t n, F&& f) {
    auto call = [&](auto t, auto e) { f(t, e); };
    if (n <= 512)
        call(std::integral_constant<int, 64>(), std::integral_constant<int, 8>());
    else if (n <= 1024)
        call(std::integral_constant<int, 64>(), std::integral_constant<int, 16>());
    else if (n <= 2048)
        call(std::integral_constant<int, 128>(), std::integral_constant<int, 16>());
    else if (n <= 4096)
        call(std::integral_constant<int, 256>(), std::integral_constant<int, 16>());
    else if (n <= 8192)
        call(std::integral_constant<int, 512>(), std::integral_constant<int, 16>());
    else if (n <= 16384)
        call(std::integral_constant<int, 1024>(), std::integral_constant<int, 16>());
    else
        call(std::integral_constant<int, 1024>(), std::integral_constant<int, 32>());
}

// f(T, W) of the row and parameter types.
template <class F>
void by_types(coc_dtype dt, coc_dtype pdt, F&& f) {
    const bool wide = pdt == COC_F32;
    if (dt == COC_F32)
        f(float(), float());
    else if (dt == COC_F16)
        wide ? f(f16_t(), float()) : f(f16_t(), f16_t());
    else
        wide ? f(bf16_t(), float()) : f(bf16_t(), bf16_t());
}

coc_status check_norm(int64_t rows, int64_t n, coc_dtype dt, coc_dtype pdt) {
    if (!dtype_valid(dt)) return fail(COC_ERR_DTYPE, "unknown dtype %d", (int)dt);
    if (pdt != dt && pdt != COC_F32) return fail(COC_ERR_DTYPE, "gamma and beta have the rows' dtype or fp32");
    const coc_status s = check_matrix(rows, n, "x");
    if (s != COC_OK) return s;
    if (n < 1 || n > kMaxNorm)
        return fail(COC_ERR_SHAPE, "a row has 1 to %lld elements (n=%lld)", (long long)kMaxNorm, (long long)n);
    return COC_OK;
}

}  // namespace
}  // namespace coc

extern "C" {

coc_status coc_layer_norm(const void* x, const void* residual, const void* gamma, const void* beta, void* y,
                          void* sum_out, float* mean, float* rstd, int64_t rows, int64_t n, float eps, coc_dtype dt,
                          coc_dtype param_dt, hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_norm(rows, n, dt, param_dt);
    if (st != COC_OK) return st;
    if (!(eps >= 0.0f)) return fail(COC_ERR_SHAPE, "eps must not be negative");
    if (rows == 0) return COC_OK;
    const int32_t es = (int32_t)elem_size(dt), ps = (int32_t)elem_size(param_dt);
    const int64_t bytes = rows * n * es, stat = rows * 4;
    const Arg args[] = {
        {x, bytes, es, false, "x"},
        {residual, residual ? bytes : 0, es, false, "residual"},
        {gamma, n * ps, ps, false, "gamma"},
        {beta, beta ? n * ps : 0, ps, false, "beta"},
        {y, bytes, es, true, "y"},
        {sum_out, residual ? bytes : 0, es, true, "sum_out"},
        {mean, stat, 4, true, "mean"},
        {rstd, stat, 4, true, "rstd"},
    };
    st = check_args(args, 8);
    if (st != COC_OK) return st;
    by_types(dt, param_dt, [&](auto t, auto w) {
        using T = decltype(t);
        using W = decltype(w);
        by_row_size(n, [&](auto tpr, auto ept) {
            constexpr int TPR = decltype(tpr)::value, EPT = decltype(ept)::value;
            constexpr int threads = TPR == 64 ? 256 : TPR;
            const int64_t grid = ceil_div(rows, threads / TPR);
            ln_forward<T, W, TPR, EPT><<<dim3((uint32_t)grid), dim3(threads), 0, stream>>>(
                (const T*)x, (const T*)residual, (const W*)gamma, (const W*)beta, (T*)y, (T*)sum_out, mean, rstd, rows,
                (int)n, eps);
        });
    });
    return launched("layer norm");
}

size_t coc_layer_norm_backward_workspace_bytes(int64_t rows, int64_t n) {
    if (rows <= 0 || n <= 0 || n > coc::kMaxNorm) return 0;
    return (size_t)(coc::backward_parts(rows, n) * 2 * n * 4);
}

coc_status coc_layer_norm_backward(const void* dy, const void* x, const void* gamma, const float* mean,
                                   const float* rstd, const void* dsum, void* dx, void* dgamma, void* dbeta,
                                   int64_t rows, int64_t n, coc_dtype dt, coc_dtype param_dt, void* ws,
                                   size_t ws_bytes, hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_norm(rows, n, dt, param_dt);
    if (st != COC_OK) return st;
    const int32_t es = (int32_t)elem_size(dt), ps = (int32_t)elem_size(param_dt);
    const int64_t bytes = rows * n * es, stat = rows * 4;
    const size_t need = coc_layer_norm_backward_workspace_bytes(rows, n);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(COC_ERR_WORKSPACE, "layer norm backward needs %zu workspace bytes (got %zu)", need,
                    ws ? ws_bytes : (size_t)0);
    const Arg args[] = {
        {dy, bytes, es, false, "dy"},
        {x, bytes, es, false, "x"},
        {gamma, n * ps, ps, false, "gamma"},
        {mean, stat, 4, false, "mean"},
        {rstd, stat, 4, false, "rstd"},
        {dsum, dsum ? bytes : 0, es, false, "dsum"},
        {dx, bytes, es, true, "dx"},
        {dgamma, n * ps, ps, true, "dgamma"},
        {dbeta, dbeta ? n * ps : 0, ps, true, "dbeta"},
        {ws, (int64_t)need, 4, true, "ws"},
    };
    st = check_args(args, 10);
    if (st != COC_OK) return st;
    const int64_t parts = rows > 0 ? backward_parts(rows, n) : 0;
    if (rows > 0) {
        by_types(dt, param_dt, [&](auto t, auto w) {
            using T = decltype(t);
            using W = decltype(w);
            by_row_size(n, [&](auto tpr, auto ept) {
                constexpr int TPR = decltype(tpr)::value, EPT = decltype(ept)::value;
                ln_backward<T, W, TPR, EPT><<<dim3((uint32_t)parts), dim3(TPR), 0, stream>>>(
                    (const T*)dy, (const T*)x, (const W*)gamma, mean, rstd, (const T*)dsum, (T*)dx, (float*)ws, rows,
                    (int)n);
            });
        });
        st = launched("layer norm backward");
        if (st != COC_OK) return st;
    }
    // without rows the sums are 0
    const dim3 grid((uint32_t)ceil_div(2 * n, 64));
    by_types(param_dt, param_dt, [&](auto w, auto) {
        using W = decltype(w);
        ln_backward_sum<W><<<grid, dim3(256), 0, stream>>>((const float*)ws, (int)parts, (int)n, (W*)dgamma,
                                                           (W*)dbeta);
    });
    return launched("layer norm backward");
}

}  // extern "C"
