// Layer norm, forward and backward, with the residual sum joined in.
#include "row_ops.h"

namespace coc {
namespace {

// The parameters beside a vector of a row, kept as stored.
template <class T, class W, RowKind KIND>
struct Params {
    static constexpr int V = (kVec<T> + kVec<W> - 1) / kVec<W>;
    Packed<W> p[V];
    __device__ __forceinline__ void load(const W* v, const Cols<T, KIND>& col, int n) {
#pragma unroll
        for (int q = 0; q < V; ++q) {
            if constexpr (KIND == kTiny)
                load_raw(v, col.c + q * kVec<W>, n, &p[q]);
            else
                __builtin_memcpy(p[q].w, v + col.c + q * kVec<W>, 16);
        }
    }
    __device__ __forceinline__ float get(int i) const { return p[i / kVec<W>].get(i % kVec<W>); }
    __device__ __forceinline__ void again() {
#pragma unroll
        for (int q = 0; q < V; ++q) repack(p[q]);
    }
};

// Forward.  TPR threads hold one row in registers, EPT elements each, so a row
// is read once: its mean, then the mean of its squared distances from it (two
// sums over registers, which lose nothing where the mean is far from zero),
// then the output.  Bound by memory: 512 x 8192 with a residual (bf16, 33.6 MB)
// 7.3 us, 4.6 TB/s; 16000 x 1001 with one 21 us, 6.0 TB/s; a lone row of 14336
// 3.4 us, which is a launch and two waits.  16 values a thread: a row of 8192
// by 512 threads took 7.2 us, by 256 threads of 32 values 11.5.  Rows past 16384
// take 1024 threads of 32; with binary32 rows or parameters 4 to 32 registers of
// them do not fit (2048 x 32768, bf16: 61 us, 4.4 TB/s; 1024 x 32768, fp32: 104
// us, 2.6).
template <class T, class W, int TPR, int EPT, RowKind KIND>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void ln_forward(
    const T* x, const T* residual, const W* gamma, const W* beta, T* y, T* sum_out, float* mean_out, float* rstd_out,
    int64_t rows, int n, float eps) {
    constexpr int VN = kVec<T>, V = EPT / VN;
    constexpr int RPB = TPR == 64 ? 4 : 1;   // rows per workgroup: several where a wave holds one
    __shared__ float buf[2][TPR / 64];
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (RPB > 1 && row >= rows) return;
    Packed<T> px[V], pr[V];
#pragma unroll
    for (int v = 0; v < V; ++v) Cols<T, KIND>(v * TPR + t, n).load(x + row * n, n, &px[v]);
    if (residual) {
#pragma unroll
        for (int v = 0; v < V; ++v) Cols<T, KIND>(v * TPR + t, n).load(residual + row * n, n, &pr[v]);
    }
    Params<T, W, KIND> g[V], b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Cols<T, KIND> col(v * TPR + t, n);
        g[v].load(gamma, col, n);
        if (beta) b[v].load(beta, col, n);
    }
    float h[V][VN], s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Cols<T, KIND> col(v * TPR + t, n);
        if (residual) {
#pragma unroll
            for (int i = 0; i < VN; ++i) h[v][i] = px[v].get(i) + pr[v].get(i);
            px[v].set(h[v]);   // the sum as stored
            col.store(sum_out + row * n, n, px[v]);
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            h[v][i] = px[v].get(i);
            s += col.has(i, n) ? h[v][i] : 0.0f;
        }
    }
    const float mean = (TPR == 64 ? lanes_sum<64>(s) : group_sum<TPR>(s, buf[0])) / (float)n;
    float q = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Cols<T, KIND> col(v * TPR + t, n);
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            h[v][i] -= mean;
            const float d = col.has(i, n) ? h[v][i] : 0.0f;
            q += d * d;
        }
    }
    const float var = (TPR == 64 ? lanes_sum<64>(q) : group_sum<TPR>(q, buf[1])) / (float)n;
    const float rstd = 1.0f / sqrtf(var + eps);
    if (t == 0) {
        mean_out[row] = mean;
        rstd_out[row] = rstd;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < VN; ++i) h[v][i] = h[v][i] * rstd * g[v].get(i) + (beta ? b[v].get(i) : 0.0f);
        Packed<T> o;
        o.set(h[v]);
        Cols<T, KIND>(v * TPR + t, n).store(y + row * n, n, o);
    }
}

constexpr int kNormThreads = 512;   // of a backward workgroup, or a row's where that is more

// Backward.  xh = (x - mean) rstd, g = dy gamma:
//   dx = rstd (g - avg(g) - xh avg(g xh)) + dsum,  dgamma = sum dy xh,  dbeta = sum dy.
// TPR threads take a row, a thread always the same columns, so the columns'
// sums stay in its registers over all its rows.  A workgroup's groups of TPR
// threads add theirs up at the end, and it leaves them as row b of `part`
// (grid x 2 x n); ln_backward_sum adds those rows in order.  While a row is
// summed the next one is on its way, into the other of two sets of registers (a
// copy between them would wait for it).  All groups make as many steps; a row
// past the last is the last one again, counted nowhere.  Bound by memory and
// the parts: 2048 x 14336 with dsum (bf16, 235 MB and 59 MB of parts) 50.8 us,
// 4.6 TB/s without the parts; without the second register set 87.  1024 threads have
// 128 registers each, too few for 16 binary32 values and their sums, or for 32 of any
// type: 28 to 43 and 68 to 188 do not fit (1500 x 14336, fp32: 87 us, 3.0 TB/s; 2048 x
// 32768, bf16: 224 us, 1.8).
template <class T, class W, int TPR, int EPT, RowKind KIND>
__global__ __launch_bounds__(TPR < kNormThreads ? kNormThreads : TPR) void ln_backward(
    const T* dy, const T* x, const W* gamma, const float* mean_in, const float* rstd_in, const T* dsum, T* dx,
    float* part, int64_t rows, int n) {
    constexpr int VN = kVec<T>, V = EPT / VN;
    constexpr int THREADS = TPR < kNormThreads ? kNormThreads : TPR, GROUPS = THREADS / TPR;
    constexpr int LEFT = GROUPS > 1 ? GROUPS / 2 : 0;   // groups whose sums go through LDS at once
    __shared__ float buf[2][2][THREADS / 64];
    __shared__ float sums[LEFT ? LEFT * TPR * VN * 2 : 1];
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    float dg[V][VN], db[V][VN];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < VN; ++i) dg[v][i] = db[v][i] = 0.0f;
    // gamma stays in registers where they suffice, or comes from the cache each time
    constexpr bool KEEP = TPR < 1024 || EPT * (int)(sizeof(T) + sizeof(W)) <= 64;
    Params<T, W, KIND> ga[V];
#pragma unroll
    for (int v = 0; v < V; ++v) ga[v].load(gamma, Cols<T, KIND>(v * TPR + t, n), n);
    auto gamma_again = [&](int v) {
        if constexpr (KEEP)
            ga[v].again();
        else
            ga[v].load(gamma, Cols<T, KIND>(v * TPR + t, n), n);
    };
    constexpr bool AHEAD = TPR < 1024 || EPT * (int)sizeof(T) <= 32;   // two sets of a row fit in the registers
    struct Row {
        Packed<T> x[V], d[V];
        float mean, rstd;
    };
    auto load = [&](int64_t row, Row& r) {
        r.mean = mean_in[row];
        r.rstd = rstd_in[row];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols<T, KIND> col(v * TPR + t, n);
            col.load(x + row * n, n, &r.x[v]);
            col.load(dy + row * n, n, &r.d[v]);
        }
    };
    auto take = [&](int64_t at, Row& r, int flip) {
        const bool live = at < rows;
        const int64_t row = live ? at : rows - 1;
        Packed<T> sum[V];
        if (AHEAD && dsum) {
#pragma unroll
            for (int v = 0; v < V; ++v) Cols<T, KIND>(v * TPR + t, n).load(dsum + row * n, n, &sum[v]);
        }
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols<T, KIND> col(v * TPR + t, n);
            gamma_again(v);
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                const float d = live && col.has(i, n) ? r.d[v].get(i) : 0.0f, xh = (r.x[v].get(i) - r.mean) * r.rstd;
                dg[v][i] += d * xh;
                db[v][i] += d;
                // added here, or d and xh would be kept beyond the barrier for it
                asm("" : "+v"(dg[v][i]), "+v"(db[v][i]));
                s1 += d * ga[v].get(i);
                s2 += d * ga[v].get(i) * xh;
            }
        }
        s1 = lanes_sum<64>(s1);
        s2 = lanes_sum<64>(s2);
        if constexpr (TPR > 64) {
            // two buffers in turn: one barrier a row
            if ((t & 63) == 0) {
                buf[flip][0][threadIdx.x >> 6] = s1;
                buf[flip][1][threadIdx.x >> 6] = s2;
            }
            __syncthreads();
            const int w0 = group * (TPR / 64);
            s1 = buf[flip][0][w0];
            s2 = buf[flip][1][w0];
#pragma unroll
            for (int w = 1; w < TPR / 64; ++w) {
                s1 += buf[flip][0][w0 + w];
                s2 += buf[flip][1][w0 + w];
            }
        }
        s1 /= (float)n;
        s2 /= (float)n;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float o[VN];
            if (!AHEAD && dsum) Cols<T, KIND>(v * TPR + t, n).load(dsum + row * n, n, &sum[v]);
            repack(r.x[v]);
            repack(r.d[v]);
            gamma_again(v);
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                const float xh = (r.x[v].get(i) - r.mean) * r.rstd;
                o[i] = r.rstd * (r.d[v].get(i) * ga[v].get(i) - s1 - xh * s2);
                if (dsum) o[i] += sum[v].get(i);
            }
            Packed<T> p;
            p.set(o);
            if (live) Cols<T, KIND>(v * TPR + t, n).store(dx + row * n, n, p);
        }
    };
    Row a, b;
    const int64_t step = (int64_t)gridDim.x * GROUPS;
    int64_t row = (int64_t)blockIdx.x * GROUPS + group;
    auto within = [&](int64_t r) { return r < rows ? r : rows - 1; };
    if constexpr (AHEAD) {
        load(within(row), a);
        for (int64_t first = blockIdx.x * GROUPS; first < rows;) {   // the same for all groups
            load(within(row + step), b);
            take(row, a, 0);
            row += step;
            first += step;
            if (first >= rows) break;
            load(within(row + step), a);
            take(row, b, 1);
            row += step;
            first += step;
        }
    } else {
        for (int flip = 0; row < rows; row += step, flip ^= 1) {
            load(row, a);
            take(row, a, flip);
        }
    }
    // group g's sums onto group g - half's, halving; a vector at a time
#pragma unroll
    for (int half = LEFT; half > 0; half >>= 1)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float* s = sums + (group % half * TPR + t) * VN * 2;
            __syncthreads();
            if (group >= half && group < 2 * half) {
#pragma unroll
                for (int i = 0; i < VN; ++i) {
                    s[i] = dg[v][i];
                    s[VN + i] = db[v][i];
                }
            }
            __syncthreads();
            if (group < half) {
#pragma unroll
                for (int i = 0; i < VN; ++i) {
                    dg[v][i] += s[i];
                    db[v][i] += s[VN + i];
                }
            }
        }
    if (group > 0) return;
    float* pr = part + (int64_t)blockIdx.x * 2 * n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Cols<T, KIND> col(v * TPR + t, n);
        if (KIND == kTiny || col.skip == 0) {
            keep_n<VN>(pr, col.c, n, dg[v]);
            keep_n<VN>(pr + n, col.c, n, db[v]);
        } else if (col.skip < VN) {
#pragma unroll
            for (int i = 0; i < VN; ++i)
                if (col.has(i, n)) {
                    pr[col.c + i] = dg[v][i];
                    pr[n + col.c + i] = db[v][i];
                }
        }
    }
}

// Sums the parts' columns: 64 columns a workgroup, its four waves a quarter of
// the parts each (in order), joined in order.  Columns [0, n) are dgamma's,
// [n, 2n) dbeta's.  256 parts of 28672 columns, just written: 6 us, 4.9 TB/s.
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

constexpr int64_t kMaxNorm = 32768;   // elements of a row: 1024 threads of 32

// Workgroups of the backward pass, one part each: a CU's worth, since the parts
// are written and read again (4096 x 8192 with dsum, bf16: 256 workgroups 61 us, 512
// 68, 128 91; 16000 x 1001: 28, 33, 36).
constexpr int64_t kMostParts = 256;
int64_t backward_parts(int64_t rows, int64_t n) {
    const int64_t groups = n <= 1024 ? 8 : n <= 2048 ? 4 : n <= 4096 ? 2 : 1;   // rows at a time
    const int64_t want = (rows + groups - 1) / groups;
    return want < kMostParts ? want : kMostParts;
}

template <RowKind K>
using Kind = std::integral_constant<RowKind, K>;

// f(threads of a row, elements of a thread, kind of the row).
template <class T, class F>
void by_row_size(int64_t n, F&& f) {
    auto call = [&](auto t, auto e) { n % kVec<T> == 0 ? f(t, e, Kind<kWhole>()) : f(t, e, Kind<kRagged>()); };
    if (n < kVec<T>)
        f(std::integral_constant<int, 64>(), std::integral_constant<int, 8>(), Kind<kTiny>());
    else if (n <= 512)
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
        by_row_size<T>(n, [&](auto tpr, auto ept, auto kind) {
            constexpr int TPR = decltype(tpr)::value, EPT = decltype(ept)::value;
            constexpr int threads = TPR == 64 ? 256 : TPR;
            const int64_t grid = ceil_div(rows, threads / TPR);
            ln_forward<T, W, TPR, EPT, decltype(kind)::value><<<dim3((uint32_t)grid), dim3(threads), 0, stream>>>(
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
            by_row_size<T>(n, [&](auto tpr, auto ept, auto kind) {
                constexpr int TPR = decltype(tpr)::value, EPT = decltype(ept)::value;
                ln_backward<T, W, TPR, EPT, decltype(kind)::value><<<dim3((uint32_t)parts), dim3(TPR < kNormThreads ? kNormThreads : TPR), 0, stream>>>(
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
