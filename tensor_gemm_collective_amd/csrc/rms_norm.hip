// Root-mean-square norm, forward and backward, with the residual sum joined in
// and an output in 8 bits.
#include "fp8.h"

namespace coc {
namespace {

// A row vector's parameters, kept as stored.
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

// Forward: h = x (+ residual, rounded to the rows' type), rstd = 1 / sqrt(mean h^2 + eps),
// y = h rstd gamma.  TPR threads hold one row in registers, EPT elements each, so
// it is read once.  FP8: the row goes out in 8 bits (fp8.h); a block's 128 columns
// lie in 16 (32: binary32 rows) neighbouring lanes, so its largest value takes
// four (five) lane steps and nothing is written before it is known.  Bound by
// memory: 4096 x 8192 with a residual into 8 bits (bf16, 236 MB) 42.5 us, 5.6 TB/s;
// a lone row of 8192 2.9 us, a launch and two waits.  16 values a thread; binary32
// rows past 16384 columns spill 4 to 8 of its 128 registers.
template <class T, class W, int TPR, int EPT, RowKind KIND, bool FP8>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void rms_forward(const T* x, const T* residual, const W* gamma,
                                                                     T* y, uint8_t* q, float* scales, T* sum_out,
                                                                     float* rstd_out, int64_t rows, int n, float eps) {
    constexpr int VN = kVec<T>, V = EPT / VN;
    constexpr int RPB = TPR == 64 ? 4 : 1;   // rows per workgroup: several where a wave holds one
    __shared__ float buf[TPR / 64];
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
    Params<T, W, KIND> g[V];
#pragma unroll
    for (int v = 0; v < V; ++v) g[v].load(gamma, Cols<T, KIND>(v * TPR + t, n), n);
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Cols<T, KIND> col(v * TPR + t, n);
        if (residual) {
            float h[VN];
#pragma unroll
            for (int i = 0; i < VN; ++i) h[i] = px[v].get(i) + pr[v].get(i);
            px[v].set(h);   // the sum as stored
            col.store(sum_out + row * n, n, px[v]);
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const float h = col.has(i, n) ? px[v].get(i) : 0.0f;
            s += h * h;
        }
    }
    const float mean = (TPR == 64 ? lanes_sum<64>(s) : group_sum<TPR>(s, buf)) / (float)n;
    const float rstd = 1.0f / sqrtf(mean + eps);
    if (t == 0) rstd_out[row] = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Cols<T, KIND> col(v * TPR + t, n);
        float o[VN];
#pragma unroll
        for (int i = 0; i < VN; ++i) o[i] = px[v].get(i) * rstd * g[v].get(i);
        if constexpr (FP8) {
            constexpr int LANES = kScaleBlock / VN;
            uint32_t top = 0;
            if (col.skip == 0) {
#pragma unroll
                for (int i = 0; i < VN; ++i) top = max(top, magnitude(o[i]));
            }
            const Fp8Scale f = fp8_scale(lanes_max<LANES>(top));
            if (col.skip == 0) {
                store_fp8<VN>(q + row * n + col.c, o, f.inverse);
                if (t % LANES == 0) scales[(int64_t)(col.c / kScaleBlock) * rows + row] = f.scale;
            }
        } else {
            Packed<T> p;
            p.set(o);
            col.store(y + row * n, n, p);
        }
    }
}

constexpr int kNormThreads = 512;   // of a backward workgroup, or a row's where that is more
constexpr int kSumThreads = 512;

// Backward.  xh = x rstd, g = dy gamma:
//   dx = rstd (g - xh avg(g xh)) + dsum,  dgamma = sum over rows of dy xh.
// TPR threads take a row, a thread always the same columns, so the columns' sums
// stay in its registers over all its rows; a workgroup leaves its own as row b of
// `part` (grid x n), which rms_backward_sum adds up in order, or a lone one in dgamma.  While a row is
// summed the next one is on its way into the other of two sets of registers.  All
// groups make as many steps; a row past the last is the last one again, counted
// nowhere.  Bound by memory and the parts: 2048 x 8192 with dsum (bf16, 134 MB and
// 8.4 MB of parts) 28.5 us, 5.0 TB/s, and 4 to 5 to add up the parts.  Two rows at a
// time in 1024 threads gained nothing there (30.2 against 30.5 us in all) and spilled
// binary32 rows (1500 x 7000: 62 against 37 us); rows past 16384 columns spill 9 (16
// bits) or 92 of 128 registers.
template <class T, class W, int TPR, int EPT, RowKind KIND>
__global__ __launch_bounds__(TPR < kNormThreads ? kNormThreads : TPR) void rms_backward(
    const T* dy, const T* x, const W* gamma, const float* rstd_in, const T* dsum, T* dx, float* part, W* dgamma,
    int64_t rows, int n) {
    constexpr int VN = kVec<T>, V = EPT / VN;
    constexpr int THREADS = TPR < kNormThreads ? kNormThreads : TPR, GROUPS = THREADS / TPR;
    constexpr int LEFT = GROUPS > 1 ? GROUPS / 2 : 0;   // groups whose sums go through LDS at once
    __shared__ float buf[2][THREADS / 64];
    __shared__ float sums[LEFT ? LEFT * TPR * VN : 1];
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    float dg[V][VN];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < VN; ++i) dg[v][i] = 0.0f;
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
        float rstd;
    };
    auto load = [&](int64_t row, Row& r) {
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
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols<T, KIND> col(v * TPR + t, n);
            gamma_again(v);
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                const float d = live && col.has(i, n) ? r.d[v].get(i) : 0.0f, xh = r.x[v].get(i) * r.rstd;
                dg[v][i] += d * xh;
                // added here, or d and xh would be kept beyond the barrier for it
                asm("" : "+v"(dg[v][i]));
                s += d * ga[v].get(i) * xh;
            }
        }
        s = lanes_sum<64>(s);
        if constexpr (TPR > 64) {
            // two buffers in turn: one barrier a row
            if ((t & 63) == 0) buf[flip][threadIdx.x >> 6] = s;
            __syncthreads();
            const int w0 = group * (TPR / 64);
            s = buf[flip][w0];
#pragma unroll
            for (int w = 1; w < TPR / 64; ++w) s += buf[flip][w0 + w];
        }
        s /= (float)n;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float o[VN];
            if (!AHEAD && dsum) Cols<T, KIND>(v * TPR + t, n).load(dsum + row * n, n, &sum[v]);
            repack(r.x[v]);
            repack(r.d[v]);
            gamma_again(v);
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                const float xh = r.x[v].get(i) * r.rstd;
                o[i] = r.rstd * (r.d[v].get(i) * ga[v].get(i) - xh * s);
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
        for (int flip = 0; row < rows; row += step, flip ^= 1) {   // one group: the same rows for all threads
            load(row, a);
            take(row, a, flip);
        }
    }
    // group g's sums onto group g - half's, halving; a vector at a time
#pragma unroll
    for (int half = LEFT; half > 0; half >>= 1)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float* s = sums + (group % half * TPR + t) * VN;
            __syncthreads();
            if (group >= half && group < 2 * half) {
#pragma unroll
                for (int i = 0; i < VN; ++i) s[i] = dg[v][i];
            }
            __syncthreads();
            if (group < half) {
#pragma unroll
                for (int i = 0; i < VN; ++i) dg[v][i] += s[i];
            }
        }
    if (group > 0) return;
    auto leave = [&](auto* to) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols<T, KIND> col(v * TPR + t, n);
            if (KIND == kTiny || col.skip == 0) {
                keep_n<VN>(to, col.c, n, dg[v]);
            } else if (col.skip < VN) {
#pragma unroll
                for (int i = 0; i < VN; ++i)
                    if (col.has(i, n)) to[col.c + i] = (std::remove_pointer_t<decltype(to)>)dg[v][i];
            }
        }
    };
    if (gridDim.x == 1)
        leave(dgamma);
    else
        leave(part + (int64_t)blockIdx.x * n);
}

// Sums the parts' columns: 32 columns a workgroup, its 16 half-waves a sixteenth of the
// parts each (in order), joined in order.  (8 half-waves: 0.3 to 0.6 us more at 256 parts,
// 32: the same.)
template <class W>
__global__ __launch_bounds__(kSumThreads) void rms_backward_sum(const float* part, int parts, int n, W* dgamma) {
    constexpr int COLS = 32, RUNS = kSumThreads / COLS;
    __shared__ float buf[RUNS][COLS];
    const int c = (int)blockIdx.x * COLS + (threadIdx.x % COLS);
    const int w = threadIdx.x / COLS;
    const int p0 = parts * w / RUNS, p1 = parts * (w + 1) / RUNS;
    float s = 0.0f;
    if (c < n) {
        int p = p0;
        for (; p + 8 <= p1; p += 8) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = part[(int64_t)(p + i) * n + c];
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
        for (; p < p1; ++p) s += part[(int64_t)p * n + c];
    }
    buf[w][threadIdx.x % COLS] = s;
    __syncthreads();
    if (w == 0 && c < n) {
        float r = buf[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < RUNS; ++i) r += buf[i][threadIdx.x];
        dgamma[c] = (W)r;
    }
}

constexpr int64_t kMaxNorm = 32768;   // elements of a row: 1024 threads of 32

// Workgroups of the backward pass, one part each: a CU's worth, since the parts
// are written and read again (2048 x 8192 with dsum: 256 workgroups 30.5 us, 512 32.1,
// 128 36).  Few rows take one, which needs no second kernel nor a workspace: up to four a
// group of threads (16 x 1148 10.5 us with the host's part, 8.8 in a graph; the two kernels 14.9
// and 6.9; six a group would take 11.4 in a graph), two where a row takes all of a
// workgroup of 1024 threads (4 x 14336, binary32: 14.8 and 15.4 against 15.0 and 8.0).
constexpr int64_t kMostParts = 256;
int64_t backward_parts(int64_t rows, int64_t n) {
    const int64_t groups = n <= 1024 ? 8 : n <= 2048 ? 4 : n <= 4096 ? 2 : 1;   // rows at a time
    const int64_t want = (rows + groups - 1) / groups;
    return want <= (n <= 8192 ? 4 : 2) ? 1 : want < kMostParts ? want : kMostParts;
}

template <RowKind K>
using Kind = std::integral_constant<RowKind, K>;

// f(threads of a row, elements of a thread, kind of the row).
template <class T, bool WHOLE, class F>
void by_row_size(int64_t n, F&& f) {
    auto call = [&](auto t, auto e) {
        if constexpr (WHOLE)
            f(t, e, Kind<kWhole>());
        else
            n % kVec<T> == 0 ? f(t, e, Kind<kWhole>()) : f(t, e, Kind<kRagged>());
    };
    if (!WHOLE && n < kVec<T>) {
        if constexpr (!WHOLE) f(std::integral_constant<int, 64>(), std::integral_constant<int, 8>(), Kind<kTiny>());
    } else if (n <= 512)
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
    if (pdt != dt && pdt != COC_F32) return fail(COC_ERR_DTYPE, "gamma has the rows' dtype or fp32");
    const coc_status s = check_matrix(rows, n, "x");
    if (s != COC_OK) return s;
    if (n < 1 || n > kMaxNorm)
        return fail(COC_ERR_SHAPE, "a row has 1 to %lld elements (n=%lld)", (long long)kMaxNorm, (long long)n);
    return COC_OK;
}

coc_status forward(const void* x, const void* residual, const void* gamma, void* y, void* q, float* scales,
                   void* sum_out, float* rstd, int64_t rows, int64_t n, float eps, coc_dtype dt, coc_dtype param_dt,
                   bool fp8, hipStream_t stream) {
    clear_error();
    coc_status st = check_norm(rows, n, dt, param_dt);
    if (st != COC_OK) return st;
    if (fp8 && n % 16 != 0) return fail(COC_ERR_SHAPE, "rows in 8 bits have a multiple of 16 elements (n=%lld)", (long long)n);
    if (!(eps >= 0.0f)) return fail(COC_ERR_SHAPE, "eps must not be negative");
    if (rows == 0) return COC_OK;
    const int32_t es = (int32_t)elem_size(dt), ps = (int32_t)elem_size(param_dt);
    const int64_t bytes = rows * n * es;
    const Arg args[] = {
        {x, bytes, es, false, "x"},
        {residual, residual ? bytes : 0, es, false, "residual"},
        {gamma, n * ps, ps, false, "gamma"},
        {y, fp8 ? 0 : bytes, es, true, "y"},
        {q, fp8 ? rows * n : 0, 16, true, "q"},
        {scales, fp8 ? ceil_div(n, kScaleBlock) * rows * 4 : 0, 4, true, "scales"},
        {sum_out, residual ? bytes : 0, es, true, "sum_out"},
        {rstd, rows * 4, 4, true, "rstd"},
    };
    st = check_args(args, 8);
    if (st != COC_OK) return st;
    by_types(dt, param_dt, [&](auto t, auto w) {
        using T = decltype(t);
        using W = decltype(w);
        auto go = [&](auto eight) {
            constexpr bool FP8 = decltype(eight)::value;
            by_row_size<T, FP8>(n, [&](auto tpr, auto ept, auto kind) {
                constexpr int TPR = decltype(tpr)::value, EPT = decltype(ept)::value;
                constexpr int threads = TPR == 64 ? 256 : TPR;
                const int64_t grid = ceil_div(rows, threads / TPR);
                rms_forward<T, W, TPR, EPT, decltype(kind)::value, FP8>
                    <<<dim3((uint32_t)grid), dim3(threads), 0, stream>>>((const T*)x, (const T*)residual, (const W*)gamma,
                                                                         (T*)y, (uint8_t*)q, scales, (T*)sum_out, rstd,
                                                                         rows, (int)n, eps);
            });
        };
        fp8 ? go(std::true_type()) : go(std::false_type());
    });
    return launched("rms norm");
}

}  // namespace
}  // namespace coc

extern "C" {

coc_status coc_rms_norm(const void* x, const void* residual, const void* gamma, void* y, void* sum_out, float* rstd,
                        int64_t rows, int64_t n, float eps, coc_dtype dt, coc_dtype param_dt, hipStream_t stream) {
    return coc::forward(x, residual, gamma, y, nullptr, nullptr, sum_out, rstd, rows, n, eps, dt, param_dt, false,
                        stream);
}

coc_status coc_rms_norm_fp8(const void* x, const void* residual, const void* gamma, void* q, float* scales,
                            void* sum_out, float* rstd, int64_t rows, int64_t n, float eps, coc_dtype dt,
                            coc_dtype param_dt, hipStream_t stream) {
    return coc::forward(x, residual, gamma, nullptr, q, scales, sum_out, rstd, rows, n, eps, dt, param_dt, true,
                        stream);
}

size_t coc_rms_norm_backward_workspace_bytes(int64_t rows, int64_t n) {
    if (rows <= 0 || n <= 0 || n > coc::kMaxNorm) return 0;
    const int64_t parts = coc::backward_parts(rows, n);
    return parts > 1 ? (size_t)(parts * n * 4) : 0;
}

coc_status coc_rms_norm_backward(const void* dy, const void* x, const void* gamma, const float* rstd, const void* dsum,
                                 void* dx, void* dgamma, int64_t rows, int64_t n, coc_dtype dt, coc_dtype param_dt,
                                 void* ws, size_t ws_bytes, hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_norm(rows, n, dt, param_dt);
    if (st != COC_OK) return st;
    const int32_t es = (int32_t)elem_size(dt), ps = (int32_t)elem_size(param_dt);
    const int64_t bytes = rows * n * es;
    const size_t need = coc_rms_norm_backward_workspace_bytes(rows, n);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(COC_ERR_WORKSPACE, "rms norm backward needs %zu workspace bytes (got %zu)", need,
                    ws ? ws_bytes : (size_t)0);
    const Arg args[] = {
        {dy, bytes, es, false, "dy"},
        {x, bytes, es, false, "x"},
        {gamma, n * ps, ps, false, "gamma"},
        {rstd, rows * 4, 4, false, "rstd"},
        {dsum, dsum ? bytes : 0, es, false, "dsum"},
        {dx, bytes, es, true, "dx"},
        {dgamma, n * ps, ps, true, "dgamma"},
        {ws, (int64_t)need, 4, true, "ws"},
    };
    st = check_args(args, 8);
    if (st != COC_OK) return st;
    const int64_t parts = rows > 0 ? backward_parts(rows, n) : 0;
    if (rows > 0) {
        by_types(dt, param_dt, [&](auto t, auto w) {
            using T = decltype(t);
            using W = decltype(w);
            by_row_size<T, false>(n, [&](auto tpr, auto ept, auto kind) {
                constexpr int TPR = decltype(tpr)::value, EPT = decltype(ept)::value;
                rms_backward<T, W, TPR, EPT, decltype(kind)::value>
                    <<<dim3((uint32_t)parts), dim3(TPR < kNormThreads ? kNormThreads : TPR), 0, stream>>>(
                        (const T*)dy, (const T*)x, (const W*)gamma, rstd, (const T*)dsum, (T*)dx, (float*)ws,
                        (W*)dgamma, rows, (int)n);
            });
        });
        st = launched("rms norm backward");
        if (st != COC_OK || parts == 1) return st;
    }
    // without rows the sums are 0
    by_types(param_dt, param_dt, [&](auto w, auto) {
        using W = decltype(w);
        rms_backward_sum<W><<<dim3((uint32_t)ceil_div(n, 32)), dim3(kSumThreads), 0, stream>>>((const float*)ws, (int)parts,
                                                                                      (int)n, (W*)dgamma);
    });
    return launched("rms norm backward");
}

}  // extern "C"
