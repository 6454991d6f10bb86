// The gated block's elementwise parts, act(gate) * up and its gradient, and the
// quantisation of rows and weights to 8 bits.
#include "fp8.h"
#include "gated_act.h"

namespace coc {
namespace {

// Row r of a rows x 2f matrix: f gate values, then f up values.  A thread takes the
// vector `col` of one row's f columns; threads are numbered through the rows.
template <class T, RowKind KIND>
struct Place {
    int64_t row;
    Cols<T, KIND> col;
    __device__ __forceinline__ Place(uint32_t i, uint32_t per_row, int f)
        : row(i / per_row), col((int)(i - (uint32_t)row * per_row), f) {}
};

// h = act(g) u, rounded once.  Memory bound: two reads and a write, a vector a thread.
template <class T, int ACT, RowKind KIND>
__global__ __launch_bounds__(256) void gated_forward(const T* gate_up, T* h, uint32_t vectors, uint32_t per_row,
                                                     int f) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    if (i >= vectors) return;
    const Place<T, KIND> at(i, per_row, f);
    const T* g = gate_up + at.row * 2 * f;
    Packed<T> pg, pu, o;
    at.col.load(g, f, &pg);
    at.col.load(g + f, f, &pu);
    float v[kVec<T>];
#pragma unroll
    for (int k = 0; k < kVec<T>; ++k) v[k] = act_of<T, ACT>(pg.get(k)) * pu.get(k);
    o.set(v);
    at.col.store(h + at.row * f, f, o);
}

// dg = dh u act'(g), du = dh act(g).  Memory bound, three reads and two writes: 4096 x 3584
// (bf16, 147 MB) 21.8 us by itself, 28 (5.2 TB/s) in front of the products of gated_ffn's gradient.
template <class T, int ACT, RowKind KIND>
__global__ __launch_bounds__(256) void gated_backward(const T* dh, const T* gate_up, T* dgate_up, uint32_t vectors,
                                                      uint32_t per_row, int f) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    if (i >= vectors) return;
    const Place<T, KIND> at(i, per_row, f);
    const T* g = gate_up + at.row * 2 * f;
    T* dg = dgate_up + at.row * 2 * f;
    Packed<T> pg, pu, pd, o;
    at.col.load(g, f, &pg);
    at.col.load(g + f, f, &pu);
    at.col.load(dh + at.row * f, f, &pd);
    float vg[kVec<T>], vu[kVec<T>];
#pragma unroll
    for (int k = 0; k < kVec<T>; ++k) {
        float value, slope;
        act_and_slope_of<T, ACT>(pg.get(k), &value, &slope);
        vg[k] = pd.get(k) * pu.get(k) * slope;
        vu[k] = pd.get(k) * value;
    }
    o.set(vg);
    at.col.store(dg, f, o);
    o.set(vu);
    at.col.store(dg + f, f, o);
}

// Rows to 8 bits with a scale for each 128 of a row (fp8.h): of x (rows x n), or
// ACT >= 0: of act(g) u, x being rows x 2n.  A block's columns lie in 16 (32:
// binary32) neighbouring lanes; a workgroup takes one column block of 16 (8) rows, so
// that its scales are neighbours in memory.  n is a multiple of 16.  Memory bound: act(g) u
// of 4096 x 3584 (bf16, 74 MB) 12.9 us, 5.7 TB/s.
template <class T, int ACT>
__global__ __launch_bounds__(256) void quantize_rows(const T* x, uint8_t* q, float* scales, int64_t rows, int n,
                                                     int blocks) {
    constexpr int VN = kVec<T>, LANES = kScaleBlock / VN, RPB = 256 / LANES;
    const int block = blockIdx.x % (uint32_t)blocks;
    const int64_t row = (int64_t)(blockIdx.x / (uint32_t)blocks) * RPB + threadIdx.x / LANES;
    const int c = block * kScaleBlock + threadIdx.x % LANES * VN;
    if (row >= rows) return;
    float v[VN];
    uint32_t top = 0;
    if (c < n) {
        Packed<T> p;
        if constexpr (ACT < 0) {
            __builtin_memcpy(p.w, x + row * n + c, 16);
#pragma unroll
            for (int k = 0; k < VN; ++k) v[k] = p.get(k);
        } else {
            Packed<T> u;
            __builtin_memcpy(p.w, x + row * 2 * n + c, 16);
            __builtin_memcpy(u.w, x + row * 2 * n + n + c, 16);
#pragma unroll
            for (int k = 0; k < VN; ++k) v[k] = act_value<ACT>(p.get(k)) * u.get(k);
        }
#pragma unroll
        for (int k = 0; k < VN; ++k) top = max(top, magnitude(v[k]));
    }
    const Fp8Scale s = fp8_scale(lanes_max<LANES>(top));
    if (c >= n) return;
    store_fp8<VN>(q + row * n + c, v, s.inverse);
    if (threadIdx.x % LANES == 0) scales[block * rows + row] = s.scale;
}

// A 128 x 128 block of x a workgroup, held in registers, so that x is read once.  Memory
// bound: 7168 x 8192 (bf16, 176 MB) 31.7 us, 5.6 TB/s.
template <class T>
__global__ __launch_bounds__(256) void quantize_blocks(const T* x, uint8_t* q, float* scales, int64_t rows, int n,
                                                       int blocks) {
    constexpr int VN = kVec<T>, LANES = kScaleBlock / VN, RPB = 256 / LANES, V = kScaleBlock / RPB;
    __shared__ uint32_t buf[4];
    const int block = blockIdx.x % (uint32_t)blocks;
    const int64_t row0 = (int64_t)(blockIdx.x / (uint32_t)blocks) * kScaleBlock;
    const int c = block * kScaleBlock + threadIdx.x % LANES * VN, r = threadIdx.x / LANES;
    Packed<T> p[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        // past the end: what is there already, counted again
        const int64_t row = min(row0 + i * RPB + r, rows - 1);
        __builtin_memcpy(p[i].w, x + row * n + min(c, n - VN), 16);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < VN; ++k) top = max(top, magnitude(p[i].get(k)));
    top = lanes_max<64>(top);
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = top;
    __syncthreads();
    const Fp8Scale s = fp8_scale(max(max(buf[0], buf[1]), max(buf[2], buf[3])));
    if (threadIdx.x == 0) scales[blockIdx.x] = s.scale;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t row = row0 + i * RPB + r;
        float v[VN];
#pragma unroll
        for (int k = 0; k < VN; ++k) v[k] = p[i].get(k);
        if (row < rows && c < n) store_fp8<VN>(q + row * n + c, v, s.inverse);
    }
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

// f(kind of a row of n elements of T).
template <class T, class F>
void by_kind(int64_t n, F&& f) {
    if (n < kVec<T>)
        f(std::integral_constant<RowKind, kTiny>());
    else if (n % kVec<T> == 0)
        f(std::integral_constant<RowKind, kWhole>());
    else
        f(std::integral_constant<RowKind, kRagged>());
}

coc_status check_gated(int64_t rows, int64_t f, coc_act act, coc_dtype dt, bool fp8) {
    if (!dtype_valid(dt)) return fail(COC_ERR_DTYPE, "unknown dtype %d", (int)dt);
    if (act != COC_ACT_SILU && act != COC_ACT_GELU) return fail(COC_ERR_DTYPE, "unknown activation %d", (int)act);
    if (f < 1 || f >= int64_t(1) << 29) return fail(COC_ERR_SHAPE, "f is 1 to 2^29 - 1 (f=%lld)", (long long)f);
    if (fp8 && f % 16 != 0) return fail(COC_ERR_SHAPE, "rows in 8 bits have a multiple of 16 elements (n=%lld)", (long long)f);
    return check_matrix(rows, 2 * f, "gate_up");
}

// x (rows x n, or rows x 2n with an activation) in 8 bits by rows.
template <int ACT>
void launch_quantize_rows(const void* x, void* q, float* scales, int64_t rows, int64_t n, coc_dtype dt,
                          hipStream_t stream) {
    by_type(dt, [&](auto t) {
        using T = decltype(t);
        constexpr int RPB = 256 / (kScaleBlock / kVec<T>);
        const int64_t blocks = ceil_div(n, kScaleBlock);
        quantize_rows<T, ACT><<<dim3((uint32_t)(ceil_div(rows, RPB) * blocks)), dim3(256), 0, stream>>>(
            (const T*)x, (uint8_t*)q, scales, rows, (int)n, (int)blocks);
    });
}

}  // namespace

void launch_gated_act_backward(const void* dh, const void* gate_up, void* dgate_up, int64_t rows, int64_t f,
                               coc_act act, coc_dtype dt, hipStream_t stream) {
    by_type(dt, [&](auto t) {
        using T = decltype(t);
        by_act(act, [&](auto a) {
            by_kind<T>(f, [&](auto kind) {
                const int64_t per_row = ceil_div(f, kVec<T>), vectors = rows * per_row;
                gated_backward<T, decltype(a)::value, decltype(kind)::value>
                    <<<dim3((uint32_t)ceil_div(vectors, 256)), dim3(256), 0, stream>>>(
                        (const T*)dh, (const T*)gate_up, (T*)dgate_up, (uint32_t)vectors, (uint32_t)per_row, (int)f);
            });
        });
    });
}

}  // namespace coc

extern "C" {

coc_status coc_gated_act(const void* gate_up, void* h, int64_t rows, int64_t f, coc_act act, coc_dtype dt,
                         hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_gated(rows, f, act, dt, false);
    if (st != COC_OK) return st;
    if (rows == 0) return COC_OK;
    const int32_t es = (int32_t)elem_size(dt);
    const Arg args[] = {{gate_up, rows * 2 * f * es, es, false, "gate_up"}, {h, rows * f * es, es, true, "h"}};
    st = check_args(args, 2);
    if (st != COC_OK) return st;
    by_type(dt, [&](auto t) {
        using T = decltype(t);
        by_act(act, [&](auto a) {
            by_kind<T>(f, [&](auto kind) {
                const int64_t per_row = ceil_div(f, kVec<T>), vectors = rows * per_row;
                gated_forward<T, decltype(a)::value, decltype(kind)::value>
                    <<<dim3((uint32_t)ceil_div(vectors, 256)), dim3(256), 0, stream>>>(
                        (const T*)gate_up, (T*)h, (uint32_t)vectors, (uint32_t)per_row, (int)f);
            });
        });
    });
    return launched("gated activation");
}

coc_status coc_gated_act_fp8(const void* gate_up, void* q, float* scales, int64_t rows, int64_t f, coc_act act,
                             coc_dtype dt, hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_gated(rows, f, act, dt, true);
    if (st != COC_OK) return st;
    if (rows == 0) return COC_OK;
    const int32_t es = (int32_t)elem_size(dt);
    const Arg args[] = {{gate_up, rows * 2 * f * es, es, false, "gate_up"},
                        {q, rows * f, 16, true, "q"},
                        {scales, ceil_div(f, kScaleBlock) * rows * 4, 4, true, "scales"}};
    st = check_args(args, 3);
    if (st != COC_OK) return st;
    by_act(act, [&](auto a) { launch_quantize_rows<decltype(a)::value>(gate_up, q, scales, rows, f, dt, stream); });
    return launched("gated activation");
}

coc_status coc_gated_act_backward(const void* dh, const void* gate_up, void* dgate_up, int64_t rows, int64_t f,
                                  coc_act act, coc_dtype dt, hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_gated(rows, f, act, dt, false);
    if (st != COC_OK) return st;
    if (rows == 0) return COC_OK;
    const int32_t es = (int32_t)elem_size(dt);
    const Arg args[] = {{dh, rows * f * es, es, false, "dh"},
                        {gate_up, rows * 2 * f * es, es, false, "gate_up"},
                        {dgate_up, rows * 2 * f * es, es, true, "dgate_up"}};
    st = check_args(args, 3);
    if (st != COC_OK) return st;
    launch_gated_act_backward(dh, gate_up, dgate_up, rows, f, act, dt, stream);
    return launched("gated activation backward");
}

coc_status coc_quantize_fp8(const void* x, void* q, float* scales, int64_t rows, int64_t n, int32_t block_rows,
                            coc_dtype dt, hipStream_t stream) {
    using namespace coc;
    clear_error();
    if (!dtype_valid(dt)) return fail(COC_ERR_DTYPE, "unknown dtype %d", (int)dt);
    if (block_rows != 1 && block_rows != kScaleBlock)
        return fail(COC_ERR_DTYPE, "a scale covers 1 or %d rows (block_rows=%d)", kScaleBlock, (int)block_rows);
    coc_status st = check_matrix(rows, n, "x");
    if (st != COC_OK) return st;
    if (n % 16 != 0) return fail(COC_ERR_SHAPE, "rows in 8 bits have a multiple of 16 elements (n=%lld)", (long long)n);
    if (rows == 0 || n == 0) return COC_OK;
    const int32_t es = (int32_t)elem_size(dt);
    const int64_t blocks = ceil_div(n, kScaleBlock), groups = ceil_div(rows, block_rows);
    const Arg args[] = {{x, rows * n * es, es, false, "x"},
                        {q, rows * n, 16, true, "q"},
                        {scales, blocks * groups * 4, 4, true, "scales"}};
    st = check_args(args, 3);
    if (st != COC_OK) return st;
    if (block_rows == 1)
        launch_quantize_rows<-1>(x, q, scales, rows, n, dt, stream);
    else
        by_type(dt, [&](auto t) {
            using T = decltype(t);
            quantize_blocks<T><<<dim3((uint32_t)(groups * blocks)), dim3(256), 0, stream>>>(
                (const T*)x, (uint8_t*)q, scales, rows, (int)n, (int)blocks);
        });
    return launched("quantize");
}

}  // extern "C"
