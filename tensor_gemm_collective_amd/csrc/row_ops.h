// Shared by the row operators (layer norm, embedding, MoE router, MoE row
// moves): argument checks on the host, and on the device 16-byte row vectors
// of any alignment, conversions, and reductions over lanes and workgroups.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "coc.h"
#include "coc_internal.h"

namespace coc {

// ------------------------------------------------------------------ host checks
// One pointer argument.  The row operators take any element-aligned address:
// their 16-byte loads and stores need no more (see load_vec).
struct Arg {
    const void* p;
    int64_t bytes;   // 0: not read or written, may be NULL
    int32_t align;   // element size
    bool out;
    const char* name;
};

inline coc_status check_args(const Arg* a, int count) {
    for (int i = 0; i < count; ++i) {
        if (a[i].bytes <= 0) continue;
        if (!a[i].p) return fail(COC_ERR_NULL, "%s is NULL", a[i].name);
        if ((uintptr_t)a[i].p % (uintptr_t)a[i].align != 0)
            return fail(COC_ERR_ALIGN, "%s is not %d-byte aligned", a[i].name, a[i].align);
    }
    for (int i = 0; i < count; ++i) {
        if (!a[i].out || a[i].bytes <= 0) continue;
        for (int j = 0; j < count; ++j) {
            if (j == i || a[j].bytes <= 0 || (a[j].out && j < i)) continue;
            const uintptr_t lo = (uintptr_t)a[i].p, lo2 = (uintptr_t)a[j].p;
            if (lo < lo2 + (uintptr_t)a[j].bytes && lo2 < lo + (uintptr_t)a[i].bytes)
                return fail(COC_ERR_ALIAS, "%s overlaps %s", a[i].name, a[j].name);
        }
    }
    return COC_OK;
}

// rows x cols of a matrix within the library's limits.  The row limit keeps
// every launch below 2^32 threads (at most 64 a row where a row is short), and
// the column limit the kernels' 32-bit column numbers, which run past a row's
// end by a workgroup's step.
inline coc_status check_matrix(int64_t rows, int64_t cols, const char* what) {
    const int64_t lim = int64_t(1) << 31;
    if (rows < 0 || cols < 0) return fail(COC_ERR_SHAPE, "%s has a negative size", what);
    if (rows >= lim || cols >= lim || rows * cols >= lim)
        return fail(COC_ERR_SHAPE, "%s has 2^31 or more elements", what);
    if (cols >= int64_t(1) << 30) return fail(COC_ERR_SHAPE, "%s has rows of 2^30 or more elements", what);
    if (rows >= int64_t(1) << 25) return fail(COC_ERR_SHAPE, "%s has 2^25 or more rows", what);
    return COC_OK;
}

inline coc_status launched(const char* what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(COC_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
    return COC_OK;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// ------------------------------------------------------------------ device: types and vectors
typedef _Float16 f16_t;
typedef __bf16 bf16_t;

// Elements of T in 16 bytes.
template <class T>
constexpr int kVec = 16 / (int)sizeof(T);

// 16 bytes of elements as four words: kept so, they take four registers (an
// array of 16-bit values takes one for each).
template <class T>
struct Packed {
    uint32_t w[4];
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[i]);
        else if constexpr (std::is_same_v<T, bf16_t>)
            return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
        else
            return (float)__builtin_bit_cast(T, (uint16_t)(w[i >> 1] >> (i & 1 ? 16 : 0)));
    }
    // from binary32, each rounded once, to nearest even
    __device__ __forceinline__ void set(const float* f) {
        typedef T t2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4)
                w[i] = __float_as_uint(f[i]);
            else
                w[i] = __builtin_bit_cast(uint32_t, t2{(T)f[2 * i], (T)f[2 * i + 1]});
        }
    }
};

// Makes the compiler unpack p anew after this point instead of keeping what it
// unpacked before it: four registers across a barrier, not eight.
template <class T>
__device__ __forceinline__ void repack(Packed<T>& p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("" : "+v"(p.w[i]));
}

// Row elements [c, c + kVec) at an address aligned to T only; those at or past n
// are 0.  Global memory takes 16-byte accesses of any alignment in the
// unaligned access mode that the HSA ABI runs in, so rows of odd length need no
// path of their own.
template <class T>
__device__ __forceinline__ void load_raw(const T* row, int c, int n, Packed<T>* p) {
    if (c + kVec<T> <= n) {
        __builtin_memcpy(p->w, row + c, 16);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t v = 0;
            if constexpr (sizeof(T) == 4) {
                if (c + i < n) __builtin_memcpy(&v, row + c + i, 4);
            } else {
                uint16_t h = 0;
                if (c + 2 * i < n) __builtin_memcpy(&h, row + c + 2 * i, 2);
                v = h;
                h = 0;
                if (c + 2 * i + 1 < n) __builtin_memcpy(&h, row + c + 2 * i + 1, 2);
                v |= (uint32_t)h << 16;
            }
            p->w[i] = v;
        }
    }
}

template <class T>
__device__ __forceinline__ void load_vec(const T* row, int c, int n, float* f) {
    Packed<T> p;
    load_raw(row, c, n, &p);
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) f[i] = p.get(i);
}

// 16 bytes that nobody reads soon: stored without keeping them in the L2
// (outputs of the big passes; see embedding.hip for what it gains).
template <class T>
__device__ __forceinline__ void stream16(T* at, const Packed<T>& p) {
    typedef uint32_t u32x4_2 __attribute__((ext_vector_type(4), aligned(2)));
    typedef uint32_t u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));
    typedef std::conditional_t<sizeof(T) == 2, u32x4_2, u32x4_4> u32x4;
    u32x4 v = {p.w[0], p.w[1], p.w[2], p.w[3]};
    __builtin_nontemporal_store(v, (u32x4*)at);
}

template <class T>
__device__ __forceinline__ void store_raw(T* row, int c, int n, const Packed<T>& p) {
    if (c + kVec<T> <= n) {
        stream16(row + c, p);
    } else {
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i)
            if (c + i < n) {
                if constexpr (sizeof(T) == 4) {
                    __builtin_memcpy(row + c + i, &p.w[i], 4);
                } else {
                    const uint16_t h = (uint16_t)(p.w[i >> 1] >> (i & 1 ? 16 : 0));
                    __builtin_memcpy(row + c + i, &h, 2);
                }
            }
    }
}

template <class T>
__device__ __forceinline__ void store_vec(T* row, int c, int n, const float* f) {
    Packed<T> p;
    p.set(f);
    store_raw(row, c, n, p);
}

// The columns a thread takes as its vector `i` of a row: [c, c + kVec), of which
// the first `skip` belong to another vector.  The row's last vector ends at its
// end, overlapping the one before, and vectors past it are there again with
// every column skipped: every load is whole and without a branch (a branch
// around a load makes the compiler wait for all loads before it goes on), sums
// leave the skipped columns out, and what is written twice is the same.
// kWhole: n is a multiple of kVec (skip is 0 or kVec); kTiny: n < kVec (one
// vector, loaded element by element; others are past the row).
enum RowKind { kWhole, kRagged, kTiny };
template <class T, RowKind KIND>
struct Cols {
    int c, skip;
    __device__ __forceinline__ Cols(int i, int n) {
        c = KIND == kTiny ? i * kVec<T> : min(i * kVec<T>, n - kVec<T>);
        skip = KIND == kTiny ? 0 : min(i * kVec<T> - c, kVec<T>);
    }
    __device__ __forceinline__ void load(const T* row, int n, Packed<T>* p) const {
        if constexpr (KIND == kTiny)
            load_raw(row, c, n, p);
        else
            __builtin_memcpy(p->w, row + c, 16);
    }
    __device__ __forceinline__ void store(T* row, int n, const Packed<T>& p) const {
        if constexpr (KIND == kTiny)
            store_raw(row, c, n, p);
        else if (skip < kVec<T>)
            stream16(row + c, p);
    }
    // Whether column c + i counts here.
    __device__ __forceinline__ bool has(int i, int n) const {
        return KIND == kTiny ? c + i < n : KIND == kWhole ? skip == 0 : i >= skip;
    }
};

// N elements of a parameter or sum vector, whose type U may be wider than the
// rows' (N: a multiple or a half of kVec<U>).
template <int N, class U>
__device__ __forceinline__ void load_n(const U* v, int c, int n, float* f) {
    if constexpr (N % kVec<U> == 0) {
#pragma unroll
        for (int i = 0; i < N; i += kVec<U>) load_vec(v, c + i, n, f + i);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = c + i < n ? (float)v[c + i] : 0.0f;
    }
}

// N values rounded to the vector's type U, for what is read again soon.
template <int N, class U>
__device__ __forceinline__ void keep_n(U* v, int c, int n, const float* f) {
    if (c + N <= n) {
        struct __attribute__((packed, aligned(sizeof(U)))) { U e[N]; } p;
#pragma unroll
        for (int i = 0; i < N; ++i) p.e[i] = (U)f[i];
        __builtin_memcpy(v + c, &p, sizeof(p));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c + i < n) v[c + i] = (U)f[i];
    }
}

// The same streamed, N a multiple of 4.
template <int N, class U>
__device__ __forceinline__ void store_n(U* v, int c, int n, const float* f) {
    if constexpr (N % kVec<U> == 0) {
#pragma unroll
        for (int i = 0; i < N; i += kVec<U>) store_vec(v, c + i, n, f + i);
    } else {
        keep_n<N>(v, c, n, f);
    }
}

// The binary32 product, rounded as such also where a conversion to fp16 follows
// (one instruction could do both in one rounding, and another variant of the
// same code not).
__device__ __forceinline__ float product(float a, float b) {
    float p = a * b;
    asm("" : "+v"(p));   // no code: what follows cannot be joined with the product
    return p;
}

// ------------------------------------------------------------------ device: reductions
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u(uint64_t v) {
    return (uint64_t)dpp_u<CTRL>((uint32_t)(v >> 32)) << 32 | dpp_u<CTRL>((uint32_t)v);
}
constexpr int kDppXor1 = 0xB1;         // quad_perm [1, 0, 3, 2]
constexpr int kDppXor2 = 0x4E;         // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141;  // within 8 lanes: the other quad
constexpr int kDppMirror = 0x140;      // within 16 lanes: the other 8

// Sum over aligned groups of LANES lanes, the same bits in each of them.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
    if constexpr (LANES >= 2) v += dpp_f<kDppXor1>(v);
    if constexpr (LANES >= 4) v += dpp_f<kDppXor2>(v);
    if constexpr (LANES >= 8) v += dpp_f<kDppHalfMirror>(v);
    if constexpr (LANES >= 16) v += dpp_f<kDppMirror>(v);
    if constexpr (LANES >= 32) v += __shfl_xor(v, 16);
    if constexpr (LANES >= 64) v += __shfl_xor(v, 32);
    return v;
}

// Largest value over aligned groups of LANES lanes.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    if constexpr (LANES >= 2) v = max(v, dpp_u<kDppXor1>(v));
    if constexpr (LANES >= 4) v = max(v, dpp_u<kDppXor2>(v));
    if constexpr (LANES >= 8) v = max(v, dpp_u<kDppHalfMirror>(v));
    if constexpr (LANES >= 16) v = max(v, dpp_u<kDppMirror>(v));
    if constexpr (LANES >= 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16));
    if constexpr (LANES >= 64) v = max(v, (uint32_t)__shfl_xor((int)v, 32));
    return v;
}

template <int LANES>
__device__ __forceinline__ uint64_t lanes_max(uint64_t v) {
    if constexpr (LANES >= 2) v = max(v, dpp_u<kDppXor1>(v));
    if constexpr (LANES >= 4) v = max(v, dpp_u<kDppXor2>(v));
    if constexpr (LANES >= 8) v = max(v, dpp_u<kDppHalfMirror>(v));
    if constexpr (LANES >= 16) v = max(v, dpp_u<kDppMirror>(v));
    if constexpr (LANES >= 32) v = max(v, (uint64_t)__shfl_xor((unsigned long long)v, 16));
    if constexpr (LANES >= 64) v = max(v, (uint64_t)__shfl_xor((unsigned long long)v, 32));
    return v;
}

// Sum over a workgroup of THREADS threads, in a fixed order; `buf` holds a
// float per wave.  Callers that reuse a buf have a barrier between.
template <int THREADS>
__device__ __forceinline__ float group_sum(float v, float* buf) {
    v = lanes_sum<64>(v);
    if constexpr (THREADS > 64) {
        if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
        __syncthreads();
        v = buf[0];
#pragma unroll
        for (int w = 1; w < THREADS / 64; ++w) v += buf[w];
    }
    return v;
}

}  // namespace coc
