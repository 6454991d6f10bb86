// What the MFMA tiles share: the order of tiles, direct-to-LDS loads and their waits, and
// an operand's stages in LDS.
//
// A stage holds 128 bytes of k (64 values of 16 bits, 128 of 8) of the tile's rows.  An
// operand is stored one of two ways:
//   k-contiguous (A as m rows of k, B as n rows of k): LDS rows of 128 bytes, chunk c of
//     row r at c ^ ((r >> 1) & 7), fragments by ds_read_b128;
//   k-major (16 bits; A as k rows of m, B as k rows of n): LDS rows of one k, fragments by
//     the transposing ds_read_b64_tr_b16, two each; the chunks of the eight k rows that
//     one pass reads (k .. k + 3 and k + 8 .. k + 11) lie in distinct banks.
// k past the end is read as zeros from g_zeros, so an operand's rows need only be whole
// 16-byte chunks.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "coc_internal.h"
#include "row_ops.h"

namespace coc {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
#define COC_LDS __attribute__((address_space(3)))

__device__ const u32x4 g_zeros = {0, 0, 0, 0};

// ------------------------------------------------------------------ tile order
// Workgroups go to the 8 XCDs (each with its own L2) round-robin by id.  XCD x takes a
// contiguous run of tile numbers, and tiles are numbered in groups of four tile rows,
// rows first, so that the tiles of an XCD share their operands' blocks.
__device__ __forceinline__ void tile_of(int b, int tiles_m, int tiles_n, int* tm, int* tn) {
    constexpr int NX = 8, GM = 4;
    const int total = tiles_m * tiles_n, q = total / NX, r = total % NX;
    const int x = b % NX, t = x * q + (x < r ? x : r) + b / NX;
    const int g = t / (GM * tiles_n), in_g = t - g * GM * tiles_n;
    const int rows = min(tiles_m - g * GM, GM);
    *tm = g * GM + in_g % rows;
    *tn = in_g / rows;
}

// ------------------------------------------------------------------ loads and waits
// 16 bytes a lane into LDS at `lds` + 16 lane (device scope: each chunk is read once by
// a workgroup, so it need not stay in the L1), addressed as a scalar base plus 32-bit
// offsets, or by pointers.  Ordered by wait_loads and the barrier alone.
__device__ __forceinline__ void load_lds(uint32_t off, const void* base, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 sc1" ::"v"(off), "s"(base), "s"(lds)
                 : "memory", "m0");
}
__device__ __forceinline__ void load_lds_at(const void* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off sc1" ::"v"(src), "s"(lds)
                 : "memory", "m0");
}
// 4 bytes a lane into LDS at `lds` + 4 lane.
__device__ __forceinline__ void load_lds4(uint32_t off, const void* base, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1 sc1" ::"v"(off), "s"(base), "s"(lds)
                 : "memory", "m0");
}
// At most N of the wave's loads in flight, and none of its LDS reads.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (0 << 8));
}
__device__ __forceinline__ void group_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) { return (uint32_t)(uintptr_t)(const COC_LDS void*)p; }

template <class T>
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
    typedef T t2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, t2{(T)lo, (T)hi});
}

__device__ __forceinline__ int row_swizzle(int r) { return (r >> 1) & 7; }
// k-major rows of W 16-byte chunks
template <int W>
__device__ __forceinline__ int k_swizzle(int k) {
    if constexpr (W >= 16)
        return ((k & 3) << 2) | (((k >> 3) & 1) << 1);
    else   // two rows a bank cycle: the lowest bit of k chooses the half
        return (((k >> 1) & 1) << 2) | (((k >> 3) & 1) << 1);
}

// ------------------------------------------------------------------ one operand in LDS
// ROWS m rows or n columns of the tile, values of ES bytes.  TRANS: stored k-major.
template <int ROWS, bool TRANS, int NW, int ES = 2>
struct Operand {
    static constexpr int STEP = 128 / ES;                             // k of a stage
    static constexpr int BYTES = ROWS * 128;
    static constexpr int INS = BYTES / 1024;                          // load instructions a stage
    static constexpr int PER_WAVE = INS / NW;
    static constexpr int CHUNKS = ROWS / 8;                           // TRANS: 16-byte chunks of a k row
    static constexpr int READS = TRANS ? 2 : 1;                       // LDS reads a fragment
    static_assert(INS % NW == 0, "loads split over the waves");
    static_assert(!TRANS || CHUNKS == 8 || CHUNKS == 16 || CHUNKS == 32, "k rows of 64, 128 or 256 elements");

    uint32_t off[PER_WAVE];   // from the stage's base, bytes
    int q0;                   // this lane's chunk of the first load
    const uint8_t* base;
    int64_t step;             // bytes from stage to stage
    uint32_t lds;             // its place in slot 0; NEXT later for each further load
    static constexpr uint32_t NEXT = NW * 1024;

    // first(local row or column) -> the global one to read; ld: elements from row to row
    template <class F>
    __device__ __forceinline__ void init(const void* p, int64_t ld, int stage0, uint32_t lds0, int wave, int lane,
                                         F&& first) {
        step = TRANS ? STEP * ld * ES : 128;
        base = (const uint8_t*)p + stage0 * step;
        q0 = wave * 64 + lane;   // load i of the waves together: neighbouring rows
#pragma unroll
        for (int i = 0; i < PER_WAVE; ++i) {
            const int q = q0 + i * NW * 64;
            if constexpr (TRANS) {
                const int k = q / CHUNKS, c = (q % CHUNKS) ^ k_swizzle<CHUNKS>(k);
                off[i] = (uint32_t)k * (uint32_t)ld * 2 + (uint32_t)first(c * 8) * 2;
            } else {
                const int r = q >> 3, c = (q & 7) ^ row_swizzle(r);
                off[i] = (uint32_t)((int64_t)first(r) * ld * ES) + (uint32_t)c * 16;
            }
        }
        lds = lds0 + wave * 1024;
    }
    // the k of load i's chunk within its stage
    __device__ __forceinline__ int at(int i) const {
        const int q = q0 + i * NW * 64;
        return TRANS ? q / CHUNKS : ((q & 7) ^ row_swizzle(q >> 3)) * (16 / ES);
    }
    // load i of stage s (counted from stage0) into the slot `slot_bytes` on; left: how
    // many k the stage has (WHOLE: all)
    template <bool WHOLE>
    __device__ __forceinline__ void load(int i, int s, uint32_t slot_bytes, int left) const {
        const uint8_t* b = base + s * step;
        const uint32_t to = __builtin_amdgcn_readfirstlane(lds + slot_bytes + i * NEXT);
        if (WHOLE || left >= STEP)
            load_lds(off[i], b, to);
        else
            load_lds_at(at(i) < left ? (const void*)(b + off[i]) : (const void*)&g_zeros, to);
    }
};

// ------------------------------------------------------------------ which tile (host)
constexpr int64_t kCus = 256;   // of an MI355X

// A tile as measured: its rows and columns (of the operands), the workgroups a CU holds,
// the time of a stage in us while there is at most one workgroup a CU (`light`) and while
// there are more (`full`), and of a tile's start and end (`ends`).  Whether it is offered
// whole, and split along k.
struct TileCost {
    int rows, cols, per_cu;
    float light, full, ends;
    bool whole, split;
};

struct Choice {
    int tile;     // index into the costs
    int stages;   // of one split
    int splits;   // 1: not split
    bool split;   // leaves sums for a joining kernel
    float us;     // estimated
};

// The tile and split of the least estimated time for an m x n product of `stages` stages:
// rounds of workgroups times a round's stages, and for a split the joining kernel (5 us of
// launches, and its sums written and read at 6 TB/s).
template <int N>
inline Choice pick(const TileCost (&costs)[N], int64_t m, int64_t n, int64_t stages) {
    Choice best{0, (int)stages, 1, false, 1e30f};
    for (int t = 0; t < N; ++t) {
        const TileCost& c = costs[t];
        const int64_t tiles = ceil_div(m, c.rows) * ceil_div(n, c.cols);
        for (int64_t s : {1, 2, 3, 4, 6, 8, 12, 16}) {
            if (s == 1 ? !(c.whole || c.split) : !c.split) continue;
            const int64_t each = ceil_div(stages, s);
            if (s > 1 && (each < 2 || ceil_div(stages, each) != s)) continue;
            const bool join = s > 1 || !c.whole;
            const int64_t groups = tiles * s;
            float us = (float)ceil_div(groups, kCus * c.per_cu) *
                       ((float)each * (groups <= kCus ? c.light : c.full) + c.ends);
            if (join) us += 5.0f + (float)(s * m * n) * (8.0f / 6e6f);
            if (us < best.us) best = {t, (int)each, (int)s, join, us};
            if (groups > 4 * kCus * c.per_cu) break;
        }
    }
    return best;
}

// f(how many splits' sums a joining kernel loads together).
template <class F>
void by_splits(int splits, F&& f) {
    if (splits <= 2)
        f(std::integral_constant<int, 2>());
    else if (splits <= 4)
        f(std::integral_constant<int, 4>());
    else if (splits <= 8)
        f(std::integral_constant<int, 8>());
    else
        f(std::integral_constant<int, 16>());
}

}  // namespace
}  // namespace coc
