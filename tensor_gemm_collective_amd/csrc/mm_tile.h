// The 16-bit MFMA tile of the gated feed-forward block's products.
//
// C (m x n) = A B over k in binary32, WM x WN waves a workgroup, each a block of FI x FJ
// v_mfma_f32_16x16x32 outputs.  k runs in stages of 64 through S LDS slots that
// direct-to-LDS loads fill ahead of the waves (lds_tile.h).  Rows and columns past m and
// n are read clamped and not stored.
//
// Large products are bound by the clock that the matrix units hold while the LDS is
// filled and read beside them (1.97 GHz, MFMAs issued 62 % of the time).  Measured on
// copies of the tile: without any wait or barrier the products of 4096 x 8192 x 7168 gain
// 4 %, with half the LDS reads 3 %, without the loads to LDS 17 %.  Eight waves of 128 x 64
// (two a SIMD) take 376 us for the gated product, 344 for dx and 381 for dw; four of 128 x
// 128 read a third less from the LDS but take 389, 345 and 567, since the transposing reads
// need more of a lone wave's time.  Wave priorities around the barrier and the barrier's
// place within the stage changed nothing.
#pragma once

#include "gated_act.h"
#include "lds_tile.h"

namespace coc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <class T>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (std::is_same_v<T, bf16_t>)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

// Fragment reads of block `j` (16 rows or columns, counted from init's `first`), k step ks (32 k).
template <int ROWS, bool TRANS>
struct Fragments {
    int place[2];
    __device__ __forceinline__ void init(int first, int lane) {
        if constexpr (TRANS) {
            // a 16-lane group g reads k 8g .. 8g + 3 (then + 4) of its 16 columns: lane
            // 4j + q points at row j's columns 4q, and lane i receives column i
            const int r = lane & 15, k = (lane >> 4) * 8 + (r >> 2);
            place[0] = k * ROWS * 2 + (r & 1) * 8;
            place[1] = (first >> 3) + ((r & 3) >> 1);   // chunk of block 0
        } else {
            const int row = first + (lane & 15);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) place[ks] = row * 128 + (((ks * 4 + (lane >> 4)) ^ row_swizzle(row)) << 4);
        }
    }
    // read h (of READS) of block j
    __device__ __forceinline__ void read(const COC_LDS uint8_t* slot, int j, int ks, int h, int lane, u32x4* f) const {
        if constexpr (TRANS) {
            // (the swizzle of k does not depend on ks, h: they add 32 and 4)
            const int k = (lane >> 4) * 8 + ((lane & 15) >> 2);
            const int c = (place[1] + j * 2) ^ k_swizzle<ROWS / 8>(k + h * 4);
            const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (COC_LDS s16x4*)(slot + place[0] + (ks * 32 + h * 4) * ROWS * 2 + c * 16));
            const u32x2 w = __builtin_bit_cast(u32x2, v);
            (*f)[2 * h] = w[0];
            (*f)[2 * h + 1] = w[1];
        } else {
            *f = *(const COC_LDS u32x4*)(slot + place[ks] + j * 16 * 128);
        }
    }
};

// ------------------------------------------------------------------ the tile
struct MmParams {
    const void *a, *b;
    void *c, *gate_up;     // of the gated product either may be NULL
    float* part;           // partial sums: splits x m x all columns
    int m, n, k;           // n: columns of C; of the gated product f
    int64_t lda, ldb;      // elements from stored row to stored row
    int tiles_m, tiles_n, stages;   // stages: of one split
    int act;
};

// GATED: B holds 2n columns, gate then up; a wave's first FJ / 2 column blocks are gate
// columns and the others the up columns beside them, so that h = act(g) u is formed in
// registers.  PART: the k range is split over blockIdx.y and binary32 sums are left in
// p.part for a joining kernel.
template <class T, bool TA, bool TB, int FI, int FJ, int WM, int WN, int S, bool GATED, bool PART>
struct MmTile {
    static constexpr int NW = WM * WN, BM = WM * FI * 16, BN = WN * FJ * 16;
    static constexpr int OUT = GATED ? BN / 2 : BN;   // columns of C a tile gives
    using A = Operand<BM, TA, NW>;
    using B = Operand<BN, !TB, NW>;
    static constexpr int SLOT = A::BYTES + B::BYTES;
    static constexpr int LDS = S * SLOT;
    static constexpr int DPW = A::PER_WAVE + B::PER_WAVE;
    static constexpr int NMM = FI * FJ, NRD = A::READS * FI + B::READS * FJ;
    static constexpr int BAR_AT = NMM / 4;
    static constexpr int RPM = (NRD + NMM - BAR_AT - 1) / (NMM - BAR_AT);   // reads an MFMA
    static_assert(PART || NW * FI * 16 * FJ * 32 <= LDS, "the staged output fits in the LDS");

    // block: the tile's number, of the launch's or of this product's
    static __device__ __forceinline__ void run(const MmParams& p, uint8_t* sm, int block) {
        int tm, tn;
        tile_of(block, p.tiles_m, p.tiles_n, &tm, &tn);
        const int m0 = tm * BM, n0 = tn * OUT;
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int wm = wave / WN, wn = wave % WN;
        const uint32_t lds0 = lds_address(sm);
        const int stage0 = PART ? (int)blockIdx.y * p.stages : 0;
        const int k0 = stage0 * 64;
        const int KT = min(p.stages, (p.k - k0 + 63) / 64);   // >= 1

        A a;
        B b;
        a.init(p.a, p.lda, stage0, lds0, wave, lane, [&](int r) { return min(m0 + r, TA ? p.m - 8 : p.m - 1); });
        b.init(p.b, p.ldb, stage0, lds0 + A::BYTES, wave, lane, [&](int c) {
            if constexpr (GATED) {
                // local column -> its wave's block -> gate or up column
                const int w = c / (FJ * 16), r = c % (FJ * 16), up = r / (FJ * 8);
                return min(n0 + w * FJ * 8 + r % (FJ * 8), p.n - 8) + up * p.n;
            } else {
                return min(n0 + c, TB ? p.n - 1 : p.n - 8);
            }
        });
        Fragments<BM, TA> fa;
        Fragments<BN, !TB> fb;
        fa.init(wm * FI * 16, lane);
        fb.init(wn * FJ * 16, lane);
        auto load = [&](int d, int s, int slot, auto WHOLE) {
            constexpr bool whole = decltype(WHOLE)::value;
            const int left = p.k - k0 - s * 64;
            if (d < A::PER_WAVE)
                a.template load<whole>(d, s, slot * SLOT, left);
            else
                b.template load<whole>(d - A::PER_WAVE, s, slot * SLOT, left);
        };
        u32x4 af[2][FI], bf[2][FJ];
        // read r of a k step's: the first row block, the columns, the other row blocks
        auto read = [&](int r, int slot, int ks, int buf) {
            const COC_LDS uint8_t* s = (const COC_LDS uint8_t*)sm + slot * SLOT;
            constexpr int AR = A::READS, BR = B::READS;
            if (r < AR)
                fa.read(s, 0, ks, r, lane, &af[buf][0]);
            else if (r < AR + BR * FJ)
                fb.read(s + A::BYTES, (r - AR) / BR, ks, (r - AR) % BR, lane, &bf[buf][(r - AR) / BR]);
            else
                fa.read(s, (r - BR * FJ) / AR, ks, (r - BR * FJ) % AR, lane, &af[buf][(r - BR * FJ) / AR]);
        };
        f32x4 acc[FI][FJ];
#pragma unroll
        for (int i = 0; i < FI; ++i)
#pragma unroll
            for (int j = 0; j < FJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        for (int s = 0; s < S && s < KT; ++s)
#pragma unroll
            for (int d = 0; d < DPW; ++d) load(d, s, s, std::false_type());
        if (KT >= S)
            wait_loads<(S - 1) * DPW>();
        else
            wait_loads<0>();
        group_barrier();
#pragma unroll
        for (int r = 0; r < NRD; ++r) read(r, 0, 0, 0);

        // One stage: two k steps.  The second's fragments are read under the first's
        // MFMAs; a quarter into the second the workgroup meets (every wave has read
        // this slot, and the next stage has arrived), then the next stage's first
        // fragments are read and stage kt + S is loaded into this slot.
        auto stage = [&](int kt, int slot, auto MORE, auto LOAD, auto WHOLE, auto WAIT) {
            constexpr bool more = decltype(MORE)::value, loads = decltype(LOAD)::value;
            const int next = slot + 1 == S ? 0 : slot + 1;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < NMM; ++s) {
                acc[s / FJ][s % FJ] = mfma16<T>(bf[0][s % FJ], af[0][s / FJ], acc[s / FJ][s % FJ]);
#pragma unroll
                for (int q = 0; q < RPM; ++q)
                    if (s * RPM + q < NRD) read(s * RPM + q, slot, 1, 1);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int s = 0; s < BAR_AT; ++s) {
                acc[s / FJ][s % FJ] = mfma16<T>(bf[1][s % FJ], af[1][s / FJ], acc[s / FJ][s % FJ]);
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (more) {
                wait_loads<decltype(WAIT)::value>();
                group_barrier();
            }
#pragma unroll
            for (int s = BAR_AT; s < NMM; ++s) {
                acc[s / FJ][s % FJ] = mfma16<T>(bf[1][s % FJ], af[1][s / FJ], acc[s / FJ][s % FJ]);
                constexpr int LEFT = NMM - BAR_AT;
                const int g = s - BAR_AT;
                if constexpr (more) {
#pragma unroll
                    for (int q = 0; q < RPM; ++q)
                        if (g * RPM + q < NRD) read(g * RPM + q, next, 0, 0);
                }
                if constexpr (loads) {
#pragma unroll
                    for (int d = 0; d < DPW; ++d)
                        if (d * LEFT / DPW == g) load(d, kt + S, slot, WHOLE);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        using yes = std::true_type;
        using no = std::false_type;
        int kt = 0, slot = 0;
        using all = std::integral_constant<int, (S - 2) * DPW>;
        using none = std::integral_constant<int, 0>;
        auto step = [&] { slot = slot + 1 == S ? 0 : slot + 1; };
        // at stage kt's barrier the stages kt + 1 .. kt + S - 1 are in flight; the last
        // stage alone may be short of k
        for (; kt + S + 1 < KT; ++kt, step()) stage(kt, slot, yes(), yes(), yes(), all());
        if (kt + S < KT) {
            stage(kt, slot, yes(), yes(), no(), all());
            ++kt;
            step();
        }
        for (; kt + 1 < KT; ++kt, step()) stage(kt, slot, yes(), no(), no(), none());
        stage(kt, slot, no(), no(), no(), none());

        // A lane holds row l % 16 and columns 4 (l / 16) .. + 3 of each 16 x 16 block.
        if constexpr (PART) {
            const int all = GATED ? 2 * p.n : p.n;
            float* out = p.part + (int64_t)blockIdx.y * p.m * all;
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int j = 0; j < FJ; ++j) {
                    const int row = m0 + (wm * FI + i) * 16 + (lane & 15);
                    const int up = GATED && j >= FJ / 2;
                    const int col = n0 + (GATED ? (wn * FJ / 2 + j % (FJ / 2)) : wn * FJ + j) * 16 + (lane >> 4) * 4;
                    if (row < p.m && col < p.n) *(f32x4*)(out + (int64_t)row * all + up * p.n + col) = acc[i][j];
                }
        } else {
            // each wave's rows through its own LDS, then whole rows to memory
            group_barrier();
            COC_LDS uint8_t* stg = (COC_LDS uint8_t*)sm + wave * (FI * 16 * FJ * 32);
            auto put = [&](auto COLS, auto&& value, uint8_t* c, int64_t ld, int64_t col_of, int col0) {
                constexpr int NJ = decltype(COLS)::value, PITCH = NJ * 32, CPR = NJ * 2, RPI = 64 / CPR;
                static_assert(64 % CPR == 0 && FI * 16 % RPI == 0, "staging layout");
#pragma unroll
                for (int i = 0; i < FI; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const int row = i * 16 + (lane & 15), ch = j * 2 + (lane >> 5);
                        const f32x4 v = value(i, j);
                        *(COC_LDS u32x2*)(stg + row * PITCH + ((ch ^ (row & (CPR - 1))) << 4) + ((lane >> 4) & 1) * 8) =
                            u32x2{round2<T>(v[0], v[1]), round2<T>(v[2], v[3])};
                    }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int t = 0; t < FI * 16 / RPI; ++t) {
                    const int row = t * RPI + lane / CPR, ch = lane % CPR;
                    const u32x4 v = *(const COC_LDS u32x4*)(stg + row * PITCH + ((ch ^ (row & (CPR - 1))) << 4));
                    const int r = m0 + wm * FI * 16 + row, col = col0 + ch * 8;
                    if (r < p.m && col < p.n) *(u32x4*)(c + (r * ld + col_of + col) * 2) = v;
                }
                __builtin_amdgcn_sched_barrier(0);
            };
            if constexpr (GATED) {
                constexpr int H = FJ / 2;
                const int col0 = n0 + wn * H * 16;
                if (p.c) by_act((coc_act)p.act, [&](auto act) {
                    put(std::integral_constant<int, H>(),
                        [&](int i, int j) {
                            f32x4 v;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                v[e] = act_value<decltype(act)::value>(acc[i][j][e]) * acc[i][j + H][e];
                            return v;
                        },
                        (uint8_t*)p.c, p.n, 0, col0);
                });
                if (p.gate_up) {
                    put(std::integral_constant<int, H>(), [&](int i, int j) { return acc[i][j]; }, (uint8_t*)p.gate_up,
                        2 * (int64_t)p.n, 0, col0);
                    put(std::integral_constant<int, H>(), [&](int i, int j) { return acc[i][j + H]; },
                        (uint8_t*)p.gate_up, 2 * (int64_t)p.n, p.n, col0);
                }
            } else {
                put(std::integral_constant<int, FJ>(), [&](int i, int j) { return acc[i][j]; }, (uint8_t*)p.c, p.n, 0,
                    n0 + wn * FJ * 16);
            }
        }
    }
};

// Waves of a SIMD: workgroups a CU holds by their LDS, times a workgroup's waves.
template <class Tile>
constexpr int kWavesSimd = (Tile::LDS > 80 * 1024 ? 1 : 2) * Tile::NW / 4;

template <class Tile>
__global__ __launch_bounds__(Tile::NW * 64, kWavesSimd<Tile>) void mm_tile(MmParams p) {
    __shared__ __attribute__((aligned(1024))) uint8_t sm[Tile::LDS];
    Tile::run(p, sm, (int)blockIdx.x);
}

}  // namespace
}  // namespace coc
