// Matrix product of 8-bit floating-point operands with a scale for each block of 128:
//   y[i][j] = sum over blocks b of  xs[b][i] ws[j / 128][b]  sum over k in b of  x[i][k] w[j][k].
// x's scales cover 128 of a row, w's 128 x 128.
#include <algorithm>

#include "fp8.h"
#include "lds_tile.h"

namespace coc {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct Fp8Params {
    const uint8_t *x, *w;
    const float *xs, *ws;
    void* y;
    float* part;   // partial sums: splits x m x n
    int m, n, k, blocks;            // blocks: of 128 along k
    int tiles_m, tiles_n, stages;   // stages: blocks of one split
};

// A lane's 32 values of a fragment as the MFMAs take them: the bytes, or (WIDE) binary16,
// which holds every e4m3 value.
template <bool WIDE>
struct Values {
    i32x8 v;
    __device__ __forceinline__ void set(i32x8 bytes) { v = bytes; }
};
template <>
struct Values<true> {
    u32x4 v[4];
    __device__ __forceinline__ void set(i32x8 bytes) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i >> 1][(i & 1) * 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(bytes[i], 1.0f, false));
            v[i >> 1][(i & 1) * 2 + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(bytes[i], 1.0f, true));
        }
    }
};

// 128 k of 16 x 16 outputs.  The 8-bit MFMA adds each lane's products in groups of eight
// neighbouring k, in which bits below 2^-13 of the largest product's power of two are
// dropped (measured: a product 2^-13 of another is kept, one of 2^-14 is not, and beyond
// the group 2^-23 is), and then the groups in binary32.  A group is off by up to 8 x 2^-13 of
// its largest product.  Typical of normal data is 2e-5 of the result, a tenth of a rounding
// to binary16; at worst one 448 x 448 beside seven small products loses them all, 4e-4 of
// the sum, and where 448 x 448 - 448 x 448 cancels they were the result.  16-bit results are
// formed so all the same, for twice the rate (4096 x 7168 x 8192: 209 against 415 us);
// those in binary32 by 16-bit MFMAs, which hold every product whole.
__device__ __forceinline__ f32x4 mfma_block(const Values<false>& a, const Values<false>& b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_block(const Values<true>& a, const Values<true>& b) {
    f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < 4; ++q)
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a.v[q]), __builtin_bit_cast(f16x8, b.v[q]), c,
                                                   0, 0, 0);
    return c;
}

// One BM x BN tile.  A stage is one block of 128 k, so each MFMA gives a whole block's sum,
// which is scaled and added to the binary32 sums by the vector units (four multiply-adds
// for each MFMA, beside the other waves' MFMAs).  The weights are the MFMA's first
// operand: a lane then holds one row of x in each 16 x 16 block and needs one scale for
// it.  A lane's 32 k of a fragment are chunks g and g + 4 of a row (g: its 16-lane group)
// for both operands; the order of k within a block is free.
//
// 4096 x 7168 x 8192 (bf16 results) 206 to 216 us, 2.2 to 2.3 PFLOP/s; the same MFMAs with
// their multiply-adds and nothing else run at 3.6 on such operands.  It is bound by the
// clock and the LDS: on copies of the tile a third of the LDS reads took 172 of 217 us, no
// loads to LDS 193, one of the four multiply-adds 199.  Its steps there: sums and loads
// where the compiler put them 1272 us (the sums were all kept to a stage's end and spilled),
// in place 285, loads in two parts a stage 222, fragments read two blocks ahead and the
// upper rows' loads waited for later 212.
template <class T, bool WIDE, int FI, int FJ, int WM, int WN, int S, bool PART>
struct Fp8Tile {
    static constexpr int NW = WM * WN, BM = WM * FI * 16, BN = WN * FJ * 16, NB = BN / kScaleBlock;
    using A = Operand<BM, false, NW, 1>;
    using B = Operand<BN, false, NW, 1>;
    static constexpr int XW = BM > 64 ? BM / 64 : 1;   // waves that load x's scales; the others load w's
    static constexpr int SCALES = (XW + 1) * 256;      // bytes: 64 a wave
    static constexpr int SLOT = A::BYTES + B::BYTES;
    static constexpr int SCALE_SLOTS = S == 2 ? 4 : 8;   // they are read until a stage's end and loaded before it
    static constexpr int LDS = S * SLOT + SCALE_SLOTS * SCALES;
    static constexpr int DPW = A::PER_WAVE + B::PER_WAVE + 1;
    // whether a stage's loads go in two parts (see stage): with as many waves as row
    // blocks, load i of the rows is the lower half of the waves' blocks for even i
    static constexpr bool HALVES = FI == NW && S == 2;
    static constexpr int LATE = HALVES ? A::PER_WAVE / 2 : 0, EARLY = DPW - LATE;   // loads of each part
    static constexpr bool STAGED = !PART && sizeof(T) == 2;   // rows go out through the LDS
    static constexpr int RING = FI >= 4 ? 4 : 2, AHEAD = FI >= 4 ? 2 : 1;   // row fragments held, and read ahead
    static_assert(FI % RING == 0, "a block's place is the same in every stage");
    static_assert(BN % kScaleBlock == 0 && kScaleBlock % (FJ * 16) == 0, "a wave's columns share a scale");
    static_assert(XW < NW, "a wave for w's scales");
    static_assert(!STAGED || BM * BN * 2 <= LDS, "the staged output fits in the LDS");

    static __device__ __forceinline__ void run(const Fp8Params& p, uint8_t* sm) {
        int tm, tn;
        tile_of(blockIdx.x, p.tiles_m, p.tiles_n, &tm, &tn);
        const int m0 = tm * BM, n0 = tn * BN;
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int wm = wave / WN, wn = wave % WN;
        const uint32_t lds0 = lds_address(sm);
        const int stage0 = PART ? (int)blockIdx.y * p.stages : 0;
        const int KT = min(p.stages, p.blocks - stage0);   // >= 1

        A a;
        B b;
        a.init(p.x, p.k, stage0, lds0, wave, lane, [&](int r) { return min(m0 + r, p.m - 1); });
        b.init(p.w, p.k, stage0, lds0 + A::BYTES, wave, lane, [&](int c) { return min(n0 + c, p.n - 1); });
        // scales: 64 rows of x, or this tile's column blocks of w over and over
        const bool of_x = wave < XW;
        const uint32_t scale_off = 4u * (uint32_t)(of_x ? min(m0 + wave * 64 + lane, p.m - 1)
                                                        : min(n0 / kScaleBlock + lane % NB, (p.n - 1) / kScaleBlock) *
                                                              p.blocks);
        const int64_t scale_step = of_x ? (int64_t)p.m * 4 : 4;
        const uint8_t* scale_base = (const uint8_t*)(of_x ? p.xs : p.ws) + stage0 * scale_step;
        const uint32_t scale_lds = lds0 + S * SLOT + (of_x ? wave : XW) * 256;
        // load d of stage s: the columns, the rows (the even loads of them), the scales, the odd loads
        auto load = [&](int d, int s, int slot, auto WHOLE) {
            constexpr bool whole = decltype(WHOLE)::value;
            constexpr int NC = B::PER_WAVE, NR = A::PER_WAVE - LATE;
            const int left = p.k - (stage0 + s) * kScaleBlock;
            if (d < NC)
                b.template load<whole>(d, s, slot * SLOT, left);
            else if (d < NC + NR)
                a.template load<whole>(HALVES ? 2 * (d - NC) : d - NC, s, slot * SLOT, left);
            else if (d == NC + NR)
                load_lds4(scale_off, scale_base + s * scale_step,
                          __builtin_amdgcn_readfirstlane(scale_lds + (s & (SCALE_SLOTS - 1)) * SCALES));
            else
                a.template load<whole>(2 * (d - EARLY) + 1, s, slot * SLOT, left);
        };

        const int ra = wm * FI * 16 + (lane & 15), rb = wn * FJ * 16 + (lane & 15);
        int pa[2], pb[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            pa[h] = ra * 128 + (((h * 4 + (lane >> 4)) ^ row_swizzle(ra)) << 4);
            pb[h] = A::BYTES + rb * 128 + (((h * 4 + (lane >> 4)) ^ row_swizzle(rb)) << 4);
        }
        const COC_LDS uint8_t* lds = (const COC_LDS uint8_t*)sm;
        auto fragment = [&](int at0, int at1) {
            const u32x4 lo = *(const COC_LDS u32x4*)(lds + at0), hi = *(const COC_LDS u32x4*)(lds + at1);
            Values<WIDE> f;
            f.set(__builtin_shufflevector(__builtin_bit_cast(i32x4, lo), __builtin_bit_cast(i32x4, hi), 0, 1, 2, 3, 4, 5,
                                          6, 7));
            return f;
        };
        auto read_a = [&](int slot, int i) {
            return fragment(slot * SLOT + pa[0] + i * 2048, slot * SLOT + pa[1] + i * 2048);
        };
        auto read_b = [&](int slot, int j) {
            return fragment(slot * SLOT + pb[0] + j * 2048, slot * SLOT + pb[1] + j * 2048);
        };
        auto scales_at = [&](int kt) { return lds + S * SLOT + (kt & (SCALE_SLOTS - 1)) * SCALES; };
        auto read_scale = [&](int kt, int i) { return *(const COC_LDS float*)(scales_at(kt) + (ra + i * 16) * 4); };
        auto read_w_scale = [&](int kt) {
            return *(const COC_LDS float*)(scales_at(kt) + XW * 256 + (NB > 1 ? wn * FJ * 16 / kScaleBlock * 4 : 0));
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
            wait_loads<(S - 1) * DPW + LATE>();
        else
            wait_loads<0>();
        group_barrier();
        Values<WIDE> fa[RING], fb[FJ];
#pragma unroll
        for (int j = 0; j < FJ; ++j) fb[j] = read_b(0, j);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) fa[i] = read_a(0, i);

        // One stage.  A row block's fragment is read AHEAD blocks before its MFMAs.  As many
        // before the stage's end the workgroup meets (every wave has read this slot, and the
        // next stage has arrived); the next stage's first fragments are read then, and stage
        // kt + S is loaded into this slot.  HALVES: the workgroup also meets half a stage
        // before that.  The columns and the lower row blocks have been read by then, and
        // their places are loaded; the upper row blocks, loaded from the other meeting on,
        // need not have arrived before.  So every load has one and a half stages to arrive
        // in, and they do not come in one burst.
        auto stage = [&](int kt, int slot, auto MORE, auto LOAD, auto WHOLE, auto WAIT) {
            constexpr bool more = decltype(MORE)::value, loads = decltype(LOAD)::value;
            constexpr int N = FI * FJ, LAST = N - AHEAD * FJ, MEET = LAST - N / 2;
            constexpr int FROM = HALVES ? MEET : LAST, SPAN = HALVES ? LAST - MEET : AHEAD * FJ;   // of the early loads
            const int next = slot + 1 == S ? 0 : slot + 1;
            constexpr int BEHIND = FJ >= 4 ? 3 : 1;   // MFMAs between one and the adding of its sums
            f32x4 sum[BEHIND + 1];   // of the last MFMAs
            float sx[2];
            const float sw = read_w_scale(kt);
            sx[0] = read_scale(kt, 0);
            auto add = [&](int t) {
                const int i = t / FJ, j = t % FJ;
                const float s = sx[i & 1];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(sum[t % (BEHIND + 1)][e], s, acc[i][j][e]);
                asm volatile("" : "+v"(acc[i][j]));   // here, not at the end of the stage
            };
#pragma unroll
            for (int t = 0; t < N; ++t) {
                const int i = t / FJ, j = t % FJ;
                if (HALVES && t == MEET) {
                    wait_loads<decltype(WAIT)::value>();
                    group_barrier();
                }
                if (more && t == LAST) {
                    wait_loads<decltype(WAIT)::value>();
                    group_barrier();
                }
                sum[t % (BEHIND + 1)] = mfma_block(fb[j], fa[i % RING]);
                if (j == BEHIND) sx[i & 1] *= sw;   // the block's first sums come now
                if (t >= BEHIND) add(t - BEHIND);
                if (j + 1 == FJ && i + 1 < FI) sx[(i + 1) & 1] = read_scale(kt, i + 1);
                if (i + AHEAD < FI) {
                    if (j == 0) fa[(i + AHEAD) % RING] = read_a(slot, i + AHEAD);
                } else if (more) {
                    if (j == 0) fa[(i + AHEAD) % RING] = read_a(next, i + AHEAD - FI);
                }
                if (more && i + 1 == FI) fb[j] = read_b(next, j);
                if constexpr (loads) {
#pragma unroll
                    for (int d = 0; d < DPW; ++d)
                        if ((d < EARLY ? d * SPAN / EARLY + FROM : (d - EARLY) * AHEAD * FJ / (LATE > 0 ? LATE : 1) + LAST) == t)
                            load(d, kt + S, slot, WHOLE);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int t = N - BEHIND; t < N; ++t) add(t);
        };
        using yes = std::true_type;
        using no = std::false_type;
        int kt = 0, slot = 0;
        // in flight when the workgroup meets; HALVES: at either meeting, those issued since the
        // ones it needs, half a stage's and half a stage's
        using all = std::integral_constant<int, HALVES ? DPW : (S - 2) * DPW>;
        using none = std::integral_constant<int, 0>;
        auto step = [&] { slot = slot + 1 == S ? 0 : slot + 1; };
        // the last stage alone may be short of k
        for (; kt + S + 1 < KT; ++kt, step()) stage(kt, slot, yes(), yes(), yes(), all());
        if (kt + S < KT) {
            stage(kt, slot, yes(), yes(), no(), all());
            ++kt;
            step();
        }
        for (; kt + 1 < KT; ++kt, step()) stage(kt, slot, yes(), no(), no(), none());
        stage(kt, slot, no(), no(), no(), none());

        // A lane holds row l % 16 and columns 4 (l / 16) .. + 3 of each 16 x 16 block.
        if constexpr (!STAGED) {
            float* out = PART ? p.part + (int64_t)blockIdx.y * p.m * p.n : (float*)p.y;
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int j = 0; j < FJ; ++j) {
                    const int row = m0 + (wm * FI + i) * 16 + (lane & 15);
                    const int col = n0 + (wn * FJ + j) * 16 + (lane >> 4) * 4;
                    if (row < p.m) keep_n<4>(out + (int64_t)row * p.n, col, p.n, (const float*)&acc[i][j]);
                }
        } else {
            group_barrier();
            constexpr int PITCH = FJ * 32, CPR = FJ * 2, RPI = 64 / CPR;
            static_assert(64 % CPR == 0 && (FI * 16) % RPI == 0, "staging layout");
            COC_LDS uint8_t* stg = (COC_LDS uint8_t*)sm + wave * (FI * 16 * PITCH);
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int j = 0; j < FJ; ++j) {
                    const int row = i * 16 + (lane & 15), ch = j * 2 + (lane >> 5);
                    *(COC_LDS u32x2*)(stg + row * PITCH + ((ch ^ (row & (CPR - 1))) << 4) + ((lane >> 4) & 1) * 8) =
                        u32x2{round2<T>(acc[i][j][0], acc[i][j][1]), round2<T>(acc[i][j][2], acc[i][j][3])};
                }
#pragma unroll
            for (int t = 0; t < FI * 16 / RPI; ++t) {
                const int row = t * RPI + lane / CPR, ch = lane % CPR;
                const u32x4 v = *(const COC_LDS u32x4*)(stg + row * PITCH + ((ch ^ (row & (CPR - 1))) << 4));
                const int r = m0 + wm * FI * 16 + row, col = n0 + wn * FJ * 16 + ch * 8;
                Packed<T> o;
                __builtin_memcpy(o.w, &v, 16);
                if (r < p.m && col < p.n) keep_raw((T*)p.y + (int64_t)r * p.n, col, p.n, o);
            }
        }
    }

    // (stored normally: a product's result is read next)
    static __device__ __forceinline__ void keep_raw(T* row, int c, int n, const Packed<T>& o) {
        if (c + kVec<T> <= n)
            __builtin_memcpy(row + c, o.w, 16);
        else
            store_raw(row, c, n, o);
    }
};

template <class Tile, int THREADS, int PER_EU>
__global__ __launch_bounds__(THREADS, PER_EU) void fp8_tile(Fp8Params p) {
    __shared__ __attribute__((aligned(1024))) uint8_t sm[Tile::LDS];
    Tile::run(p, sm);
}

// Up to 16 rows: a pass over the weights.  A workgroup takes 16 FJ rows of w and all of k,
// its W waves every W-th block of 128 each, straight from memory into the MFMA's registers
// (a load instruction reads 64 bytes of each of 16 rows, four blocks are loaded together);
// the waves' sums are joined through the LDS, in order.
template <class T, bool WIDE, int FJ, int W>
__global__ __launch_bounds__(W * 64) void fp8_rows(Fp8Params p) {
    constexpr int U = 4;
    __shared__ float part[W][FJ][16][17];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * FJ, r = lane & 15, g = lane >> 4;
    const uint8_t* pw[FJ];
    const float* ws[FJ];
#pragma unroll
    for (int j = 0; j < FJ; ++j) {
        pw[j] = p.w + (int64_t)min(n0 + j * 16 + r, p.n - 1) * p.k + g * 16;
        ws[j] = p.ws + (int64_t)(min(n0 + j * 16, p.n - 1) / kScaleBlock) * p.blocks;
    }
    const int mine = min(r, p.m - 1);
    const uint8_t* px = p.x + (int64_t)mine * p.k + g * 16;
    const float* xs = p.xs + mine;
    f32x4 acc[FJ];
#pragma unroll
    for (int j = 0; j < FJ; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto take = [&](const uint8_t* at, int b, bool whole) {
        // this lane's chunks g and g + 4 of block b
        const int k = b * kScaleBlock + g * 16;
        u32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
        if (whole || k < p.k) lo = *(const u32x4*)(at + (int64_t)b * kScaleBlock);
        if (whole || k + 64 < p.k) hi = *(const u32x4*)(at + (int64_t)b * kScaleBlock + 64);
        return __builtin_shufflevector(__builtin_bit_cast(i32x4, lo), __builtin_bit_cast(i32x4, hi), 0, 1, 2, 3, 4, 5, 6,
                                       7);
    };
    auto blocks = [&](int b, auto COUNT, bool whole) {
        constexpr int C = decltype(COUNT)::value;
        i32x8 w[C][FJ], x[C];
        float sw[C][FJ], sx[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = b + c * W;
#pragma unroll
            for (int j = 0; j < FJ; ++j) w[c][j] = take(pw[j], at, whole);
            x[c] = take(px, at, whole);
#pragma unroll
            for (int j = 0; j < FJ; ++j) sw[c][j] = ws[j][at];
            sx[c] = xs[(int64_t)at * p.m];
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            Values<WIDE> vx;
            vx.set(x[c]);
#pragma unroll
            for (int j = 0; j < FJ; ++j) {
                Values<WIDE> vw;
                vw.set(w[c][j]);
                const f32x4 v = mfma_block(vw, vx);
                const float s = sw[c][j] * sx[c];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(v[e], s, acc[j][e]);
            }
        }
    };
    const int whole = p.k / kScaleBlock;
    int b = wave;
    for (; b + (U - 1) * W < whole; b += U * W) blocks(b, std::integral_constant<int, U>(), true);
    for (; b < p.blocks; b += W) blocks(b, std::integral_constant<int, 1>(), b < whole);
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[wave][j][r][g * 4 + e] = acc[j][e];
    __syncthreads();
    const int t = threadIdx.x;
    if (t >= FJ * 256) return;
    const int j = t >> 8, row = (t >> 4) & 15, col = t & 15, n = n0 + j * 16 + col;
    float v = part[0][j][row][col];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w][j][row][col];
    if (row < p.m && n < p.n) ((T*)p.y)[(int64_t)row * p.n + n] = (T)v;
}

// Adds the splits' sums in order.  Four columns a thread, U splits loaded together.
template <class T, int U>
__global__ __launch_bounds__(256) void fp8_join(const float* part, T* y, int64_t m, int n, int splits) {
    const int per_row = (n + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= m * per_row) return;
    const int64_t row = i / per_row;
    const int col = (int)(i - row * per_row) * 4;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = 0; s0 < splits; s0 += U) {
        float t[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u)   // past the last: the last again, not added
            load_vec(part + (min(s0 + u, splits - 1) * m + row) * n, col, n, t[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += s0 + u < splits ? t[u][e] : 0.0f;
    }
    keep_n<4>(y + row * n, col, n, v);
}

// The tiles, their stages of 128 k timed on products of 100 to 4000 rows.  Tiles of 32 rows
// always leave sums to join.  Binary32 results have no tile of 256 x 256: their 16-bit
// fragments do not fit its registers.
enum { kTile256, kTile128, kTile64, kTile32, kRows32, kRows16 };
constexpr TileCost kCosts[] = {
    {256, 256, 1, 1.25f, 1.65f, 4.0f, true, false},
    {128, 128, 2, 0.57f, 0.95f, 2.5f, true, true},
    {64, 128, 2, 0.36f, 0.66f, 1.5f, true, true},
    {32, 128, 2, 0.31f, 0.50f, 1.2f, false, true},
};
constexpr TileCost kWideCosts[] = {
    kCosts[kTile256],   // (not offered)
    {128, 128, 2, 1.05f, 1.85f, 3.0f, true, true},
    {64, 128, 2, 0.64f, 1.13f, 2.0f, true, true},
    {32, 128, 2, 0.49f, 0.85f, 1.5f, false, true},
};

// Up to 16 rows go straight from memory: 7168 x 8192, bf16, one row 12.1 us (a 16-row tile
// of split k and its join 14.0; 59 MB, 4.9 TB/s); with 16 weight rows a workgroup every one reads all of x,
// so from 5 rows on it takes 32 (8 rows 14.1 against 13.5 us, 16 rows 16.6 against 14.5, one
// row 12.1 against 13.0).
Choice choose(int64_t m, int64_t n, int64_t k, bool wide) {
    const int64_t stages = ceil_div(k, kScaleBlock);
    if (m <= 16) return {m <= 4 ? kRows16 : kRows32, 0, 1, false, 0.0f};
    const TileCost* costs = wide ? kWideCosts : kCosts;
    if (m <= 32) {
        const TileCost few[] = {costs[kTile64], costs[kTile32]};
        Choice c = pick(few, m, n, stages);
        c.tile += kTile64;
        return c;
    }
    if (wide) {
        const TileCost some[] = {costs[kTile128], costs[kTile64]};
        Choice c = pick(some, m, n, stages);
        c.tile += kTile128;
        return c;
    }
    const TileCost all[] = {costs[kTile256], costs[kTile128], costs[kTile64]};
    return pick(all, m, n, stages);
}

size_t part_bytes(int64_t m, int64_t n, int64_t k, bool wide) {
    const Choice c = choose(m, n, k, wide);
    return c.split ? (size_t)(c.splits * m * n * 4) : 0;
}

template <class Tile, int THREADS, int PER_EU>
void launch_tile(Fp8Params p, const Choice& c, hipStream_t stream) {
    p.tiles_m = (int)ceil_div(p.m, Tile::BM);
    p.tiles_n = (int)ceil_div(p.n, Tile::BN);
    p.stages = c.stages;
    fp8_tile<Tile, THREADS, PER_EU>
        <<<dim3((uint32_t)(p.tiles_m * p.tiles_n), (uint32_t)c.splits), dim3(THREADS), 0, stream>>>(p);
}

coc_status check_product(int64_t m, int64_t n, int64_t k, coc_dtype dt) {
    if (!dtype_valid(dt)) return fail(COC_ERR_DTYPE, "unknown dtype %d", (int)dt);
    if (k < 0 || k % 16 != 0) return fail(COC_ERR_SHAPE, "k is a multiple of 16 (k=%lld)", (long long)k);
    coc_status st = check_matrix(m, k, "x");
    if (st == COC_OK) st = check_matrix(n, k, "w");
    if (st == COC_OK) st = check_matrix(m, n, "y");
    return st;
}

template <class T>
__global__ __launch_bounds__(256) void fp8_zeros(T* y, int64_t count) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < count) y[i] = (T)0.0f;
}

}  // namespace
}  // namespace coc

extern "C" {

size_t coc_matmul_fp8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (m <= 0 || n <= 0 || k <= 0 || coc::check_product(m, n, k, COC_F32) != COC_OK) return 0;
    return std::max(coc::part_bytes(m, n, k, false), coc::part_bytes(m, n, k, true));
}

coc_status coc_matmul_fp8(const void* x, const float* x_scales, const void* w, const float* w_scales, void* y,
                          int64_t m, int64_t n, int64_t k, coc_dtype dt, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_product(m, n, k, dt);
    if (st != COC_OK) return st;
    if (m == 0 || n == 0) return COC_OK;
    const size_t need = coc_matmul_fp8_workspace_bytes(m, n, k);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(COC_ERR_WORKSPACE, "matmul_fp8 needs %zu workspace bytes (got %zu)", need,
                    ws ? ws_bytes : (size_t)0);
    const int32_t es = (int32_t)elem_size(dt);
    const int64_t blocks = ceil_div(k, kScaleBlock);
    const Arg args[] = {{x, m * k, 16, false, "x"},
                        {x_scales, blocks * m * 4, 4, false, "x_scales"},
                        {w, n * k, 16, false, "w"},
                        {w_scales, ceil_div(n, kScaleBlock) * blocks * 4, 4, false, "w_scales"},
                        {y, m * n * es, es, true, "y"},
                        {ws, (int64_t)need, 16, true, "ws"}};
    st = check_args(args, 6);
    if (st != COC_OK) return st;
    auto by_out = [&](auto&& f) {
        if (dt == COC_F32)
            f(float());
        else if (dt == COC_F16)
            f(f16_t());
        else
            f(bf16_t());
    };
    if (k == 0) {
        by_out([&](auto t) {
            using T = decltype(t);
            fp8_zeros<T><<<dim3((uint32_t)ceil_div(m * n, 256)), dim3(256), 0, stream>>>((T*)y, m * n);
        });
        return launched("matmul_fp8");
    }
    Fp8Params p{};
    p.x = (const uint8_t*)x;
    p.w = (const uint8_t*)w;
    p.xs = x_scales;
    p.ws = w_scales;
    p.y = y;
    p.part = (float*)ws;
    p.m = (int)m;
    p.n = (int)n;
    p.k = (int)k;
    p.blocks = (int)blocks;
    const Choice c = choose(m, n, k, dt == COC_F32);
    auto go = [&](auto t, auto wide) {
        using T = decltype(t);
        constexpr bool WIDE = decltype(wide)::value;
        switch (c.tile) {
            case kTile256:
                if constexpr (!WIDE) launch_tile<Fp8Tile<T, WIDE, 8, 4, 2, 4, 2, false>, 512, 2>(p, c, stream);
                break;
            case kTile128:
                if (c.split)
                    launch_tile<Fp8Tile<float, WIDE, 4, 4, 2, 2, 2, true>, 256, 2>(p, c, stream);
                else
                    launch_tile<Fp8Tile<T, WIDE, 4, 4, 2, 2, 2, false>, 256, 2>(p, c, stream);
                break;
            case kTile64:
                if (c.split)
                    launch_tile<Fp8Tile<float, WIDE, 2, 2, 2, 4, 3, true>, 512, 4>(p, c, stream);
                else
                    launch_tile<Fp8Tile<T, WIDE, 2, 2, 2, 4, 3, false>, 512, 4>(p, c, stream);
                break;
            case kTile32: launch_tile<Fp8Tile<float, WIDE, 2, 2, 1, 4, 3, true>, 256, 2>(p, c, stream); break;
            case kRows32: fp8_rows<T, WIDE, 2, 16><<<dim3((uint32_t)ceil_div(n, 32)), dim3(1024), 0, stream>>>(p); break;
            default: fp8_rows<T, WIDE, 1, 8><<<dim3((uint32_t)ceil_div(n, 16)), dim3(512), 0, stream>>>(p); break;
        }
    };
    if (dt == COC_F32)
        go(float(), std::true_type());
    else if (dt == COC_F16)
        go(f16_t(), std::false_type());
    else
        go(bf16_t(), std::false_type());
    st = launched("matmul_fp8");
    if (st != COC_OK || !c.split) return st;
    by_out([&](auto t) {
        using T = decltype(t);
        by_splits(c.splits, [&](auto u) {
            fp8_join<T, decltype(u)::value><<<dim3((uint32_t)ceil_div(m * ceil_div(n, 4), 256)), dim3(256), 0, stream>>>(
                (const float*)ws, (T*)y, m, (int)n, c.splits);
        });
    });
    return launched("matmul_fp8 join");
}

}  // extern "C"
