// The gated feed-forward block in 16 bits: h = act(x Wg) * (x Wu), and its backward
// pass.  The gate and up weights are one d x 2f matrix, as the column-parallel matmul
// takes them.
//
// The backward pass rounds the projections' gradient to 16 bits, as both products' operand:
// an error of one rounding of each term, so that dx and dw are off by about 1.4 times their
// own rounding.  In 32 bits it would take twice the products' time.
#include "mm_tile.h"

namespace coc {
namespace {

// ------------------------------------------------------------------ joining split sums
// One token through 8192 x 7168 (bf16, 117 MB): 23 us for the split tiles, 5.1 TB/s, and 4
// for the join.  Tiles of 16 columns and all of k, which need no join, took 52 to 60 us:
// their loads are of 32 neighbouring bytes.
//
// Adds the splits' sums in order: h and gate_up (either may be NULL) of the gated
// product, or the plain product's result.  Four columns a thread, U splits loaded together.
template <class T, bool GATED, int U>
__global__ __launch_bounds__(256) void mm_join(const float* part, T* c, T* gate_up, int64_t m, int n, int splits,
                                               int act) {
    const int per_row = n / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= m * per_row) return;
    const int64_t row = i / per_row;
    const int col = (int)(i - row * per_row) * 4;
    const int64_t all = GATED ? 2 * n : n;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f}, u = v;
    for (int s0 = 0; s0 < splits; s0 += U) {
        f32x4 g[U], w[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {   // past the last: the last again, not added
            const float* p = part + (min(s0 + k, splits - 1) * m + row) * all + col;
            g[k] = *(const f32x4*)p;
            if (GATED) w[k] = *(const f32x4*)(p + n);
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (s0 + k < splits) {
                v += g[k];
                if (GATED) u += w[k];
            }
    }
    auto put = [&](T* at, f32x4 o) { *(u32x2*)at = u32x2{round2<T>(o[0], o[1]), round2<T>(o[2], o[3])}; };
    if constexpr (GATED) {
        if (gate_up) {
            put(gate_up + row * 2 * n + col, v);
            put(gate_up + row * 2 * n + n + col, u);
        }
        if (!c) return;
        by_act((coc_act)act, [&](auto a) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = act_value<decltype(a)::value>(v[e]) * u[e];
        });
    }
    put(c + row * n + col, v);
}

template <class T>
__global__ __launch_bounds__(256) void fill_zeros(T* p, int64_t vectors) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < vectors) *(u32x4*)(p + i * 8) = u32x4{0, 0, 0, 0};
}

// ------------------------------------------------------------------ which tile
// The tiles, their stages of 64 k timed on products of 100 to 1500 rows.  The largest reads
// its operands least often.  128 x 128 comes with four slots, one workgroup a CU, for
// products of few tiles, and with two slots and two workgroups a CU.
//
// What the small tiles (24 KB a stage of 64 x 128) are bound by is not one thing: six slots for
// three, waves that share a stage's k and read a third less from the LDS, half the LDS reads, no
// barriers and loads that keep their lines in the L1 all took the same time (non-temporal ones up
// to 1.8 times it); on a copy whose loads all hit the L2 1024 x 2048 x 4096 took 27 of 28 us, 3313
// x 304 x 4056 24 of 29 and 128 x 7168 x 8192, unsplit, 41 of 81; with no loads 17, 16 and 27.
enum { kTile256, kTile128Deep, kTile128, kTile64, kTile32 };
constexpr TileCost kCosts[] = {
    {256, 256, 1, 1.35f, 1.50f, 6.0f, true, false}, {128, 128, 1, 0.55f, 0.55f, 3.0f, true, false},
    {128, 128, 2, 0.84f, 0.94f, 3.0f, true, true},  {64, 128, 2, 0.38f, 0.80f, 2.0f, true, true},
    {32, 128, 2, 0.40f, 0.60f, 1.5f, true, true},
};

// m x n outputs (n: f of the gated product, whose tiles hold twice as many columns of B).
// Up to 32 rows take a tile of as few (one row through 8192 x 7168 26.2 us, by 64 x 128 26.9;
// 16 rows 27.9 and 28.1; a tile of 16 rows took the same).  ta: A is stored k-major.
Choice choose(int64_t m, int64_t n, int64_t k, bool gated, bool ta) {
    const int64_t cols = gated ? 2 * n : n, stages = ceil_div(k, 64);
    if (m > 32 || ta) {
        constexpr TileCost large[] = {kCosts[0], kCosts[1], kCosts[2], kCosts[3]};
        return pick(large, m, cols, stages);
    }
    constexpr TileCost few[] = {kCosts[kTile32]};
    Choice c = pick(few, m, cols, stages);
    c.tile = kTile32;
    return c;
}

size_t part_bytes(int64_t m, int64_t n, int64_t k, bool gated, bool ta = false) {
    const Choice c = choose(m, n, k, gated, ta);
    return c.split ? (size_t)(c.splits * m * (gated ? 2 * n : n) * 4) : 0;
}

template <class Tile>
void launch_tile(MmParams p, const Choice& c, hipStream_t stream) {
    p.tiles_m = (int)ceil_div(p.m, Tile::BM);
    p.tiles_n = (int)ceil_div(p.n, Tile::OUT);
    p.stages = c.stages;
    mm_tile<Tile><<<dim3((uint32_t)(p.tiles_m * p.tiles_n), (uint32_t)c.splits), dim3(Tile::NW * 64), 0, stream>>>(p);
}

// C = A B of these sizes by the chosen tile, joined where it is split.
template <class T, bool TA, bool TB, bool GATED>
coc_status product(MmParams p, const Choice& c, hipStream_t stream) {
    switch (c.tile) {
        case kTile256: launch_tile<MmTile<T, TA, TB, 8, 4, 2, 4, 2, GATED, false>>(p, c, stream); break;
        case kTile128Deep: launch_tile<MmTile<T, TA, TB, 4, 2, 2, 4, 4, GATED, false>>(p, c, stream); break;
        case kTile128:
            if (c.split)
                launch_tile<MmTile<T, TA, TB, 4, 4, 2, 2, 2, GATED, true>>(p, c, stream);
            else
                launch_tile<MmTile<T, TA, TB, 4, 4, 2, 2, 2, GATED, false>>(p, c, stream);
            break;
        case kTile64:
            if (c.split)
                launch_tile<MmTile<T, TA, TB, 2, 2, 2, 4, 3, GATED, true>>(p, c, stream);
            else
                launch_tile<MmTile<T, TA, TB, 2, 2, 2, 4, 3, GATED, false>>(p, c, stream);
            break;
        default:
            if constexpr (!TA) {
                if (c.split)
                    launch_tile<MmTile<T, TA, TB, 2, 2, 1, 4, 4, GATED, true>>(p, c, stream);
                else
                    launch_tile<MmTile<T, TA, TB, 2, 2, 1, 4, 4, GATED, false>>(p, c, stream);
            }
            break;
    }
    coc_status st = launched("gated feed-forward product");
    if (st != COC_OK || !c.split) return st;
    by_splits(c.splits, [&](auto u) {
        mm_join<T, GATED, decltype(u)::value>
            <<<dim3((uint32_t)ceil_div((int64_t)p.m * (p.n / 4), 256)), dim3(256), 0, stream>>>(
                p.part, (T*)p.c, (T*)p.gate_up, p.m, p.n, c.splits, p.act);
    });
    return launched("gated feed-forward join");
}

// The backward pass's two products, dx (m x d over 2f) and dw (d x 2f over m), in one
// launch of the same tile: their workgroups fill the rounds together, where each alone
// leaves a round partly empty, and a small pass is spared a launch.  The longer tiles go
// first.  With the activation's gradient, 4096 x 8192 x 7168: 756 us (one by one 767); 2659 x
// 6416 x 2880, whose 286 and 312 tiles take two rounds each alone: 203 (244).
template <class X, class W>
__global__ __launch_bounds__(X::NW * 64, kWavesSimd<X>) void mm_pair(MmParams x, MmParams w, int x0, int w0) {
    static_assert(X::NW == W::NW && X::LDS == W::LDS, "one launch for both");
    __shared__ __attribute__((aligned(1024))) uint8_t sm[X::LDS];
    const int b = (int)blockIdx.x;
    if (b >= x0 && (x0 >= w0 || b < w0))
        X::run(x, sm, b - x0);
    else
        W::run(w, sm, b - w0);
}

struct Pair {
    int tile;   // -1: each by itself
    float us;
};
Pair choose_pair(int64_t m, int64_t d, int64_t f) {
    const int64_t sx = ceil_div(2 * f, 64), sw = ceil_div(m, 64);
    Pair best{-1, choose(m, d, 2 * f, false, false).us + choose(d, 2 * f, m, false, true).us + 4.0f};
    for (int t : {kTile256, kTile128Deep, kTile128, kTile64}) {
        const TileCost& c = kCosts[t];
        const int64_t tx = ceil_div(m, c.rows) * ceil_div(d, c.cols), tw = ceil_div(d, c.rows) * ceil_div(2 * f, c.cols);
        const int64_t slots = kCus * c.per_cu;
        const float stage = tx + tw <= kCus ? c.light : c.full;
        // evenly shared, but for the last tiles' half; at least the longest tile
        const float longest = (float)(sx > sw ? sx : sw) * stage + c.ends;
        float us = ((float)(tx * sx + tw * sw) * stage + (float)(tx + tw) * c.ends) / (float)slots;
        us = tx + tw <= slots ? longest : us + 0.5f * ((float)(sx < sw ? sx : sw) * stage + c.ends);
        if (us < longest) us = longest;
        if (us < best.us) best = {t, us};
    }
    return best;
}

// One of them alone takes the tile without a split too, so that it has the same bits (each
// output adds its products in the order of k, whatever the tile; a split adds sums).
Choice unsplit(int64_t m, int64_t n, int64_t k) {
    TileCost whole[4];
    for (int t = 0; t < 4; ++t) {
        whole[t] = kCosts[t];
        whole[t].split = false;
    }
    return pick(whole, m, n, ceil_div(k, 64));
}

template <class X, class W>
void launch_pair(MmParams x, MmParams w, hipStream_t stream) {
    for (MmParams* p : {&x, &w}) {
        p->tiles_m = (int)ceil_div(p->m, X::BM);
        p->tiles_n = (int)ceil_div(p->n, X::BN);
        p->stages = (int)ceil_div(p->k, 64);
    }
    const int tx = x.tiles_m * x.tiles_n, tw = w.tiles_m * w.tiles_n;
    const bool x_first = x.stages >= w.stages;
    mm_pair<X, W><<<dim3((uint32_t)(tx + tw)), dim3(X::NW * 64), 0, stream>>>(x, w, x_first ? 0 : tw, x_first ? tx : 0);
}

template <class T>
coc_status product_pair(int tile, const MmParams& x, const MmParams& w, hipStream_t stream) {
    switch (tile) {
        case kTile256:
            launch_pair<MmTile<T, false, true, 8, 4, 2, 4, 2, false, false>, MmTile<T, true, false, 8, 4, 2, 4, 2, false, false>>(x, w, stream);
            break;
        case kTile128Deep:
            launch_pair<MmTile<T, false, true, 4, 2, 2, 4, 4, false, false>, MmTile<T, true, false, 4, 2, 2, 4, 4, false, false>>(x, w, stream);
            break;
        case kTile128:
            launch_pair<MmTile<T, false, true, 4, 4, 2, 2, 2, false, false>, MmTile<T, true, false, 4, 4, 2, 2, 2, false, false>>(x, w, stream);
            break;
        default:
            launch_pair<MmTile<T, false, true, 2, 2, 2, 4, 3, false, false>, MmTile<T, true, false, 2, 2, 2, 4, 3, false, false>>(x, w, stream);
            break;
    }
    return launched("gated feed-forward backward");
}

template <class F>
coc_status by_type16(coc_dtype dt, F&& f) {
    return dt == COC_F16 ? f(f16_t()) : f(bf16_t());
}

coc_status check_ffn(int64_t m, int64_t d, int64_t f, coc_act act, coc_dtype dt) {
    if (dt != COC_BF16 && dt != COC_F16) return fail(COC_ERR_DTYPE, "gated feed-forward: bf16 or fp16 only");
    if (act != COC_ACT_SILU && act != COC_ACT_GELU) return fail(COC_ERR_DTYPE, "unknown activation %d", (int)act);
    if (d < 8 || f < 8 || d % 8 != 0 || f % 8 != 0)
        return fail(COC_ERR_SHAPE, "d and f are positive multiples of 8 (d=%lld f=%lld)", (long long)d, (long long)f);
    const int64_t lim = int64_t(1) << 31;
    if (d >= lim || f >= lim / 2) return fail(COC_ERR_SHAPE, "w has 2^31 or more elements");
    coc_status st = check_matrix(m, d, "x");
    if (st == COC_OK) st = check_matrix(m, 2 * f, "gate_up");
    if (st == COC_OK) st = check_matrix(d, 2 * f, "w");
    return st;
}

MmParams operands(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t m, int64_t n, int64_t k) {
    MmParams p{};
    p.a = a;
    p.b = b;
    p.lda = lda;
    p.ldb = ldb;
    p.m = (int)m;
    p.n = (int)n;
    p.k = (int)k;
    return p;
}

coc_status gated_product(const void* x, const void* w, void* h, void* gate_up, int64_t m, int64_t d, int64_t f,
                         coc_act act, coc_dtype dt, void* part, hipStream_t stream) {
    MmParams p = operands(x, d, w, 2 * f, m, f, d);
    p.c = h;
    p.gate_up = gate_up;
    p.act = act;
    p.part = (float*)part;
    return by_type16(dt, [&](auto t) { return product<decltype(t), false, false, true>(p, choose(m, f, d, true, false), stream); });
}

struct BackwardSpace {
    size_t dgate_up, part;   // bytes: the projections' gradient, then the products' split sums
    BackwardSpace(int64_t m, int64_t d, int64_t f) {
        dgate_up = (size_t)round_up(m * 2 * f * 2, 256);
        const size_t a = part_bytes(m, f, d, true), b = part_bytes(m, d, 2 * f, false),
                     c = part_bytes(d, 2 * f, m, false, true);
        part = a > b ? (a > c ? a : c) : (b > c ? b : c);
    }
};

}  // namespace
}  // namespace coc

extern "C" {

size_t coc_gated_ffn_workspace_bytes(int64_t m, int64_t d, int64_t f) {
    if (m <= 0 || coc::check_ffn(m, d, f, COC_ACT_SILU, COC_BF16) != COC_OK) return 0;
    return coc::part_bytes(m, f, d, true);
}

coc_status coc_gated_ffn(const void* x, const void* w, void* h, void* gate_up, int64_t m, int64_t d, int64_t f,
                         coc_act act, coc_dtype dt, void* ws, size_t ws_bytes, hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_ffn(m, d, f, act, dt);
    if (st != COC_OK) return st;
    if (m == 0) return COC_OK;
    const size_t need = part_bytes(m, f, d, true);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(COC_ERR_WORKSPACE, "gated feed-forward needs %zu workspace bytes (got %zu)", need,
                    ws ? ws_bytes : (size_t)0);
    const Arg args[] = {{x, m * d * 2, 16, false, "x"},
                        {w, d * 2 * f * 2, 16, false, "w"},
                        {h, m * f * 2, 16, true, "h"},
                        {gate_up, gate_up ? m * 2 * f * 2 : 0, 16, true, "gate_up"},
                        {ws, (int64_t)need, 16, true, "ws"}};
    st = check_args(args, 5);
    if (st != COC_OK) return st;
    return gated_product(x, w, h, gate_up, m, d, f, act, dt, ws, stream);
}

size_t coc_gated_ffn_backward_workspace_bytes(int64_t m, int64_t d, int64_t f) {
    if (m <= 0 || coc::check_ffn(m, d, f, COC_ACT_SILU, COC_BF16) != COC_OK) return 0;
    const coc::BackwardSpace s(m, d, f);
    return s.dgate_up + s.part;
}

coc_status coc_gated_ffn_backward(const void* dh, const void* x, const void* w, const void* gate_up, void* dx, void* dw,
                                  int64_t m, int64_t d, int64_t f, coc_act act, coc_dtype dt, void* ws,
                                  size_t ws_bytes, hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_ffn(m, d, f, act, dt);
    if (st != COC_OK) return st;
    const size_t need = coc_gated_ffn_backward_workspace_bytes(m, d, f);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(COC_ERR_WORKSPACE, "gated feed-forward backward needs %zu workspace bytes (got %zu)", need,
                    ws ? ws_bytes : (size_t)0);
    const int64_t weights = d * 2 * f * 2;
    const Arg args[] = {{dh, m * f * 2, 16, false, "dh"},
                        {x, m * d * 2, 16, false, "x"},
                        {w, weights, 16, false, "w"},
                        {gate_up, gate_up ? m * 2 * f * 2 : 0, 16, false, "gate_up"},
                        {dx, dx ? m * d * 2 : 0, 16, true, "dx"},
                        {dw, dw ? weights : 0, 16, true, "dw"},
                        {ws, (int64_t)need, 16, true, "ws"}};
    st = check_args(args, 7);
    if (st != COC_OK) return st;
    if (m == 0) {
        // no rows: the weights' gradient is 0
        if (!dw) return COC_OK;
        fill_zeros<uint16_t><<<dim3((uint32_t)ceil_div(weights / 16, 256)), dim3(256), 0, stream>>>((uint16_t*)dw,
                                                                                                 weights / 16);
        return launched("gated feed-forward backward");
    }
    if (!dx && !dw) return COC_OK;
    const BackwardSpace space(m, d, f);
    void* const dgu = ws;
    void* const part = (uint8_t*)ws + space.dgate_up;
    if (!gate_up) {
        // the projections again, where their gradient will be
        st = gated_product(x, w, nullptr, dgu, m, d, f, act, dt, part, stream);
        if (st != COC_OK) return st;
    }
    launch_gated_act_backward(dh, gate_up ? gate_up : dgu, dgu, m, f, act, dt, stream);
    st = launched("gated feed-forward backward");
    if (st != COC_OK) return st;
    return by_type16(dt, [&](auto t) {
        using T = decltype(t);
        MmParams x_ = operands(dgu, 2 * f, w, 2 * f, m, d, 2 * f), w_ = operands(x, d, dgu, 2 * f, d, 2 * f, m);
        x_.c = dx;
        w_.c = dw;
        x_.part = w_.part = (float*)part;
        const Pair pair = choose_pair(m, d, f);
        const bool whole = pair.tile >= 0;
        if (whole && dx && dw) return product_pair<T>(pair.tile, x_, w_, stream);
        coc_status s = COC_OK;
        if (dx)
            s = product<T, false, true, false>(x_, whole ? unsplit(m, d, 2 * f) : choose(m, d, 2 * f, false, false),
                                               stream);
        if (s == COC_OK && dw)
            s = product<T, true, false, false>(w_, whole ? unsplit(d, 2 * f, m) : choose(d, 2 * f, m, false, true),
                                               stream);
        return s;
    });
}

}  // extern "C"
