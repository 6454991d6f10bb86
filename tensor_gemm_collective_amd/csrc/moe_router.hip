// MoE router: softmax, top-k selection, per-expert counts, send positions and
// the balance loss, and their gradient.
#include "row_ops.h"

namespace coc {
namespace {

constexpr int kMaxExperts = 512;
constexpr int kMaxTopk = 16;
constexpr int kPerLane = 8;     // experts a lane holds
constexpr int kThreads = 512;
constexpr int kChunk = 256;     // tokens a workgroup ranks at a time
constexpr int kWords = kChunk / 32;
constexpr int kMostBlocks = 256;

// exp(x) for x <= 0.  x log2(e) is split into its rounded product and what
// that rounding lost; exp2 takes the first, the second enters to first order.
__device__ __forceinline__ float exp_neg(float x) {
    constexpr float kLog2e = 1.44269504088896340736f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.693147180559945309417f;
    x = fmaxf(x, -200.0f);   // exp is 0 there; -inf would make the correction NaN
    const float hi = x * kLog2e;
    const float lo = fmaf(x, kLog2e, -hi) + x * kLog2eLow;
    const float e = __builtin_amdgcn_exp2f(hi);
    return fmaf(e * kLn2, lo, e);
}

// A lane's logits as binary32 (-inf past the last expert).  Lane l of a
// token's LG lanes holds experts [8 l, 8 l + 8).
template <class T>
__device__ __forceinline__ void load_logits(const T* row, int e0, int experts, float* x) {
    if (e0 + kPerLane <= experts) {
        load_n<kPerLane>(row, e0, experts, x);
    } else {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) x[i] = e0 + i < experts ? (float)row[e0 + i] : -INFINITY;
    }
}

// Unsigned order of logits: larger key, larger logit; every NaN above +inf,
// -inf and lower is key 0x007fffff, nothing (taken) is 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.0f);   // -0 orders as +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;

// Softmax of a token over its LG lanes: x becomes exp(x - max).  Returns
// whether the token takes part (its mask is set and a logit is above -inf).
template <int LG>
__device__ __forceinline__ bool softmax_parts(float* x, const uint32_t* key, bool live, float* total) {
    uint32_t mk = 0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) mk = max(mk, key[i]);
    mk = lanes_max<LG>(mk);
    live = live && mk > kKeyNegInf;
    const float top = __uint_as_float(mk & 0x80000000u ? mk ^ 0x80000000u : ~mk);   // NaN stays NaN
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        x[i] = !live ? 0.0f : x[i] == -INFINITY ? (top != top || top == INFINITY ? top - top : 0.0f)
                            : (x[i] != x[i] || top - top != 0.0f ? x[i] - top : exp_neg(x[i] - top));
        s += x[i];
    }
    *total = lanes_sum<LG>(s);
    return live;
}

// Where the parts of a launch are: the tokens of piece p are
// [tokens p / pieces, tokens (p + 1) / pieces), cut into `per` runs for as
// many workgroups, so that no workgroup's run crosses a piece.
struct Runs {
    int64_t tokens;
    int32_t pieces, per;
    __host__ __device__ int64_t piece_begin(int64_t p) const { return tokens * p / pieces; }
    __host__ __device__ int64_t begin(int b) const {
        const int64_t p = b / per, i = b % per, t0 = piece_begin(p);
        return t0 + (piece_begin(p + 1) - t0) * i / per;
    }
    __host__ __device__ int64_t end(int b) const {
        const int64_t p = b / per, i = b % per, t0 = piece_begin(p);
        return t0 + (piece_begin(p + 1) - t0) * (i + 1) / per;
    }
};

// Workgroup b routes its run.  Softmax and selection: LG lanes a token, k
// rounds of "largest key, lowest expert".  A chunk's choices go into a bit per
// (expert, token) in LDS; a choice's rank among its expert's is then the
// number of bits before it, whatever order the waves ran in.  Leaves each
// position's rank within the run, the run's counts (hist), probability sums
// and number of tokens that take part.
template <class T, int LG>
__global__ __launch_bounds__(kThreads) void route_runs(const T* logits, int64_t ld, const uint8_t* mask, Runs runs,
                                                       int experts, int topk, int renormalize, int32_t* ids,
                                                       float* gates, int32_t* positions, int32_t* hist, float* psum,
                                                       int32_t* nvalid) {
    constexpr int GROUPS = kThreads / LG;
    extern __shared__ uint32_t lds[];
    uint32_t* bits = lds;                                  // experts x kWords
    int32_t* seen = (int32_t*)(bits + experts * kWords);   // experts: choices of earlier chunks
    float* under = (float*)(seen + experts);               // kChunk: 1 / the gates' denominator
    int16_t* cid = (int16_t*)(under + kChunk);             // kChunk x topk
    float* cval = (float*)(cid + kChunk * kMaxTopk);       // kChunk x topk
    __shared__ int32_t taken;
    const int group = threadIdx.x / LG, lane = threadIdx.x % LG;
    const int e0 = lane * kPerLane;
    const int64_t t0 = runs.begin(blockIdx.x), t1 = runs.end(blockIdx.x);
    for (int e = threadIdx.x; e < experts; e += kThreads) seen[e] = 0;
    if (threadIdx.x == 0) taken = 0;
    float ps[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) ps[i] = 0.0f;
    int mine = 0;
    for (int64_t c0 = t0; c0 < t1; c0 += kChunk) {
        const int len = (int)min((int64_t)kChunk, t1 - c0);
        for (int i = threadIdx.x; i < experts * kWords; i += kThreads) bits[i] = 0;
        __syncthreads();
        for (int tl = group; tl < len; tl += GROUPS) {
            const int64_t t = c0 + tl;
            float x[kPerLane], total;
            uint32_t key[kPerLane];
            load_logits(logits + t * ld, e0, experts, x);
            bool live = !mask || mask[t] != 0;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) key[i] = e0 + i < experts ? order_key(x[i]) : 0;
            live = softmax_parts<LG>(x, key, live, &total);
            const float inv = live ? 1.0f / total : 0.0f;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) ps[i] += live ? x[i] * inv : 0.0f;
            if (lane == 0) mine += live;
            float chosen = 0.0f;
            for (int j = 0; j < topk; ++j) {
                uint32_t best = 0;
#pragma unroll
                for (int i = 0; i < kPerLane; ++i) best = max(best, key[i]);
                best = lanes_max<LG>(best);
                const bool any = live && best > kKeyNegInf;
                // the lowest expert with that key
                uint32_t at = 0;   // 0xffff - expert, so the lowest is the largest
                float v = 0.0f;
#pragma unroll
                for (int i = kPerLane - 1; i >= 0; --i)
                    if (key[i] == best) {
                        at = 0xffffu - (uint32_t)(e0 + i);
                        v = x[i];
                    }
                const uint32_t win = lanes_max<LG>(at);
                const int e = any ? (int)(0xffffu - win) : -1;
                const bool owner = any && at == win && at != 0;
                if (owner) {
                    cval[tl * topk + j] = v;
                    atomicOr(&bits[e * kWords + (tl >> 5)], 1u << (tl & 31));
                }
                if (lane == 0) {
                    cid[tl * topk + j] = (int16_t)e;
                    if (!any) cval[tl * topk + j] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < kPerLane; ++i)
                    if (e0 + i == e) key[i] = 0;
                chosen += lanes_sum<LG>(owner ? v : 0.0f);
            }
            if (lane == 0) under[tl] = renormalize ? chosen : total;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < len * topk; i += kThreads) {
            const int tl = i / topk;
            const int e = cid[i];
            int rank = -1;
            if (e >= 0) {
                rank = seen[e];
                for (int w = 0; w < (tl >> 5); ++w) rank += __popc(bits[e * kWords + w]);
                rank += __popc(bits[e * kWords + (tl >> 5)] & ((1u << (tl & 31)) - 1u));
            }
            const int64_t o = c0 * topk + i;
            ids[o] = e;
            gates[o] = e >= 0 ? cval[i] / under[tl] : 0.0f;
            positions[o] = rank;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < experts; e += kThreads) {
            int n = seen[e];
            for (int w = 0; w < kWords; ++w) n += __popc(bits[e * kWords + w]);
            seen[e] = n;
        }
        __syncthreads();
    }
    if (lane == 0 && mine) atomicAdd(&taken, mine);
    // probability sums: a wave's groups by shuffles, the waves in order
    float* wsum = (float*)bits;   // kThreads / 64 x experts: at most as large as bits
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        float v = ps[i];
#pragma unroll
        for (int d = LG; d < 64; d <<= 1) v += __shfl_xor(v, d);
        ps[i] = v;
    }
    __syncthreads();
    if ((threadIdx.x & 63) < LG) {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
            if (e0 + i < experts) wsum[(threadIdx.x >> 6) * experts + e0 + i] = ps[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += kThreads) {
        float s = 0.0f;
        for (int w = 0; w < kThreads / 64; ++w) s += wsum[w * experts + e];
        psum[(int64_t)blockIdx.x * experts + e] = s;
        hist[(int64_t)blockIdx.x * experts + e] = seen[e];
    }
    if (threadIdx.x == 0) nvalid[blockIdx.x] = taken;
}
static_assert(kThreads / 64 <= kWords, "the waves' sums fit where the bits were");

// One wave an expert: hist[b] becomes the choices of the piece's earlier runs;
// counts and probability sums.
__global__ __launch_bounds__(64) void scan_runs(int32_t* hist, const float* psum, Runs runs, int experts,
                                                int64_t* counts, float* prob_sums) {
    const int e = blockIdx.x, lane = threadIdx.x;
    float s = 0.0f;
    for (int p = 0; p < runs.pieces; ++p) {
        int32_t base = 0;
        for (int i = 0; i < runs.per; i += 64) {
            const bool in = i + lane < runs.per;
            const int64_t b = (int64_t)p * runs.per + i + lane;
            const int32_t v = in ? hist[b * experts + e] : 0;
            int32_t inc = v;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int32_t up = __shfl_up(inc, d);
                if (lane >= d) inc += up;
            }
            if (in) {
                hist[b * experts + e] = base + inc - v;
                s += psum[b * experts + e];
            }
            base += __shfl(inc, 63);
        }
        if (lane == 0) counts[(int64_t)p * experts + e] = base;
    }
    s = lanes_sum<64>(s);
    if (lane == 0) prob_sums[e] = s;
}

// Turns ranks within a run into send rows: first the rows of all (destination,
// piece, expert) before, from the counts, then the piece's earlier runs.
// Workgroup 0 also writes the loss and the number of tokens.
__global__ __launch_bounds__(256) void place_rows(const int32_t* ids, int32_t* positions, const int32_t* hist,
                                                  const int32_t* nvalid, int blocks, Runs runs, int experts,
                                                  int world, int topk,
                                                  const int64_t* counts, const float* prob_sums, float coef,
                                                  float* loss, int64_t* valid) {
    extern __shared__ uint32_t lds[];
    int32_t* first = (int32_t*)lds;   // experts: this piece's first row of each
    const int p = blockIdx.x / runs.per, local = experts / world;
    for (int e = threadIdx.x; e < experts && blocks > 0; e += 256) {
        const int dest = e / local;
        int64_t row = 0;
        for (int q = 0; q < runs.pieces; ++q)
            for (int f = 0; f < experts; ++f) {
                const int fd = f / local;
                if (fd < dest || (fd == dest && (q < p || (q == p && f < e)))) row += counts[(int64_t)q * experts + f];
            }
        first[e] = (int32_t)row + hist[(int64_t)blockIdx.x * experts + e];
    }
    __syncthreads();
    const int64_t i1 = runs.end(blockIdx.x) * topk;
    for (int64_t i = runs.begin(blockIdx.x) * topk + threadIdx.x; i < i1; i += 256) {
        const int e = ids[i];
        if (e >= 0) positions[i] += first[e];
    }
    if (blockIdx.x == 0 && threadIdx.x < 64) {
        int64_t n = 0;
        for (int b = threadIdx.x; b < blocks; b += 64) n += nvalid[b];
        float s = 0.0f;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) n += __shfl_xor((long long)n, d);
        for (int e = threadIdx.x; e < experts; e += 64) {
            int64_t c = 0;
            for (int q = 0; q < runs.pieces; ++q) c += counts[(int64_t)q * experts + e];
            s += (float)c / (float)(n > 0 ? n : 1) * (prob_sums[e] / (float)(n > 0 ? n : 1));
        }
        s = lanes_sum<64>(s);
        if (threadIdx.x == 0) {
            *valid = n;
            *loss = coef * (float)experts / (float)topk * s;
        }
    }
}

// dlogits = p (a - <p, a>) + the gates' term, a_e the loss's derivative by p_e
// with the counts held fixed, for LG lanes a token.
template <class T, int LG>
__global__ __launch_bounds__(kThreads) void route_backward(const T* logits, int64_t ld, const uint8_t* mask,
                                                           const int32_t* ids, const float* gates,
                                                           const int64_t* counts, const int64_t* valid,
                                                           const float* dgates, const float* dloss, T* dlogits,
                                                           int64_t ld_out, int64_t tokens, int experts, int pieces,
                                                           int topk, float coef, int renormalize) {
    constexpr int GROUPS = kThreads / LG;
    const int group = threadIdx.x / LG, lane = threadIdx.x % LG;
    const int e0 = lane * kPerLane;
    float a[kPerLane];
    const float n = (float)(valid[0] > 0 ? valid[0] : 1);
    const float w = dloss ? dloss[0] * coef * (float)experts / (float)topk / n / n : 0.0f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        int64_t c = 0;
        if (e0 + i < experts)
            for (int q = 0; q < pieces; ++q) c += counts[(int64_t)q * experts + e0 + i];
        a[i] = w * (float)c;
    }
    for (int64_t t = (int64_t)blockIdx.x * GROUPS + group; t < tokens; t += (int64_t)gridDim.x * GROUPS) {
        float x[kPerLane], total;
        uint32_t key[kPerLane];
        load_logits(logits + t * ld, e0, experts, x);
        bool live = !mask || mask[t] != 0;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) key[i] = e0 + i < experts ? order_key(x[i]) : 0;
        live = softmax_parts<LG>(x, key, live, &total);
        const float inv = live ? 1.0f / total : 0.0f;
        float pa = 0.0f;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            x[i] *= inv;
            pa += x[i] * a[i];
        }
        pa = lanes_sum<LG>(pa);
        float inner = 0.0f, add[kPerLane];
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) add[i] = 0.0f;
        if (dgates) {
            for (int j = 0; j < topk; ++j)
                if (ids[t * topk + j] >= 0) inner += gates[t * topk + j] * dgates[t * topk + j];
            for (int j = 0; j < topk; ++j) {
                const int e = ids[t * topk + j];
                if (e < 0) continue;
                const float g = gates[t * topk + j] * (dgates[t * topk + j] - (renormalize ? inner : 0.0f));
#pragma unroll
                for (int i = 0; i < kPerLane; ++i)
                    if (e0 + i == e) add[i] += g;
            }
        }
        const float off = pa + (renormalize ? 0.0f : inner);
        T* out = dlogits + t * ld_out;
        float o[kPerLane];
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) o[i] = live ? x[i] * (a[i] - off) + add[i] : 0.0f;
#pragma unroll
        for (int i = 0; i < kPerLane; i += kVec<T>) store_vec(out, e0 + i, experts, &o[i]);
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

template <class F>
void by_experts(int64_t experts, F&& f) {
    if (experts <= 8)
        f(std::integral_constant<int, 1>());
    else if (experts <= 16)
        f(std::integral_constant<int, 2>());
    else if (experts <= 32)
        f(std::integral_constant<int, 4>());
    else if (experts <= 64)
        f(std::integral_constant<int, 8>());
    else if (experts <= 128)
        f(std::integral_constant<int, 16>());
    else if (experts <= 256)
        f(std::integral_constant<int, 32>());
    else
        f(std::integral_constant<int, 64>());
}

Runs make_runs(int64_t tokens, int32_t pieces) {
    const int64_t longest = ceil_div(tokens, pieces);
    int64_t per = ceil_div(longest, 64);
    const int64_t most = kMostBlocks / pieces;
    if (per > most) per = most;
    if (per < 1) per = 1;
    return {tokens, pieces, (int32_t)per};
}

coc_status check_router(int64_t tokens, int32_t experts, int32_t topk, int32_t pieces, int64_t ld, coc_dtype dt) {
    if (!dtype_valid(dt)) return fail(COC_ERR_DTYPE, "unknown dtype %d", (int)dt);
    if (experts < 1 || experts > kMaxExperts)
        return fail(COC_ERR_SHAPE, "experts must be in [1, %d] (got %d)", kMaxExperts, experts);
    if (topk < 1 || topk > kMaxTopk || topk > experts)
        return fail(COC_ERR_SHAPE, "topk must be in [1, min(experts, %d)] (got %d)", kMaxTopk, topk);
    if (pieces < 1 || pieces > COC_MAX_SPLIT)
        return fail(COC_ERR_SPLIT, "pieces must be in [1, %d] (got %d)", COC_MAX_SPLIT, pieces);
    if (ld < experts) return fail(COC_ERR_SHAPE, "the logits' row stride is below the number of experts");
    coc_status s = check_matrix(tokens, ld, "the logits");
    if (s != COC_OK) return s;
    return check_matrix(tokens, topk, "ids");
}

}  // namespace
}  // namespace coc

extern "C" {

size_t coc_moe_router_workspace_bytes(int64_t tokens, int32_t experts, int32_t pieces) {
    if (tokens <= 0 || experts < 1 || experts > coc::kMaxExperts || pieces < 1 || pieces > COC_MAX_SPLIT) return 0;
    const coc::Runs r = coc::make_runs(tokens, pieces);
    return (size_t)r.pieces * (size_t)r.per * (size_t)(experts * 8 + 4);
}

coc_status coc_moe_router(const void* logits, int64_t ld, const uint8_t* mask, int32_t* ids, float* gates,
                          int32_t* positions, int64_t* counts, float* prob_sums, float* loss, int64_t* valid,
                          int64_t tokens, int32_t experts, int32_t topk, int32_t pieces, int32_t world, float coef,
                          int32_t renormalize, coc_dtype dt, void* ws, size_t ws_bytes, hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_router(tokens, experts, topk, pieces, ld, dt);
    if (st != COC_OK) return st;
    if (world < 1 || world > COC_MAX_WORLD || experts % world != 0)
        return fail(COC_ERR_WORLD, "world must be in [1, %d] and divide the experts (world=%d, experts=%d)",
                    COC_MAX_WORLD, world, experts);
    const size_t need = coc_moe_router_workspace_bytes(tokens, experts, pieces);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(COC_ERR_WORKSPACE, "the router needs %zu workspace bytes (got %zu)", need,
                    ws ? ws_bytes : (size_t)0);
    const int32_t es = (int32_t)elem_size(dt);
    const int64_t choices = tokens * topk * 4;
    const Arg args[] = {
        {logits, tokens > 0 ? ((tokens - 1) * ld + experts) * es : 0, es, false, "logits"},
        {mask, mask ? tokens : 0, 1, false, "mask"},
        {ids, choices, 4, true, "ids"},
        {gates, choices, 4, true, "gates"},
        {positions, choices, 4, true, "positions"},
        {counts, (int64_t)pieces * experts * 8, 8, true, "counts"},
        {prob_sums, (int64_t)experts * 4, 4, true, "prob_sums"},
        {loss, 4, 4, true, "loss"},
        {valid, 8, 8, true, "valid"},
        {ws, (int64_t)need, 4, true, "ws"},
    };
    st = check_args(args, 10);
    if (st != COC_OK) return st;
    // without tokens: no runs, zero counts and loss
    Runs runs = make_runs(tokens > 0 ? tokens : 1, pieces);
    runs.tokens = tokens;
    if (tokens == 0) runs.per = 0;
    const int blocks = runs.pieces * runs.per;
    int32_t* hist = (int32_t*)ws;
    float* psum = (float*)(hist + (int64_t)blocks * experts);
    int32_t* nvalid = (int32_t*)(psum + (int64_t)blocks * experts);
    if (blocks > 0) {
        const size_t lds = (size_t)experts * (kWords + 1) * 4 + kChunk * 4 + kChunk * kMaxTopk * 2 +
                           (size_t)kChunk * topk * 4;
        by_type(dt, [&](auto t) {
            using T = decltype(t);
            by_experts(experts, [&](auto lg) {
                route_runs<T, decltype(lg)::value><<<dim3(blocks), dim3(kThreads), lds, stream>>>(
                    (const T*)logits, ld, mask, runs, experts, topk, renormalize, ids, gates, positions, hist, psum,
                    nvalid);
            });
        });
        st = launched("router");
        if (st != COC_OK) return st;
    }
    scan_runs<<<dim3(experts), dim3(64), 0, stream>>>(hist, psum, runs, experts, counts, prob_sums);
    st = launched("router");
    if (st != COC_OK) return st;
    if (runs.per == 0) runs.per = 1;   // one workgroup without tokens writes the loss
    place_rows<<<dim3(blocks > 0 ? blocks : 1), dim3(256), (size_t)experts * 4, stream>>>(
        ids, positions, hist, nvalid, blocks, runs, experts, world, topk, counts, prob_sums, coef, loss, valid);
    return launched("router");
}

coc_status coc_moe_router_backward(const void* logits, int64_t ld, const uint8_t* mask, const int32_t* ids,
                                   const float* gates, const int64_t* counts, const int64_t* valid,
                                   const float* dgates, const float* dloss, void* dlogits, int64_t ld_out,
                                   int64_t tokens, int32_t experts, int32_t topk, int32_t pieces, float coef,
                                   int32_t renormalize, coc_dtype dt, hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_router(tokens, experts, topk, pieces, ld, dt);
    if (st != COC_OK) return st;
    if (ld_out < experts) return fail(COC_ERR_SHAPE, "the gradient's row stride is below the number of experts");
    st = check_matrix(tokens, ld_out, "the gradient");
    if (st != COC_OK) return st;
    if (tokens == 0) return COC_OK;
    const int32_t es = (int32_t)elem_size(dt);
    const int64_t choices = tokens * topk * 4;
    const Arg args[] = {
        {logits, ((tokens - 1) * ld + experts) * es, es, false, "logits"},
        {mask, mask ? tokens : 0, 1, false, "mask"},
        {ids, choices, 4, false, "ids"},
        {gates, choices, 4, false, "gates"},
        {counts, (int64_t)pieces * experts * 8, 8, false, "counts"},
        {valid, 8, 8, false, "valid"},
        {dgates, dgates ? choices : 0, 4, false, "dgates"},
        {dloss, dloss ? 4 : 0, 4, false, "dloss"},
        {dlogits, ((tokens - 1) * ld_out + experts) * es, es, true, "dlogits"},
    };
    st = check_args(args, 9);
    if (st != COC_OK) return st;
    by_type(dt, [&](auto t) {
        using T = decltype(t);
        by_experts(experts, [&](auto lg) {
            constexpr int LG = decltype(lg)::value;
            int64_t grid = ceil_div(tokens, kThreads / LG);
            if (grid > 2048) grid = 2048;
            route_backward<T, LG><<<dim3((uint32_t)grid), dim3(kThreads), 0, stream>>>(
                (const T*)logits, ld, mask, ids, gates, counts, valid, dgates, dloss, (T*)dlogits, ld_out, tokens,
                experts, pieces, topk, coef, renormalize);
        });
    });
    return launched("router backward");
}

}  // extern "C"
