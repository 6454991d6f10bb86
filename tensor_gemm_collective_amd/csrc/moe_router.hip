// MoE router: softmax, top-k selection, per-expert counts, send positions and
// the balance loss, and their gradient.
#include "row_ops.h"

namespace coc {
namespace {

constexpr int kMaxExperts = 512;
constexpr int kMaxTopk = 16;
constexpr int kPerLane = 8;         // experts a lane holds
// Threads of a forward workgroup, and the most workgroups (runs): 65536 x 128 top 8
// 28.7 us; 256 threads of 1024 workgroups 32.5, 1024 of 256 30.2.
constexpr int kThreads = 512;
constexpr int kMostBlocks = 512;
constexpr int kLeastRun = 32;       // tokens of a run
constexpr int kAlone = 1024;        // threads of the workgroup that routes alone
constexpr int kChunk = 256;         // tokens a workgroup ranks at a time
constexpr int kWords = kChunk / 32;

constexpr float kLog2e = 1.44269504088896340736f;

// A choice's key: the logit's bits in unsigned order above 0xffff - expert, so
// that keys differ and the largest is the largest logit's lowest expert.  16
// bits hold a 16-bit logit's order, 32 a binary32's.  Every NaN orders above
// +inf, -0 as +0; a key at or below kNone stands for no choice (-inf, or 0
// for what is not there or has been taken).
template <class T>
struct Order {
    typedef uint32_t Key;
    static constexpr uint32_t kNegInf = std::is_same_v<T, bf16_t> ? 0x007fu : 0x03ffu;
    // x holds a T exactly: its bits are the upper half of a bfloat16's binary32
    __device__ static uint32_t high(float x) {
        if constexpr (std::is_same_v<T, bf16_t>) return __float_as_uint(x);
        return (uint32_t)__builtin_bit_cast(uint16_t, (T)x) << 16;
    }
    __device__ static float value(uint32_t b) { return (float)__builtin_bit_cast(T, (uint16_t)(b >> 16)); }
    __device__ static Key key(uint32_t o, uint32_t e) { return (o & 0xffff0000u) | (0xffffu - e); }
    __device__ static uint32_t order(Key k) { return k & 0xffff0000u; }
};
template <>
struct Order<float> {
    typedef uint64_t Key;
    static constexpr uint32_t kNegInf = 0x007fffffu;
    __device__ static uint32_t high(float x) { return __float_as_uint(x); }
    __device__ static float value(uint32_t b) { return __uint_as_float(b); }
    __device__ static Key key(uint32_t o, uint32_t e) { return (uint64_t)o << 16 | (0xffffu - e); }
    __device__ static uint32_t order(Key k) { return (uint32_t)(k >> 16); }
};
template <class T>
using Key = typename Order<T>::Key;
template <class T>
constexpr Key<T> kNone = ((Key<T>)Order<T>::kNegInf << 16) | 0xffffu;

template <class T>
__device__ __forceinline__ int key_expert(Key<T> k) { return 0xffff - (int)(k & 0xffffu); }
template <class T>
__device__ __forceinline__ float key_logit(Key<T> k) {
    const uint32_t o = Order<T>::order(k);
    return Order<T>::value(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// 8 of a lane's logits, kept as stored until they are used.
template <class T>
struct Logits {
    static constexpr int kWords = kPerLane * (int)sizeof(T) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[i]);
        else
            return (float)__builtin_bit_cast(T, (uint16_t)(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu));
    }
};

// Experts [e0, e0 + 8) of a row; -inf past the last one.  EIGHTS: their number
// is a multiple of 8.
template <bool EIGHTS, class T>
__device__ __forceinline__ void load_logits(const T* row, int e0, int experts, Logits<T>* l) {
    constexpr uint32_t ninf = sizeof(T) == 4 ? 0xff800000u : std::is_same_v<T, bf16_t> ? 0xff80ff80u : 0xfc00fc00u;
#pragma unroll
    for (int i = 0; i < Logits<T>::kWords; ++i) l->w[i] = ninf;
    if (e0 + kPerLane <= experts) {
        __builtin_memcpy(l->w, row + e0, sizeof(l->w));
    } else if (!EIGHTS && e0 < experts) {
        for (int i = 0; i < experts - e0; ++i) {
            uint32_t v = 0;
            __builtin_memcpy(&v, row + e0 + i, sizeof(T));
#pragma unroll
            for (int q = 0; q < Logits<T>::kWords; ++q) {   // no indexed registers
                if constexpr (sizeof(T) == 4) {
                    if (q == i) l->w[q] = v;
                } else if (q == i >> 1) {
                    l->w[q] = i & 1 ? (l->w[q] & 0xffffu) | v << 16 : (l->w[q] & 0xffff0000u) | v;
                }
            }
        }
    }
}

template <class T>
__device__ __forceinline__ void make_keys(const float* x, int e0, int experts, Key<T>* key) {
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kPerLane; i += 2) nan |= __builtin_isunordered(x[i], x[i + 1]);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const uint32_t b = Order<T>::high(x[i] + 0.0f);
        key[i] = Order<T>::key(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u), e0 + i);
    }
    if (__any(nan)) {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
            if (x[i] != x[i]) key[i] = Order<T>::key(0xffffffffu, e0 + i);
    }
    if (e0 + kPerLane > experts) {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
            if (e0 + i >= experts) key[i] = 0;
    }
}

// A lane's keys from the largest down (19 exchanges, odd-even merge).
template <class K>
__device__ __forceinline__ void sort_keys(K* k) {
    auto ce = [&](int a, int b) {
        const K hi = max(k[a], k[b]), lo = min(k[a], k[b]);
        k[a] = hi;
        k[b] = lo;
    };
    ce(0, 1); ce(2, 3); ce(4, 5); ce(6, 7);
    ce(0, 2); ce(1, 3); ce(4, 6); ce(5, 7);
    ce(1, 2); ce(5, 6);
    ce(0, 4); ce(1, 5); ce(2, 6); ce(3, 7);
    ce(2, 4); ce(3, 5);
    ce(1, 2); ce(3, 4); ce(5, 6);
}
static_assert(kPerLane == 8, "sort_keys orders 8 keys");

// exp(x - top) is 2^(x log2(e) - c) with c = top log2(e) rounded: what that
// rounding does is common to a token's experts and leaves the quotients, as long
// as it is small beside an exponent's range.  Up to kHuge it is at most 2^-4 (half
// a step of c, which is below 2^21), so that the largest exponential is within 5 %
// of 1.  Past kHuge, where it grows with the logits until every exponential
// overflows or vanishes (from about 2^31 on), the difference is taken first.
constexpr float kHuge = 0x1p20f;
__device__ __forceinline__ float exp_below(float x, float top) {
    const bool huge = fabsf(top) > kHuge;
    return __builtin_amdgcn_exp2f(huge ? (x - top) * kLog2e : fmaf(x, kLog2e, -(top * kLog2e)));
}

// x becomes exp(x - top).  Returns the factor that makes them
// probabilities: 0 for a token that takes no part, NaN where the largest logit
// is not finite.  A token that takes no part counts as one of -inf alone,
// whatever it holds: its exponentials are 0, so that 0 times them is.
template <int LG>
__device__ __forceinline__ float softmax_parts(float* x, float top, bool live) {
    if (!live) top = -INFINITY;
    float c = top * kLog2e;
    if (__any(!(fabsf(top) <= kHuge))) {
        if (!(fabsf(top) < INFINITY)) {
            c = 0.0f;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) x[i] = -INFINITY;
        } else if (fabsf(top) > kHuge) {
            c = 0.0f;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) x[i] -= top;
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], kLog2e, -c));
        s += x[i];
    }
    s = lanes_sum<LG>(s);
    return live ? 1.0f / s + (top - top) : 0.0f;
}

// The tokens of piece p are [tokens p / pieces, tokens (p + 1) / pieces), cut
// into `per` runs of `len` for as many workgroups (the last ones shorter or
// empty), so that no run crosses a piece.
struct Runs {
    int32_t tokens, pieces, per, len;
    __host__ __device__ int32_t piece_begin(int p) const { return (int32_t)((uint32_t)tokens * p / pieces); }
    __host__ __device__ int32_t blocks() const { return pieces * per; }
    __device__ void run(int b, int32_t* t0, int32_t* t1) const {
        const int p = b / per, end = piece_begin(p + 1);
        *t0 = min(piece_begin(p) + (b - p * per) * len, end);
        *t1 = min(*t0 + len, end);
    }
};

// What the router writes, and its workspace.
struct RouterOut {
    int32_t* ids;
    float* gates;
    int32_t* positions;
    int64_t* counts;
    float* prob_sums;
    float* loss;
    int64_t* valid;
    int32_t* hist;      // experts x blocks: a run's choices
    int32_t* base;      // blocks x experts: those of the piece's earlier runs
    float* psum;        // experts x blocks
    int32_t* nvalid;    // blocks
};

// First rows.  Rows are ordered by destination, piece, expert; entry i of that
// order is counts[piece][expert] of slot(i).
__device__ __forceinline__ void slot(int i, int pieces, int local, int* piece, int* expert) {
    const int dest = i / (pieces * local), in = i % (pieces * local);
    *piece = in / local;
    *expert = dest * local + in % local;
}

// The rows before each entry: THREADS threads scan runs of entries; each calls
// put(piece, expert, rows before).  `buf` holds a value per wave.
template <int THREADS, class Get, class Put>
__device__ __forceinline__ void first_rows(int entries, int pieces, int local, int32_t* buf, Get&& get, Put&& put) {
    const int each = (entries + THREADS - 1) / THREADS;
    const int i0 = threadIdx.x * each, lane = threadIdx.x & 63;
    int32_t sum = 0;
    for (int i = i0; i < min(i0 + each, entries); ++i) {
        int p, e;
        slot(i, pieces, local, &p, &e);
        sum += get(p, e);
    }
    int32_t inc = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t up = __shfl_up(inc, d);
        if (lane >= d) inc += up;
    }
    if (lane == 63) buf[threadIdx.x >> 6] = inc;
    __syncthreads();
    int32_t row = inc - sum;
    for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) row += buf[w];
    for (int i = i0; i < min(i0 + each, entries); ++i) {
        int p, e;
        slot(i, pieces, local, &p, &e);
        put(p, e, row);
        row += get(p, e);
    }
}

__device__ __forceinline__ float loss_term(float count, float prob_sum, float n) { return count / n * (prob_sum / n); }

// One token over its LG lanes, lane l holding experts [8 l, 8 l + 8).  The lane
// orders its keys, and each of the topk rounds takes the largest of the lanes'
// first keys and moves the list it came from up by one.  Lane 0 writes the
// chosen keys (0: none), the largest logit and the probabilities' factor; ps
// collects the probabilities.  Returns whether the token takes part.
template <class T, int LG>
__device__ __forceinline__ bool route_token(const Logits<T>& l, bool take, int lane, int experts, int topk, float* ps,
                                            uint64_t* slots, float* topv, float* factor) {
    typedef Key<T> K;
    K key[kPerLane];
    float x[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) x[i] = l.get(i);
    make_keys<T>(x, lane * kPerLane, experts, key);
    sort_keys(key);
    K best = lanes_max<LG>(key[0]);
    const float top = key_logit<T>(best);
    const bool live = take && best > kNone<T>;
    const float inv = softmax_parts<LG>(x, top, live);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) ps[i] = fmaf(x[i], inv, ps[i]);
    for (int j = 0;;) {
        if (lane == 0) slots[j] = live ? best : 0;
        if (++j == topk) break;
        if (key[0] == best) {
#pragma unroll
            for (int i = 0; i + 1 < kPerLane; ++i) key[i] = key[i + 1];
            key[kPerLane - 1] = 0;
        }
        best = lanes_max<LG>(key[0]);
    }
    if (lane == 0) {
        *topv = top;
        *factor = inv;
    }
    return live;
}

// Turns a choice's slot from its key into expert + 1 and exp(logit - top), 0
// for none.  Returns the expert, or -1.
template <class T>
__device__ __forceinline__ int open_slot(uint64_t* slot, float top) {
    const Key<T> k = (Key<T>)*slot;
    if (k <= kNone<T>) {
        *slot = 0;
        return -1;
    }
    const int e = key_expert<T>(k);
    *slot = (uint64_t)(e + 1) << 32 | __float_as_uint(exp_below(key_logit<T>(k), top));
    return e;
}
__device__ __forceinline__ int slot_expert(uint64_t slot) { return (int)(slot >> 32) - 1; }

// The gate of slot j of a token's topk.  Where the largest logit is not finite
// the factor is NaN, and so are the gates.
__device__ __forceinline__ float gate_of(const uint64_t* slots, int j, int topk, float factor, int renormalize) {
    if (slots[j] == 0) return 0.0f;
    const float e = __uint_as_float((uint32_t)slots[j]);
    if (!renormalize) return e * factor;
    float sum = 0.0f;
    for (int i = 0; i < topk; ++i) sum += __uint_as_float((uint32_t)slots[i]);
    return e / sum + (factor - factor);
}

// The number of bits of a row of words in [from, to).
__device__ __forceinline__ int count_bits(const uint32_t* words, int from, int to) {
    int n = 0;
    for (int w = from >> 5; w <= (to - 1) >> 5; ++w) {
        uint32_t v = words[w];
        if (w == from >> 5) v &= ~0u << (from & 31);
        if (w == to >> 5) v &= ~(~0u << (to & 31));
        n += __popc(v);
    }
    return n;
}

// The probability sums of a workgroup: a wave's groups by shuffles, the waves
// in order.  put(expert, sum).
template <int THREADS, int LG, class Put>
__device__ __forceinline__ void sum_probs(float* ps, float* wsum, int experts, Put&& put) {
    const int e0 = threadIdx.x % LG * kPerLane;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
#pragma unroll
        for (int d = LG; d < 64; d <<= 1) ps[i] += __shfl_xor(ps[i], d);
    if ((threadIdx.x & 63) < LG) {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
            if (e0 + i < experts) wsum[(threadIdx.x >> 6) * experts + e0 + i] = ps[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += THREADS) {
        float s = 0.0f;
        for (int w = 0; w < THREADS / 64; ++w) s += wsum[w * experts + e];
        put(e, s);
    }
}

// Workgroup b routes its run.  A chunk's choices go into a bit per (expert,
// token) in LDS, and a choice's rank among its expert's is the number of bits
// before it, whatever order the waves ran in.  Leaves each position's rank
// within the run, the run's counts, probability sums and number of tokens that
// take part.  Bound by its instructions, not by memory: 65536 x 128 top 8 (bf16,
// 16.8 MB of logits) 19.1 us, of which the waves issue vector instructions for
// 10.5 (about 320 for four tokens of 16 lanes: 70 for the keys, 38 for the
// order, 45 for the exponentials, 130 for the rounds).  Sixteen logits a lane
// gained 1 us in bf16 and lost 6 in fp32, 32 a lane ran out of registers.
template <class T, int LG, bool EIGHTS>
__global__ __launch_bounds__(kThreads) void route_runs(const T* logits, int64_t ld, const uint8_t* mask, Runs runs,
                                                       int experts, int topk, int renormalize, RouterOut out) {
    constexpr int GROUPS = kThreads / LG;
    extern __shared__ uint64_t lds[];
    uint64_t* slots = lds;                                   // kChunk x topk: the choices
    uint32_t* bits = (uint32_t*)(slots + kChunk * topk);     // experts x kWords
    int32_t* seen = (int32_t*)(bits + experts * kWords);     // experts: choices of earlier chunks
    float* tops = (float*)(seen + experts);                  // kChunk: a token's largest logit
    float* factors = tops + kChunk;                          // kChunk
    __shared__ int32_t taken;
    const int group = threadIdx.x / LG, lane = threadIdx.x % LG;
    const float per_topk = 1.0f / (float)topk;
    int32_t t0, t1;
    runs.run(blockIdx.x, &t0, &t1);
    for (int e = threadIdx.x; e < experts; e += kThreads) seen[e] = 0;
    if (threadIdx.x == 0) taken = 0;
    float ps[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) ps[i] = 0.0f;
    int mine = 0;
    for (int32_t c0 = t0; c0 < t1; c0 += kChunk) {
        const int len = min(kChunk, t1 - c0);
        for (int i = threadIdx.x; i < experts * kWords; i += kThreads) bits[i] = 0;
        Logits<T> next;
        bool valid = true;
        auto fetch = [&](int tl) {
            load_logits<EIGHTS>(logits + (c0 + tl) * ld, lane * kPerLane, experts, &next);
            valid = !mask || mask[c0 + tl] != 0;
        };
        if (group < len) fetch(group);
        for (int tl = group; tl < len; tl += GROUPS) {
            const Logits<T> l = next;
            const bool take = valid;
            if (tl + GROUPS < len) fetch(tl + GROUPS);   // the next token's logits are on their way meanwhile
            const bool live =
                route_token<T, LG>(l, take, lane, experts, topk, ps, slots + tl * topk, tops + tl, factors + tl);
            if (lane == 0) mine += live;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < len * topk; i += kThreads) {
            const int tl = (int)(((float)i + 0.5f) * per_topk);   // i / topk: i is small
            const int e = open_slot<T>(slots + i, tops[tl]);
            if (e >= 0) atomicOr(&bits[e * kWords + (tl >> 5)], 1u << (tl & 31));
            out.ids[(int64_t)c0 * topk + i] = e;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < len * topk; i += kThreads) {
            const int tl = (int)(((float)i + 0.5f) * per_topk), e = slot_expert(slots[i]);
            out.gates[(int64_t)c0 * topk + i] =
                gate_of(slots + tl * topk, i - tl * topk, topk, factors[tl], renormalize);
            out.positions[(int64_t)c0 * topk + i] = e < 0 ? -1 : seen[e] + count_bits(bits + e * kWords, 0, tl);
        }
        __syncthreads();
        for (int e = threadIdx.x; e < experts; e += kThreads) seen[e] += count_bits(bits + e * kWords, 0, len);
        __syncthreads();
    }
    if (lane == 0 && mine) atomicAdd(&taken, mine);
    const int64_t blocks = runs.blocks();
    // the waves' sums go where the bits were
    sum_probs<kThreads, LG>(ps, (float*)bits, experts, [&](int e, float s) {
        out.psum[e * blocks + blockIdx.x] = s;
        out.hist[e * blocks + blockIdx.x] = seen[e];
    });
    if (threadIdx.x == 0) out.nvalid[blockIdx.x] = taken;
}
static_assert(kMaxExperts <= 512, "place_rows: two experts a thread");
static_assert(kThreads / 64 <= kWords, "the waves' sums fit where the bits were");

// All tokens in one workgroup and one step: LG lanes a token, at most kAlone
// lanes.  The ranks are counted from the token's piece on, so no run ends
// where a piece does.  300 x 16 top 2 in 4 pieces: 8.4 us, five barriers and
// the waits between them; the three launches of the other path took 26.
template <class T, int LG>
__global__ __launch_bounds__(kAlone) void route_alone(const T* logits, int64_t ld, const uint8_t* mask, Runs runs,
                                                      int experts, int world, int topk, int renormalize, float coef,
                                                      RouterOut out) {
    extern __shared__ uint64_t lds[];
    const int tokens = runs.tokens, pieces = runs.pieces;
    const int words = (tokens + 31) >> 5;
    uint64_t* slots = lds;                                          // tokens x topk
    uint32_t* bits = (uint32_t*)(slots + tokens * topk);            // experts x words
    float* tops = (float*)(bits + experts * words);                 // tokens
    float* factors = tops + tokens;                                 // tokens
    int32_t* cnt = (int32_t*)(factors + tokens);                    // pieces x experts
    int32_t* row = cnt + pieces * experts;                          // pieces x experts
    float* wsum = (float*)(row + pieces * experts);                 // kAlone / 64 x experts
    __shared__ int32_t taken;
    __shared__ int32_t scan[kAlone / 64];
    __shared__ float lsum[kAlone / 64];
    const int tl = threadIdx.x / LG, lane = threadIdx.x % LG;
    Logits<T> l;
    bool valid = true;
    if (tl < tokens) {
        load_logits<false>(logits + tl * ld, lane * kPerLane, experts, &l);
        valid = !mask || mask[tl] != 0;
    }
    if (threadIdx.x == 0) taken = 0;
    for (int i = threadIdx.x; i < experts * words; i += kAlone) bits[i] = 0;
    float ps[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) ps[i] = 0.0f;
    bool live = false;
    if (tl < tokens)
        live = route_token<T, LG>(l, valid, lane, experts, topk, ps, slots + tl * topk, tops + tl, factors + tl);
    __syncthreads();
    if (lane == 0 && live) atomicAdd(&taken, 1);
    for (int i = threadIdx.x; i < tokens * topk; i += kAlone) {
        const int t = i / topk, e = open_slot<T>(slots + i, tops[t]);
        if (e >= 0) atomicOr(&bits[e * words + (t >> 5)], 1u << (t & 31));
        out.ids[i] = e;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < pieces * experts; i += kAlone) {
        const int q = i / experts, e = i % experts;
        const int c = count_bits(bits + e * words, runs.piece_begin(q), runs.piece_begin(q + 1));
        cnt[i] = c;
        out.counts[i] = c;
    }
    __syncthreads();
    const float n = (float)max(taken, 1);
    float term = 0.0f;
    sum_probs<kAlone, LG>(ps, wsum, experts, [&](int e, float s) {
        int32_t c = 0;
        for (int q = 0; q < pieces; ++q) c += cnt[q * experts + e];
        out.prob_sums[e] = s;
        term += loss_term((float)c, s, n);
    });
    term = group_sum<kAlone>(term, lsum);
    if (threadIdx.x == 0) {
        *out.valid = taken;
        *out.loss = coef * (float)experts / (float)topk * term;
    }
    first_rows<kAlone>(pieces * experts, pieces, experts / world, scan,
                       [&](int p, int e) { return cnt[p * experts + e]; },
                       [&](int p, int e, int32_t r) { row[p * experts + e] = r; });
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * topk; i += kAlone) {
        const int t = i / topk, e = slot_expert(slots[i]);
        int at = -1;
        if (e >= 0) {
            int q = 0;
            while (t >= runs.piece_begin(q + 1)) ++q;
            at = row[q * experts + e] + count_bits(bits + e * words, runs.piece_begin(q), t);
        }
        out.gates[i] = gate_of(slots + t * topk, i - t * topk, topk, factors[t], renormalize);
        out.positions[i] = at;
    }
}

// One workgroup an expert, four runs a thread: each run's base, the counts and
// the probability sums.  128 experts of 512 runs: 4.2 us, a launch and a wait (a
// workgroup for 16 experts, reading rows instead of columns, 12.6).
__global__ __launch_bounds__(kMostBlocks / 4) void scan_runs(Runs runs, RouterOut out) {
    constexpr int THREADS = kMostBlocks / 4;
    __shared__ int32_t waves[THREADS / 64];
    __shared__ int32_t before[COC_MAX_SPLIT + 1];   // choices before each piece
    __shared__ float lsum[THREADS / 64];
    const int e = blockIdx.x, experts = gridDim.x, lane = threadIdx.x & 63, blocks = runs.blocks();
    const int32_t* hist = out.hist + (int64_t)e * blocks;
    const float* psum = out.psum + (int64_t)e * blocks;
    const int b0 = threadIdx.x * 4;
    int32_t v[4], sum = 0;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool in = b0 + i < blocks;
        v[i] = in ? hist[b0 + i] : 0;
        s += in ? psum[b0 + i] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t h = v[i];
        v[i] = sum;
        sum += h;
    }
    int32_t inc = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t up = __shfl_up(inc, d);
        if (lane >= d) inc += up;
    }
    if (lane == 63) waves[threadIdx.x >> 6] = inc;
    __syncthreads();
    int32_t base = inc - sum;
    for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) base += waves[w];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] += base;
        if (b0 + i < blocks && (b0 + i) % runs.per == 0) before[(b0 + i) / runs.per] = v[i];
    }
    if (threadIdx.x == THREADS - 1) before[runs.pieces] = base + sum;
    s = group_sum<THREADS>(s, lsum);   // its barrier also covers `before`
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (b0 + i < blocks)
            out.base[(int64_t)(b0 + i) * experts + e] = v[i] - before[(b0 + i) / runs.per];
    if (threadIdx.x < (unsigned)runs.pieces)
        out.counts[threadIdx.x * experts + e] = before[threadIdx.x + 1] - before[threadIdx.x];
    if (threadIdx.x == 0) out.prob_sums[e] = s;
}

// Turns a run's ranks into send rows: the rows before its (piece, expert), from
// the counts, and the choices of the piece's earlier runs.  What it reads is
// asked for at once, so that it waits for memory once: 7.0 us for 524288
// choices.  Workgroup 0 also writes the loss and the number of tokens.
__global__ __launch_bounds__(256) void place_rows(Runs runs, int experts, int world, int topk, float coef,
                                                  RouterOut out) {
    constexpr int kAhead = 4;
    extern __shared__ uint64_t lds[];
    int32_t* row = (int32_t*)lds;   // experts: the run's first row of each
    __shared__ int32_t scan[4];
    const int blocks = runs.blocks(), piece = blockIdx.x / runs.per;
    int32_t t0, t1;
    runs.run(blockIdx.x, &t0, &t1);
    const int i0 = t0 * topk + threadIdx.x, i1 = t1 * topk;
    int32_t id[kAhead], at[kAhead], base[2];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
        id[q] = i0 + q * 256 < i1 ? out.ids[i0 + q * 256] : -1;
        at[q] = i0 + q * 256 < i1 ? out.positions[i0 + q * 256] : -1;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int e = threadIdx.x + q * 256;
        base[q] = e < experts ? out.base[(int64_t)blockIdx.x * experts + e] : 0;
    }
    first_rows<256>(runs.pieces * experts, runs.pieces, experts / world, scan,
                    [&](int p, int e) { return (int32_t)out.counts[p * experts + e]; },
                    [&](int p, int e, int32_t r) { if (p == piece) row[e] = r; });
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int e = threadIdx.x + q * 256;
        if (e < experts) row[e] += base[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
        if (id[q] >= 0) out.positions[i0 + q * 256] = at[q] + row[id[q]];
    for (int i = i0 + kAhead * 256; i < i1; i += 256) {
        const int e = out.ids[i];
        if (e >= 0) out.positions[i] += row[e];
    }
    if (blockIdx.x == 0 && threadIdx.x < 64) {
        int32_t taken = 0;
        for (int b = threadIdx.x; b < blocks; b += 64) taken += out.nvalid[b];
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) taken += __shfl_xor(taken, d);
        const float n = (float)max(taken, 1);
        float s = 0.0f;
        for (int e = threadIdx.x; e < experts; e += 64) {
            int64_t c = 0;
            for (int q = 0; q < runs.pieces; ++q) c += out.counts[q * experts + e];
            s += loss_term((float)c, out.prob_sums[e], n);
        }
        s = lanes_sum<64>(s);
        if (threadIdx.x == 0) {
            *out.valid = taken;
            *out.loss = coef * (float)experts / (float)topk * s;
        }
    }
}

// A binary32's bits in unsigned order, every NaN the largest.
__device__ __forceinline__ uint32_t order_bits(float x) {
    const uint32_t b = __float_as_uint(x);
    return x != x ? 0xffffffffu : b & 0x80000000u ? ~b : b | 0x80000000u;
}

// dlogits = p (a - <p, a>) + the gates' term, a_e the loss's derivative by p_e
// with the counts held fixed, for LG lanes a token.  The token's choices are
// shared out over its lanes; what a choice adds goes to the lane that holds its
// expert through LDS, where a token's lanes (one wave) keep 8 LG zeros; an id that
// is no expert's is no choice, and so never a place there.  Bound by
// memory and the waits at its ends: 65536 x 64 top 4 (fp32, 36.8 MB) 9.1 us, 4.0
// TB/s; with every lane reading every choice 18.
//
// A workgroup begins by reading the counts.  256 threads, and 512 where there are
// more counts, for more than 128 experts (8192 x 16 top 2, fp16: 256 threads 3.2
// us, 512 3.5; 65536 x 8 top 2, bf16: 3.6 and 3.9; 20000 x 512 top 8, bf16: 14.2 and
// 13.6).
constexpr int back_threads(int lanes) { return lanes > 16 ? 512 : 256; }
// Its workgroups fill all of the GPU's threads with 16-bit logits and half of them
// with binary32 (twice the bytes a thread has on their way); the tokens past that
// are fetched while others are worked on.  65536 x 64 top 4, fp32: half 9.1 us, all
// 10.5; 65536 x 128 top 8: fp32 17.3 and 20.0, bf16 11.8 and 11.0.
template <class T>
int64_t back_blocks(int64_t tokens, int lanes) {
    const int threads = back_threads(lanes);
    const int64_t most = 256 * 2048 / threads / (sizeof(T) == 4 ? 2 : 1), once = ceil_div(tokens, threads / lanes);
    return once < most ? once : most;
}

template <class T, int LG, bool EIGHTS>
__global__ __launch_bounds__(back_threads(LG)) void route_backward(
    const T* logits, int64_t ld, const uint8_t* mask, const int32_t* ids, const float* gates, const int64_t* counts,
    const int64_t* valid, const float* dgates, const float* dloss, T* dlogits, int64_t ld_out, int tokens, int experts,
    int pieces, int topk, float coef, int renormalize) {
    constexpr int THREADS = back_threads(LG), GROUPS = THREADS / LG;
    __shared__ float extra[GROUPS][LG * kPerLane];
    __shared__ float da[LG * kPerLane];
    const int group = threadIdx.x / LG, lane = threadIdx.x % LG;
    const int e0 = lane * kPerLane;
    const int step = gridDim.x * GROUPS;
    int t = blockIdx.x * GROUPS + group;
    Logits<T> next;
    int id0 = -1;              // the lane's first choice
    float gate0 = 0.0f, dgate0 = 0.0f;
    bool take = false;
    auto chosen = [&](int id) { return (uint32_t)id < (uint32_t)experts; };
    auto fetch = [&](int at) {
        load_logits<EIGHTS>(logits + at * ld, e0, experts, &next);
        take = !mask || mask[at] != 0;
        if (dgates && lane < topk) {
            const int64_t o = (int64_t)at * topk + lane;
            id0 = ids[o];
            gate0 = gates[o];
            dgate0 = dgates[o];
        }
    };
    if (t < tokens) fetch(t);
    const float n = (float)(valid[0] > 0 ? valid[0] : 1);
    const float w = dloss ? dloss[0] * coef * (float)experts / (float)topk / n / n : 0.0f;
    for (int e = threadIdx.x; e < LG * kPerLane; e += THREADS) {
        int64_t c = 0;
        if (e < experts)
            for (int q = 0; q < pieces; ++q) c += counts[(int64_t)q * experts + e];
        da[e] = w * (float)c;
    }
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) extra[group][e0 + i] = 0.0f;
    __syncthreads();
    float a[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) a[i] = da[e0 + i];
    for (; t < tokens; t += step) {
        float x[kPerLane];
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) x[i] = next.get(i);
        const int id = id0;
        const float gate = gate0, dgate = dgate0;
        const bool wanted = take;
        if (t + step < tokens) fetch(t + step);
        uint32_t top_key = 0;   // the largest logit's order, as in make_keys; NaN largest
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) top_key = max(top_key, order_bits(x[i]));
        top_key = lanes_max<LG>(top_key);
        const bool live = wanted && top_key > Order<float>::kNegInf;
        const float top = __uint_as_float(top_key & 0x80000000u ? top_key ^ 0x80000000u : ~top_key);
        const float inv = softmax_parts<LG>(x, top, live);
        float pa = 0.0f;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            x[i] *= inv;
            pa += x[i] * a[i];
        }
        float off = lanes_sum<LG>(pa);
        if (dgates) {
            const int64_t o = (int64_t)t * topk;
            float inner = chosen(id) ? gate * dgate : 0.0f;
            for (int j = lane + LG; j < topk; j += LG)
                if (chosen(ids[o + j])) inner += gates[o + j] * dgates[o + j];
            inner = lanes_sum<LG>(inner);
            const float less = renormalize ? inner : 0.0f;
            if (!renormalize) off += inner;
            if (chosen(id)) extra[group][id] = gate * (dgate - less);
            for (int j = lane + LG; j < topk; j += LG)
                if (chosen(ids[o + j])) extra[group][ids[o + j]] = gates[o + j] * (dgates[o + j] - less);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        T* out = dlogits + t * ld_out;
        float v[kPerLane];
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) v[i] = live ? x[i] * (a[i] - off) + extra[group][e0 + i] : 0.0f;
        if (dgates) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) extra[group][e0 + i] = 0.0f;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
#pragma unroll
        for (int i = 0; i < kPerLane; i += kVec<T>) store_vec(out, e0 + i, experts, &v[i]);
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

// f(lanes of a token, whether the experts are a multiple of 8).
template <int LG = 1, class F>
void by_experts(int32_t experts, F&& f) {
    if (experts <= LG * kPerLane || LG == 64)
        experts % kPerLane == 0 ? f(std::integral_constant<int, LG>(), std::true_type())
                                : f(std::integral_constant<int, LG>(), std::false_type());
    else
        by_experts<LG < 64 ? 2 * LG : 64>(experts, f);
}

Runs make_runs(int64_t tokens, int32_t pieces) {
    const int64_t longest = ceil_div(tokens, pieces);
    int64_t len = ceil_div(longest, kMostBlocks / pieces);
    if (len < kLeastRun) len = kLeastRun;
    const int64_t per = longest > 0 ? ceil_div(longest, len) : 1;
    return {(int32_t)tokens, pieces, (int32_t)per, (int32_t)len};
}

// Lanes for a token's logits.
int lanes_of(int32_t experts) {
    int l = 1;
    while (l * kPerLane < experts) l *= 2;
    return l;
}

// Whether one workgroup routes all tokens, in one launch: a lane for every 8
// logits, and its tables in 64 KiB of LDS (at most 48 KiB of keys).
bool alone(int64_t tokens, int32_t experts, int32_t pieces) {
    return tokens * lanes_of(experts) <= kAlone && tokens * (experts < kMaxTopk ? experts : kMaxTopk) <= 6144 &&
           pieces * experts <= 512;
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
    if (tokens < 0 || experts < 1 || experts > coc::kMaxExperts || pieces < 1 || pieces > COC_MAX_SPLIT) return 0;
    if (coc::alone(tokens, experts, pieces)) return 0;
    return (size_t)coc::make_runs(tokens, pieces).blocks() * (size_t)(experts * 12 + 4);
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
    Runs runs = make_runs(tokens, pieces);
    const int64_t blocks = runs.blocks();
    int32_t* w = (int32_t*)ws;
    RouterOut out{ids, gates, positions, counts, prob_sums, loss, valid, w, w + blocks * experts,
                  (float*)w + 2 * blocks * experts, w + 3 * blocks * experts};
    const bool one = alone(tokens, experts, pieces);   // without tokens too, where there are few experts
    by_type(dt, [&](auto t) {
        using T = decltype(t);
        if (one) {
            const size_t words = (size_t)ceil_div(tokens, 32);
            const size_t lds = (size_t)tokens * topk * 8 + experts * words * 4 + (size_t)tokens * 8 +
                               (size_t)pieces * experts * 8 + kAlone / 64 * (size_t)experts * 4;
            by_experts(experts, [&](auto lg, auto) {
                route_alone<T, decltype(lg)::value><<<dim3(1), dim3(kAlone), lds, stream>>>(
                    (const T*)logits, ld, mask, runs, experts, world, topk, renormalize, coef, out);
            });
            return;
        }
        const size_t lds = kChunk * topk * 8 + (size_t)experts * (kWords + 1) * 4 + kChunk * 8;
        by_experts(experts, [&](auto lg, auto eights) {
            route_runs<T, decltype(lg)::value, decltype(eights)::value>
                <<<dim3((uint32_t)blocks), dim3(kThreads), lds, stream>>>((const T*)logits, ld, mask, runs, experts,
                                                                          topk, renormalize, out);
        });
    });
    st = launched("router");
    if (st != COC_OK || one) return st;
    scan_runs<<<dim3(experts), dim3(kMostBlocks / 4), 0, stream>>>(runs, out);
    st = launched("router");
    if (st != COC_OK) return st;
    place_rows<<<dim3((uint32_t)blocks), dim3(256), (size_t)experts * 4, stream>>>(runs, experts, world, topk, coef,
                                                                                  out);
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
        by_experts(experts, [&](auto lg, auto eights) {
            constexpr int LG = decltype(lg)::value;
            const dim3 grid((uint32_t)back_blocks<T>(tokens, LG)), threads(back_threads(LG));
            route_backward<T, LG, decltype(eights)::value><<<grid, threads, 0, stream>>>(
                (const T*)logits, ld, mask, ids, gates, counts, valid, dgates, dloss, (T*)dlogits, ld_out, (int)tokens,
                experts, pieces, topk, coef, renormalize);
        });
    });
    return launched("router backward");
}

}  // extern "C"
