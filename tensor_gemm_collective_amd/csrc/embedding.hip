// Embedding lookup of one vocabulary shard, and its gradient by sorted tokens.
#include "row_ops.h"

namespace coc {
namespace {

// The table row of a token's id, or -1 where the id is another rank's (or none).
template <class I>
__device__ __forceinline__ int64_t local_row(const I* ids, int64_t t, int64_t start, int64_t vocab) {
    const int64_t id = (int64_t)ids[t];
    return id >= start && id - start < vocab ? id - start : -1;   // start >= 0: no overflow
}

// y[t] = scale table[id - start], or zeros.  tpr threads a token.  Bound by
// memory: 4096 tokens of 8192 of one shard in eight (bf16, 75 MB) 12-13 us, 6
// TB/s (repeated ids are read from cache); 32768 x 4096, each id once (537 MB), 93 us,
// 5.8 TB/s.
template <class T, class I, RowKind KIND>
__global__ __launch_bounds__(256) void embed_rows(const I* ids, const T* table, T* y, int64_t tokens, int n,
                                                  int64_t start, int64_t vocab, float scale, int tpr) {
    constexpr int VN = kVec<T>;
    const int per = 256 / tpr;
    const int64_t t = (int64_t)blockIdx.x * per + threadIdx.x / tpr;
    if (t >= tokens) return;
    const int64_t r = local_row(ids, t, start, vocab);
    for (int v = (int)(threadIdx.x % tpr); v * VN < n; v += tpr) {
        const Cols<T, KIND> col(v, n);
        Packed<T> p = {};
        if (r >= 0) {
            col.load(table + r * n, n, &p);
            float f[VN];
#pragma unroll
            for (int i = 0; i < VN; ++i) f[i] = product(p.get(i), scale);
            p.set(f);
        }
        col.store(y + t * n, n, p);
    }
}

// ------------------------------------------------------------------ the tokens in order of their rows
// A key is row << 32 | token.  The tokens are sorted by their rows with a radix
// sort from the rows' lowest digit up, each pass keeping the order of equal
// digits, so the tokens of a row stay in their order.  Other ranks' tokens get
// row = vocab and come last.  A pass over more than one tile of kTile keys
// takes two launches: the tiles' digit counts (count_digits), then every key to
// its place (place_keys); up to one tile is sorted in a single launch (sort_tile).
// The keys are little data, so the launches and the waits in each bound it:
// 32768 tokens in 2 passes 4.8 + 7.4 us each, 1001 tokens 6.1 us.  (Sorted lists
// of 1024 merged by binary search took 69 us for the same 32768.)
constexpr int kTile = 2048;           // keys of a workgroup, two a thread
constexpr int kSort = kTile / 2;      // its threads
constexpr int kWaves = kSort / 64;
constexpr int kDigit = 10;            // the most bits of a digit
constexpr int kBins = 1 << kDigit;
static_assert(kBins == kSort, "a thread a bin");

__device__ __forceinline__ uint32_t key_row(uint64_t key) { return (uint32_t)(key >> 32); }

template <class I>
__device__ __forceinline__ uint64_t token_key(const I* ids, int64_t t, int64_t start, int64_t vocab) {
    const int64_t r = local_row(ids, t, start, vocab);
    return (uint64_t)(r >= 0 ? r : vocab) << 32 | (uint64_t)t;
}

// What a tile's sort keeps in LDS: per wave and bin the wave's keys, then the
// tile's keys of that bin in earlier waves.
struct TileSort {
    uint16_t wave[kWaves][kBins];
    int32_t waves[kWaves];    // of a scan over the bins
};

// Thread i's place r of a tile: wave w holds places [128 w, 128 w + 128).
__device__ __forceinline__ int tile_place(int r) {
    return (int)(threadIdx.x >> 6) * 128 + r * 64 + (int)(threadIdx.x & 63);
}

// For the digits of a thread's two keys (valid or not): their ranks among the
// tile's keys of that digit, in places' order.  `bits` ballots find the lanes
// of a wave that hold the same digit.  Returns the tile's keys of bin
// threadIdx.x.
__device__ __forceinline__ int32_t tile_ranks(TileSort* s, const uint32_t* digit, const bool* valid, int bits,
                                              int32_t* rank) {
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const bool bin = (int)threadIdx.x < 1 << bits;   // this thread's bin is one of the digit's
    if (bin) {
#pragma unroll
        for (int q = 0; q < kWaves; ++q) s->wave[q][threadIdx.x] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        uint64_t same = __ballot(valid[r]);
        for (int b = 0; b < bits; ++b) {
            const bool one = digit[r] >> b & 1;
            const uint64_t m = __ballot(one);
            same &= one ? m : ~m;
        }
        const int before = __popcll(same & ((uint64_t(1) << lane) - 1));
        if (valid[r]) {
            const int base = s->wave[w][digit[r]];
            rank[r] = base + before;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (before == 0) s->wave[w][digit[r]] = (uint16_t)(base + __popcll(same));
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    int32_t run = 0;
    if (bin) {
        int32_t v[kWaves];
#pragma unroll
        for (int q = 0; q < kWaves; ++q) v[q] = s->wave[q][threadIdx.x];
#pragma unroll
        for (int q = 0; q < kWaves; ++q) {
            s->wave[q][threadIdx.x] = (uint16_t)run;
            run += v[q];
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r)
        if (valid[r]) rank[r] += s->wave[w][digit[r]];
    return run;
}

// The sum of v over the threads before this one.
__device__ __forceinline__ int32_t scan_bins(TileSort* s, int32_t v) {
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    int32_t inc = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t up = __shfl_up(inc, d);
        if (lane >= d) inc += up;
    }
    if (lane == 63) s->waves[w] = inc;
    __syncthreads();
    int32_t base = inc - v;
    for (int q = 0; q < w; ++q) base += s->waves[q];
    return base;
}

// flags: a byte a table row, 1 where a token has it.

// At most one tile: all passes in LDS.  The one workgroup also clears the flags: 1000
// tokens take 7.8 us over 32000 rows, 18 over 262144 and 527 over 2^24.
template <class I>
__global__ __launch_bounds__(kSort) void sort_tile(const I* ids, uint64_t* keys, uint8_t* flags, int tokens,
                                                   int64_t start, int64_t vocab, int bits, int passes) {
    __shared__ TileSort s;
    __shared__ uint64_t buf[kTile];
    __shared__ int32_t first[kBins];
    if (flags)
        for (int64_t r = threadIdx.x; r < vocab; r += kSort) flags[r] = 0;
    uint64_t key[2];
    bool valid[2];
    uint32_t digit[2];
    int32_t rank[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int t = tile_place(r);
        valid[r] = t < tokens;
        key[r] = valid[r] ? token_key(ids, t, start, vocab) : 0;
    }
    for (int p = 0; p < passes; ++p) {
#pragma unroll
        for (int r = 0; r < 2; ++r) digit[r] = key_row(key[r]) >> (p * bits) & ((1u << bits) - 1);
        const int32_t count = tile_ranks(&s, digit, valid, bits, rank);
        first[threadIdx.x] = scan_bins(&s, count);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 2; ++r)
            if (valid[r]) buf[first[digit[r]] + rank[r]] = key[r];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 2; ++r)
            if (valid[r]) key[r] = buf[tile_place(r)];
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
        if (valid[r]) {
            keys[tile_place(r)] = key[r];
            if (flags && key_row(key[r]) < vocab) flags[key_row(key[r])] = 1;   // after the barriers above
        }
}

// counts[tile][bin]: the tile's keys of each digit.  keys NULL: the first pass,
// which also clears the flags.
template <class I>
__global__ __launch_bounds__(kSort) void count_digits(const I* ids, const uint64_t* keys, int32_t* counts,
                                                      uint8_t* flags, int64_t tokens, int64_t start, int64_t vocab,
                                                      int shift, int bits) {
    __shared__ int32_t n[kBins];
    n[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int64_t t = (int64_t)blockIdx.x * kTile + r * kSort + threadIdx.x;
        if (t < tokens) {
            const uint64_t key = keys ? keys[t] : token_key(ids, t, start, vocab);
            atomicAdd(&n[key_row(key) >> shift & ((1u << bits) - 1)], 1);
        }
    }
    if (!keys && flags)
        for (int64_t r = (int64_t)blockIdx.x * kSort + threadIdx.x; r < vocab; r += (int64_t)gridDim.x * kSort)
            flags[r] = 0;
    __syncthreads();
    counts[(int64_t)blockIdx.x * kBins + threadIdx.x] = n[threadIdx.x];
}

// Every key of a tile to its place: the keys of smaller digits, those of its
// digit in earlier tiles, and its rank in the tile.  Every tile reads every tile's
// counts, 1 MB in all for 32768 tokens, but 1 GB for 2^20 (65 us a pass) and 17 GB for
// 2^22 (687 us): it is made for the batches of one step, and past a million tokens
// a scan of the counts in a launch of its own would be due.
template <class I>
__global__ __launch_bounds__(kSort) void place_keys(const I* ids, const uint64_t* keys, const int32_t* counts,
                                                    uint64_t* out, uint8_t* flags, int64_t tokens, int64_t start,
                                                    int64_t vocab, int shift, int bits) {
    constexpr int BATCH = 16;
    __shared__ TileSort s;
    __shared__ int32_t first[kBins];
    uint64_t key[2];
    bool valid[2];
    uint32_t digit[2];
    int32_t rank[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int64_t t = (int64_t)blockIdx.x * kTile + tile_place(r);
        valid[r] = t < tokens;
        key[r] = !valid[r] ? 0 : keys ? keys[t] : token_key(ids, t, start, vocab);
        digit[r] = key_row(key[r]) >> shift & ((1u << bits) - 1);
    }
    int32_t all = 0, before = 0;
    const int tiles = gridDim.x, me = blockIdx.x;
    for (int q = 0; q < tiles; q += BATCH) {
        int32_t v[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) v[i] = q + i < tiles ? counts[(int64_t)(q + i) * kBins + threadIdx.x] : 0;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            all += v[i];
            before += q + i < me ? v[i] : 0;
        }
    }
    tile_ranks(&s, digit, valid, bits, rank);
    first[threadIdx.x] = scan_bins(&s, all) + before;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r)
        if (valid[r]) {
            out[first[digit[r]] + rank[r]] = key[r];
            if (!keys && flags && key_row(key[r]) < vocab) flags[key_row(key[r])] = 1;
        }
}

// ------------------------------------------------------------------ the sums
// The sorted keys are cut into pieces of plen.  A workgroup adds a piece's
// rows of dy over some columns, run by run (a run: the tokens of one table
// row), in order.  A run inside its piece is done and goes out; one that goes
// on past its piece leaves its binary32 sum in `part`: slot 0 of a piece for
// the run it took over from the piece before, slot 1 for one that begins in it.
constexpr int kLeastPiece = 8, kMostPiece = 64;
// Table rows a workgroup clears among: 4 of 8192 columns, more of shorter ones
// (32768 x 4096, bf16: 4 rows 171 us, 16 175, 64 188).
int zero_rows(int64_t n) { return n >= 2048 ? 4 : (int)(n <= 8 ? 1024 : 8192 / n); }

// A row's columns [c, c + N), the first `skip` of which another thread writes
// too: adding to what is there is left to that one.
template <int N, class G>
__device__ __forceinline__ void write_grad(G* g, int c, int n, float* acc, float scale, bool accumulate,
                                           int skip = 0) {
    if (accumulate) {
        float old[N];
        load_n<N>(g, c, n, old);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(scale, acc[i], old[i]);
        if (skip > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i >= skip && c + i < n) g[c + i] = (G)acc[i];
            return;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = product(acc[i], scale);
    }
    store_n<N>(g, c, n, acc);
}

// Bound by memory: 32768 x 4096 over 32000 rows (bf16, 531 MB and 17 MB of parts)
// 105 us, 5.2 TB/s.  Eight rows are on their way at a time; the gradient and the
// zeros are streamed past the L2 (175 us for the whole operator with plain
// stores, 152 with streamed ones).  The clearing workgroups come last and fill
// the CUs that the pieces leave.
//
// The first `sums` workgroups take 256 / tpr pieces over tpr vectors of columns
// each; the others clear the rows without tokens among `zrows` each.
template <class T, class G, RowKind KIND>
__global__ __launch_bounds__(256) void sum_pieces(const uint64_t* keys, const uint8_t* flags, const T* dy, G* grad,
                                                  float* part, int plen, int64_t tokens, int n, int64_t vocab, float scale, int accumulate,
                                                  int tpr, int colblocks, int sums, int zrows) {
    constexpr int VN = kVec<T>, BATCH = 8;
    __shared__ uint32_t srow[32 * kMostPiece + 2], stok[32 * kMostPiece + 2];
    if ((int)blockIdx.x >= sums) {
        const int64_t r0 = (int64_t)((int)blockIdx.x - sums) * zrows;
        const int rows = (int)min((int64_t)zrows, vocab - r0), vecs = (n + kVec<G> - 1) / kVec<G>;
        const float z[kVec<G>] = {};
        for (int i = threadIdx.x; i < rows * vecs; i += 256) {
            const int r = i / vecs;
            if (!flags[r0 + r]) store_vec(grad + (r0 + r) * n, (i - r * vecs) * kVec<G>, n, z);
        }
        return;
    }
    const int64_t block = blockIdx.x;
    const int per = 256 / tpr, mine = threadIdx.x / tpr;
    const int64_t first_piece = block / colblocks * per;
    const uint32_t none = (uint32_t)vocab;
    // entry j: key first_piece plen + j - 1
    for (int j = threadIdx.x; j < per * plen + 2; j += 256) {
        const int64_t k = first_piece * plen + j - 1;
        const uint64_t key = k >= 0 && k < tokens ? keys[k] : (uint64_t)none << 32;
        srow[j] = key_row(key);
        stok[j] = (uint32_t)key;
    }
    __syncthreads();
    const int64_t piece = first_piece + mine;
    const int vec = (int)(block % colblocks) * tpr + threadIdx.x % tpr;
    if (vec * VN >= n) return;
    const Cols<T, KIND> col(vec, n);
    const int c = col.c;
    const uint32_t* rows = srow + 1 + mine * plen;
    const uint32_t* toks = stok + 1 + mine * plen;
    uint32_t cur = rows[0];
    if (cur == none) return;
    bool first = cur == rows[-1];   // the run began in the piece before
    float acc[VN];
#pragma unroll
    for (int i = 0; i < VN; ++i) acc[i] = 0.0f;
    float* slots = part + piece * 2 * n;
    for (int k = 0; k < plen && cur != none; k += BATCH) {
        Packed<T> v[BATCH];
#pragma unroll
        for (int q = 0; q < BATCH; ++q)   // past the last of this rank's tokens: any row, unused
            col.load(dy + (int64_t)(rows[k + q] == none ? toks[0] : toks[k + q]) * n, n, &v[q]);
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            const uint32_t r = rows[k + q];
            if (r != cur) {
                if (first)
                    keep_n<VN>(slots, c, n, acc);
                else
                    write_grad<VN>(grad + (int64_t)cur * n, c, n, acc, scale, accumulate, col.skip);
                first = false;
                cur = r;
#pragma unroll
                for (int i = 0; i < VN; ++i) acc[i] = 0.0f;
                if (r == none) break;
            }
#pragma unroll
            for (int i = 0; i < VN; ++i) acc[i] += v[q].get(i);
        }
    }
    if (cur == none) return;
    if (first || cur == rows[plen])
        keep_n<VN>(slots + (first ? 0 : n), c, n, acc);
    else
        write_grad<VN>(grad + (int64_t)cur * n, c, n, acc, scale, accumulate, col.skip);
}

// The runs that span pieces, summed from their parts in order.  A wave looks at
// the run that begins in its piece and adds up to kShort parts by itself; the
// workgroup's longer runs then go one by one to its four waves, a quarter of
// the parts each.  Bound by three waits for memory in a row: 6.9 us of the 32768
// tokens' 137, most of it before the first part arrives.
constexpr int kShort = 16;
template <class G>
__global__ __launch_bounds__(256) void sum_parts(const uint64_t* keys, const float* part, G* grad, int plen, int64_t tokens,
                                                 int n, int64_t vocab, float scale, int accumulate, int64_t pieces,
                                                 int colblocks) {
    constexpr int BATCH = 8;
    __shared__ float buf[4][64][4];
    __shared__ int32_t length[4], run_row[4];   // pieces a wave's long run goes on into, or 0
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int64_t piece0 = (int64_t)(blockIdx.x / colblocks) * 4;
    const int c = (int)(blockIdx.x % colblocks) * 256 + l * 4;
    // s += parts [p0, p1) of slot 0 of the pieces after `piece`
    auto add = [&](float* s, int64_t piece, int64_t p0, int64_t p1) {
        for (int64_t p = p0; p < p1; p += BATCH) {
            float f[BATCH][4];
#pragma unroll
            for (int q = 0; q < BATCH; ++q) load_vec(part + (piece + 1 + min(p + q, p1 - 1)) * 2 * n, c, n, f[q]);
#pragma unroll
            for (int q = 0; q < BATCH; ++q)
                if (p + q < p1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[i] += f[q][i];
                }
        }
    };
    const int64_t piece = piece0 + w;
    int64_t m = 0;
    uint32_t row = 0;
    if (piece < pieces) {   // a piece that another follows
        const int64_t k0 = piece * plen, k1 = k0 + plen;
        row = key_row(keys[k1 - 1]);
        const uint32_t next = key_row(keys[k1]), start = key_row(keys[k0]);
        const uint32_t before = k0 > 0 ? key_row(keys[k0 - 1]) : ~0u;
        // a run that goes on from here and did not begin before
        if (row != (uint32_t)vocab && next == row && !(start == row && before == row))
            for (;;) {
                const int64_t end = (piece + 2 + m + l) * plen;   // the first key after that piece
                const uint64_t over = __ballot(end >= tokens || key_row(keys[end]) != row);
                if (over) {
                    m += __builtin_ctzll(over) + 1;
                    break;
                }
                m += 64;
            }
    }
    if (m > 0 && m <= kShort) {
        float s[4];
        load_vec(part + (piece * 2 + 1) * n, c, n, s);
        add(s, piece, 0, m);
        write_grad<4>(grad + (int64_t)row * n, c, n, s, scale, accumulate);
    }
    if (l == 0) {
        length[w] = m > kShort ? (int32_t)m : 0;
        run_row[w] = (int32_t)row;
    }
    __syncthreads();
    for (int r = 0; r < 4; ++r) {
        const int64_t len = length[r];
        if (len == 0) continue;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (w == 0) load_vec(part + ((piece0 + r) * 2 + 1) * n, c, n, s);
        add(s, piece0 + r, len * w / 4, len * (w + 1) / 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) buf[w][l][i] = s[i];
        __syncthreads();
        if (w == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = buf[0][l][i] + buf[1][l][i] + buf[2][l][i] + buf[3][l][i];
            write_grad<4>(grad + (int64_t)run_row[r] * n, c, n, s, scale, accumulate);
        }
        __syncthreads();
    }
}

// Zeros everywhere, where there are no tokens.
template <class G>
__global__ __launch_bounds__(256) void zero_all(G* grad, int64_t count) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256)
        grad[i] = (G)0.0f;
}

// Threads for a row of `vecs` vectors: a power of two, 8 to 256.
int threads_per_row(int64_t vecs) {
    int t = 8;
    while (t < 256 && t < vecs) t *= 2;
    return t;
}

// A piece's length: enough workgroups to fill the GPU first (1024), then as few
// pieces as that leaves, for the runs they cut (32768 tokens x 4096, bf16: 64
// keys 165 us, 32 175, 16 186; 1001 x 515, fp32: 8 keys against 32 a third of
// the time).
int piece_length(int64_t tokens, int64_t row_vecs) {
    const int64_t want = tokens * ceil_div(row_vecs, 256) / 1024;
    int p = kLeastPiece;
    while (p < kMostPiece && p < want) p *= 2;
    return p;
}

// The workspace: two key arrays, the digit counts, the flags and the parts.
struct GradLayout {
    int64_t keys, counts, flags, part;   // bytes
    int64_t all() const { return 2 * keys + counts + flags + part; }
};

GradLayout grad_layout(int64_t tokens, int64_t vocab, int64_t n) {
    return {round_up(tokens * 8, 256), tokens > kTile ? ceil_div(tokens, kTile) * kBins * 4 : 0, round_up(vocab, 256),
            ceil_div(tokens, piece_length(tokens, ceil_div(n, 8))) * 2 * n * 4};   // 8: the longest vectors, most pieces
}

// f(kind of a row of n).
template <class T, class F>
void by_kind(int64_t n, F&& f) {
    if (n < kVec<T>)
        f(std::integral_constant<RowKind, kTiny>());
    else
        f(std::integral_constant<RowKind, kRagged>());
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

coc_status check_embedding(int64_t tokens, int64_t vocab, int64_t n, coc_dtype dt, coc_index it, int64_t start) {
    if (!dtype_valid(dt)) return fail(COC_ERR_DTYPE, "unknown dtype %d", (int)dt);
    if (it != COC_I32 && it != COC_I64) return fail(COC_ERR_DTYPE, "ids are int32 or int64");
    if (start < 0) return fail(COC_ERR_SHAPE, "the shard's first id is negative");
    if (n < 1) return fail(COC_ERR_SHAPE, "a row has at least one element (n=%lld)", (long long)n);
    coc_status s = check_matrix(vocab, n, "the table");
    if (s != COC_OK) return s;
    return check_matrix(tokens, n, "the tokens' matrix");
}

}  // namespace
}  // namespace coc

extern "C" {

coc_status coc_embedding(const void* ids, coc_index id_type, const void* table, void* y, int64_t tokens,
                         int64_t vocab, int64_t n, int64_t start, float scale, coc_dtype dt, hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_embedding(tokens, vocab, n, dt, id_type, start);
    if (st != COC_OK) return st;
    const int32_t es = (int32_t)elem_size(dt), is = id_type == COC_I32 ? 4 : 8;
    const Arg args[] = {
        {ids, tokens * is, is, false, "ids"},
        {table, tokens > 0 ? vocab * n * es : 0, es, false, "table"},
        {y, tokens * n * es, es, true, "y"},
    };
    st = check_args(args, 3);
    if (st != COC_OK) return st;
    if (tokens == 0) return COC_OK;
    by_type(dt, [&](auto t) {
        using T = decltype(t);
        const int tpr = threads_per_row(ceil_div(n, kVec<T>));
        const dim3 grid((uint32_t)ceil_div(tokens, 256 / tpr));
        by_kind<T>(n, [&](auto kind) {
            constexpr RowKind K = decltype(kind)::value;
            if (id_type == COC_I32)
                embed_rows<T, int32_t, K><<<grid, dim3(256), 0, stream>>>((const int32_t*)ids, (const T*)table, (T*)y,
                                                                          tokens, (int)n, start, vocab, scale, tpr);
            else
                embed_rows<T, int64_t, K><<<grid, dim3(256), 0, stream>>>((const int64_t*)ids, (const T*)table, (T*)y,
                                                                          tokens, (int)n, start, vocab, scale, tpr);
        });
    });
    return launched("embedding");
}

size_t coc_embedding_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t n) {
    using namespace coc;
    if (tokens <= 0 || vocab <= 0 || n <= 0 || check_matrix(tokens, n, "the tokens' matrix") != COC_OK ||
        check_matrix(vocab, n, "the table") != COC_OK)
        return 0;
    return (size_t)grad_layout(tokens, vocab, n).all();
}

coc_status coc_embedding_grad(const void* ids, coc_index id_type, const void* dy, void* grad, int64_t tokens,
                              int64_t vocab, int64_t n, int64_t start, float scale, int32_t accumulate, coc_dtype dt,
                              coc_dtype grad_dt, void* ws, size_t ws_bytes, hipStream_t stream) {
    using namespace coc;
    clear_error();
    coc_status st = check_embedding(tokens, vocab, n, dt, id_type, start);
    if (st != COC_OK) return st;
    if (grad_dt != dt && grad_dt != COC_F32)
        return fail(COC_ERR_DTYPE, "the gradient has dy's dtype or fp32");
    const size_t need = coc_embedding_grad_workspace_bytes(tokens, vocab, n);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(COC_ERR_WORKSPACE, "embedding gradient needs %zu workspace bytes (got %zu)", need,
                    ws ? ws_bytes : (size_t)0);
    const int32_t es = (int32_t)elem_size(dt), gs = (int32_t)elem_size(grad_dt), is = id_type == COC_I32 ? 4 : 8;
    const Arg args[] = {
        {ids, tokens * is, is, false, "ids"},
        {dy, tokens * n * es, es, false, "dy"},
        {grad, vocab * n * gs, gs, true, "grad"},
        {ws, (int64_t)need, 8, true, "ws"},
    };
    st = check_args(args, 4);
    if (st != COC_OK) return st;
    if (vocab == 0 || (tokens == 0 && accumulate)) return COC_OK;
    const GradLayout lay = grad_layout(tokens, vocab, n);
    uint64_t* keys = (uint64_t*)ws;
    uint64_t* other = (uint64_t*)((char*)ws + lay.keys);
    int32_t* counts = (int32_t*)((char*)ws + 2 * lay.keys);
    uint8_t* flags = accumulate ? nullptr : (uint8_t*)counts + lay.counts;
    float* part = (float*)((char*)counts + lay.counts + lay.flags);
    const int plen = piece_length(tokens, ceil_div(n, 16 / es));
    if (tokens > 0) {
        int width = 1;   // bits of the rows, vocab itself among them
        while (vocab >> width) ++width;
        const int passes = (width + kDigit - 1) / kDigit, bits = (width + passes - 1) / passes;
        const dim3 tiles((uint32_t)ceil_div(tokens, kTile));
        auto sort = [&](auto id) {
            using I = decltype(id);
            const I* in = (const I*)ids;
            if (tokens <= kTile) {
                sort_tile<I><<<dim3(1), dim3(kSort), 0, stream>>>(in, keys, flags, (int)tokens, start, vocab, bits,
                                                                  passes);
                return launched("embedding gradient");
            }
            for (int p = 0; p < passes; ++p) {
                const uint64_t* from = p ? keys : nullptr;
                count_digits<I><<<tiles, dim3(kSort), 0, stream>>>(in, from, counts, flags, tokens, start, vocab,
                                                                   p * bits, bits);
                const coc_status s = launched("embedding gradient");
                if (s != COC_OK) return s;
                place_keys<I><<<tiles, dim3(kSort), 0, stream>>>(in, from, counts, other, flags, tokens, start, vocab,
                                                                 p * bits, bits);
                uint64_t* k = keys;
                keys = other;
                other = k;
            }
            return launched("embedding gradient");
        };
        st = id_type == COC_I32 ? sort(int32_t()) : sort(int64_t());
        if (st != COC_OK) return st;
    }
    by_type(grad_dt, [&](auto g) {
        using G = decltype(g);
        if (tokens == 0) {
            zero_all<G><<<dim3(2048), dim3(256), 0, stream>>>((G*)grad, vocab * n);
            return;
        }
        by_type(dt, [&](auto t) {
            using T = decltype(t);
            if constexpr (std::is_same_v<G, T> || std::is_same_v<G, float>) {
                const int tpr = threads_per_row(ceil_div(n, kVec<T>));
                const int64_t cols = ceil_div(ceil_div(n, kVec<T>), tpr);
                const int64_t pieces = ceil_div(ceil_div(tokens, plen), 256 / tpr);
                const int64_t zeros = accumulate ? 0 : ceil_div(vocab, zero_rows(n));
                by_kind<T>(n, [&](auto kind) {
                    sum_pieces<T, G, decltype(kind)::value><<<dim3((uint32_t)(pieces * cols + zeros)), dim3(256), 0,
                                                              stream>>>(
                        keys, flags, (const T*)dy, (G*)grad, part, plen, tokens, (int)n, vocab, scale, accumulate,
                        tpr, (int)cols, (int)(pieces * cols), zero_rows(n));
                });
            }
        });
        const int64_t cols = ceil_div(n, 256), followed = (tokens - 1) / plen;
        if (followed > 0)   // pieces that another follows
            sum_parts<G><<<dim3((uint32_t)(ceil_div(followed, 4) * cols)), dim3(256), 0, stream>>>(
                keys, part, (G*)grad, plen, tokens, (int)n, vocab, scale, accumulate, followed, (int)cols);
    });
    return launched("embedding gradient");
}

}  // extern "C"
