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

// y[t] = scale table[id - start], or zeros.  tpr threads a token.
template <class T, class I>
__global__ __launch_bounds__(256) void embed_rows(const I* ids, const T* table, T* y, int64_t tokens, int n,
                                                  int64_t start, int64_t vocab, float scale, int tpr) {
    constexpr int VN = kVec<T>;
    const int per = 256 / tpr;
    const int64_t t = (int64_t)blockIdx.x * per + threadIdx.x / tpr;
    if (t >= tokens) return;
    const int64_t r = local_row(ids, t, start, vocab);
    for (int c = (int)(threadIdx.x % tpr) * VN; c < n; c += tpr * VN) {
        float f[VN];
        if (r >= 0) {
            load_vec(table + r * n, c, n, f);
#pragma unroll
            for (int i = 0; i < VN; ++i) f[i] *= scale;
        } else {
#pragma unroll
            for (int i = 0; i < VN; ++i) f[i] = 0.0f;
        }
        store_vec(y + t * n, c, n, f);
    }
}

// ------------------------------------------------------------------ the tokens in order of their rows
// A key is row << 32 | token, so ordering the keys orders the tokens of a row
// by token and no two keys are equal.  Other ranks' tokens get row = vocab and
// come last.
constexpr int kList = 1024;    // keys one workgroup sorts
constexpr int kLists = 32;     // lists one merge pass joins

// Workgroup b sorts tokens [b kList, ...) in LDS (bitonic: its steps do not
// depend on the data).
template <class I>
__global__ __launch_bounds__(kList / 2) void sort_lists(const I* ids, uint64_t* keys, int64_t tokens, int64_t start,
                                                        int64_t vocab) {
    __shared__ uint64_t k[kList];
    const int64_t base = (int64_t)blockIdx.x * kList;
    for (int i = threadIdx.x; i < kList; i += kList / 2) {
        const int64_t t = base + i;
        uint64_t key = ~(uint64_t)0;
        if (t < tokens) {
            const int64_t r = local_row(ids, t, start, vocab);
            key = (uint64_t)(r >= 0 ? r : vocab) << 32 | (uint64_t)t;
        }
        k[i] = key;
    }
    __syncthreads();
    for (int size = 2; size <= kList; size <<= 1)
        for (int half = size >> 1; half > 0; half >>= 1) {
            const int i = threadIdx.x;
            const int lo = 2 * i - (i & (half - 1)), hi = lo + half;
            const bool up = (lo & size) == 0;
            const uint64_t a = k[lo], b = k[hi];
            if ((a > b) == up) {
                k[lo] = b;
                k[hi] = a;
            }
            __syncthreads();
        }
    for (int i = threadIdx.x; i < kList; i += kList / 2)
        if (base + i < tokens) keys[base + i] = k[i];
}

// Keys of list[0, len) below `key`.
__device__ __forceinline__ int64_t below(const uint64_t* list, int64_t len, uint64_t key) {
    int64_t lo = 0;
    while (len > 0) {
        const int64_t h = len >> 1;
        if (list[lo + h] < key) {
            lo += h + 1;
            len -= h + 1;
        } else {
            len = h;
        }
    }
    return lo;
}

// Joins groups of kLists sorted lists of `len` keys: a key's place is the
// number of smaller keys in its group's lists.
__global__ __launch_bounds__(256) void merge_lists(const uint64_t* in, uint64_t* out, int64_t tokens, int64_t len) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= tokens) return;
    const uint64_t key = in[i];
    const int64_t group = i / (len * kLists) * (len * kLists);
    const int64_t own = i / len * len;
    int64_t place = i - own;
    for (int l = 0; l < kLists; ++l) {
        const int64_t b = group + l * len;
        if (b >= tokens) break;
        if (b != own) place += below(in + b, min(len, tokens - b), key);
    }
    out[group + place] = key;
}

// ------------------------------------------------------------------ the sums
// The sorted keys are cut into pieces of kPiece.  A workgroup adds a piece's
// rows of dy over some columns, run by run (a run: the tokens of one table
// row), in order.  A run inside its piece is done and goes out; one that goes
// on past its piece leaves its binary32 sum in `part`: slot 0 of a piece for
// the run it took over from the piece before, slot 1 for one that begins in it.
constexpr int kPiece = 32;

__device__ __forceinline__ uint32_t key_row(uint64_t key) { return (uint32_t)(key >> 32); }

template <class G>
__device__ __forceinline__ void write_grad(G* g, int c, int n, const float* acc, int count, float scale,
                                           bool accumulate) {
    for (int i = 0; i < count; ++i)
        if (c + i < n) g[c + i] = (G)(scale * acc[i] + (accumulate ? (float)g[c + i] : 0.0f));
}

template <class T, class G>
__global__ __launch_bounds__(256) void sum_pieces(const uint64_t* keys, const T* dy, G* grad, float* part,
                                                  int64_t tokens, int n, int64_t vocab, float scale, int accumulate,
                                                  int tpr, int64_t colblocks) {
    constexpr int VN = kVec<T>;
    const int per = 256 / tpr;
    const int64_t piece = blockIdx.x / colblocks * per + threadIdx.x / tpr;
    const int c = (int)((blockIdx.x % colblocks) * tpr + threadIdx.x % tpr) * VN;
    const int64_t k0 = piece * kPiece, k1 = min(k0 + kPiece, tokens);
    if (k0 >= tokens || c >= n) return;
    const uint32_t none = (uint32_t)vocab;
    const uint32_t before = k0 > 0 ? key_row(keys[k0 - 1]) : none;
    const uint32_t after = k1 < tokens ? key_row(keys[k1]) : none;
    uint32_t cur = key_row(keys[k0]);
    bool first = cur == before;
    float acc[VN];
#pragma unroll
    for (int i = 0; i < VN; ++i) acc[i] = 0.0f;
    for (int64_t k = k0; k < k1 && cur != none; ++k) {
        const uint64_t key = keys[k];
        const uint32_t r = key_row(key);
        if (r != cur) {
            if (first)
                for (int i = 0; i < VN; ++i) { if (c + i < n) part[(piece * 2) * n + c + i] = acc[i]; }
            else
                write_grad(grad + (int64_t)cur * n, c, n, acc, VN, scale, accumulate);
            first = false;
            cur = r;
#pragma unroll
            for (int i = 0; i < VN; ++i) acc[i] = 0.0f;
            if (cur == none) break;
        }
        float f[VN];
        load_vec(dy + (int64_t)(uint32_t)key * n, c, n, f);
#pragma unroll
        for (int i = 0; i < VN; ++i) acc[i] += f[i];
    }
    if (cur == none) return;
    if (first || cur == after) {
        float* p = part + (piece * 2 + (first ? 0 : 1)) * n;
        for (int i = 0; i < VN; ++i)
            if (c + i < n) p[c + i] = acc[i];
    } else {
        write_grad(grad + (int64_t)cur * n, c, n, acc, VN, scale, accumulate);
    }
}

// The runs that span pieces: the workgroup of the piece a run begins in adds
// its parts in order, the four waves a quarter of them each.
template <class G>
__global__ __launch_bounds__(256) void sum_parts(const uint64_t* keys, const float* part, G* grad, int64_t tokens,
                                                 int n, int64_t vocab, float scale, int accumulate,
                                                 int64_t colblocks) {
    __shared__ float buf[4][64][4];
    const int64_t piece = blockIdx.x / colblocks;
    const int64_t k0 = piece * kPiece, k1 = k0 + kPiece;
    if (k1 >= tokens) return;
    const uint32_t row = key_row(keys[k1 - 1]);
    if (row == (uint32_t)vocab || key_row(keys[k1]) != row) return;            // no run goes on from here
    if (k0 > 0 && key_row(keys[k0]) == row && key_row(keys[k0 - 1]) == row) return;   // it began before
    const int64_t end = below(keys, tokens, (uint64_t)(row + 1) << 32);
    const int64_t last = (end - 1) / kPiece;
    const int64_t m = last - piece;   // parts of slot 0, after the one of slot 1
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int c = (int)(blockIdx.x % colblocks) * 256 + l * 4;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (w == 0) load_vec(part + (piece * 2 + 1) * n, c, n, s);
    for (int64_t p = m * w / 4; p < m * (w + 1) / 4; ++p) {
        float f[4];
        load_vec(part + (piece + 1 + p) * 2 * n, c, n, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += f[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) buf[w][l][i] = s[i];
    __syncthreads();
    if (w == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = buf[0][l][i] + buf[1][l][i] + buf[2][l][i] + buf[3][l][i];
        write_grad(grad + (int64_t)row * n, c, n, s, 4, scale, accumulate);
    }
}

// Zeros in the rows no token has.  tpr threads a row.
template <class G>
__global__ __launch_bounds__(256) void zero_rows(const uint64_t* keys, G* grad, int64_t tokens, int n, int64_t vocab,
                                                 int tpr) {
    const int64_t r = (int64_t)blockIdx.x * (256 / tpr) + threadIdx.x / tpr;
    if (r >= vocab) return;
    const int64_t at = below(keys, tokens, (uint64_t)r << 32);
    if (at < tokens && key_row(keys[at]) == (uint32_t)r) return;
    const float z[8] = {};
    for (int c = (int)(threadIdx.x % tpr) * kVec<G>; c < n; c += tpr * kVec<G>) store_vec(grad + r * n, c, n, z);
}

// Threads for a row of `vecs` vectors: a power of two, 8 to 256.
int threads_per_row(int64_t vecs) {
    int t = 8;
    while (t < 256 && t < vecs) t *= 2;
    return t;
}

struct GradLayout {
    int64_t keys;    // bytes of one key array (there are two)
    int64_t part;    // bytes of the parts
};

GradLayout grad_layout(int64_t tokens, int64_t n) {
    return {round_up(tokens * 8, 256), ceil_div(tokens, kPiece) * 2 * n * 4};
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
        if (id_type == COC_I32)
            embed_rows<T, int32_t><<<grid, dim3(256), 0, stream>>>((const int32_t*)ids, (const T*)table, (T*)y,
                                                                   tokens, (int)n, start, vocab, scale, tpr);
        else
            embed_rows<T, int64_t><<<grid, dim3(256), 0, stream>>>((const int64_t*)ids, (const T*)table, (T*)y,
                                                                   tokens, (int)n, start, vocab, scale, tpr);
    });
    return launched("embedding");
}

size_t coc_embedding_grad_workspace_bytes(int64_t tokens, int64_t n) {
    if (tokens <= 0 || n <= 0 || coc::check_matrix(tokens, n, "the tokens' matrix") != COC_OK) return 0;
    const coc::GradLayout l = coc::grad_layout(tokens, n);
    return (size_t)(2 * l.keys + l.part);
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
    const size_t need = coc_embedding_grad_workspace_bytes(tokens, n);
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
    const GradLayout lay = grad_layout(tokens, n);
    uint64_t* keys = (uint64_t*)ws;
    uint64_t* other = (uint64_t*)((char*)ws + lay.keys);
    float* part = (float*)((char*)ws + 2 * lay.keys);
    if (tokens > 0) {
        const dim3 grid((uint32_t)ceil_div(tokens, kList));
        if (id_type == COC_I32)
            sort_lists<int32_t><<<grid, dim3(kList / 2), 0, stream>>>((const int32_t*)ids, keys, tokens, start, vocab);
        else
            sort_lists<int64_t><<<grid, dim3(kList / 2), 0, stream>>>((const int64_t*)ids, keys, tokens, start, vocab);
        st = launched("embedding gradient");
        if (st != COC_OK) return st;
        for (int64_t len = kList; len < tokens; len *= kLists) {
            merge_lists<<<dim3((uint32_t)ceil_div(tokens, 256)), dim3(256), 0, stream>>>(keys, other, tokens, len);
            st = launched("embedding gradient");
            if (st != COC_OK) return st;
            uint64_t* k = keys;
            keys = other;
            other = k;
        }
    }
    by_type(grad_dt, [&](auto g) {
        using G = decltype(g);
        if (tokens > 0) {
            by_type(dt, [&](auto t) {
                using T = decltype(t);
                if constexpr (std::is_same_v<G, T> || std::is_same_v<G, float>) {
                    const int tpr = threads_per_row(ceil_div(n, kVec<T>));
                    const int64_t cols = ceil_div(ceil_div(n, kVec<T>), tpr);
                    const int64_t pieces = ceil_div(ceil_div(tokens, kPiece), 256 / tpr);
                    sum_pieces<T, G><<<dim3((uint32_t)(pieces * cols)), dim3(256), 0, stream>>>(
                        keys, (const T*)dy, (G*)grad, part, tokens, (int)n, vocab, scale, accumulate, tpr, cols);
                }
            });
            const int64_t cols = ceil_div(n, 256);
            sum_parts<G><<<dim3((uint32_t)(ceil_div(tokens, kPiece) * cols)), dim3(256), 0, stream>>>(
                keys, part, (G*)grad, tokens, (int)n, vocab, scale, accumulate, cols);
        }
        if (!accumulate) {
            const int tpr = threads_per_row(ceil_div(n, kVec<G>));
            zero_rows<G><<<dim3((uint32_t)ceil_div(vocab, 256 / tpr)), dim3(256), 0, stream>>>(
                keys, (G*)grad, tokens, (int)n, vocab, tpr);
        }
    });
    return launched("embedding gradient");
}

}  // extern "C"
