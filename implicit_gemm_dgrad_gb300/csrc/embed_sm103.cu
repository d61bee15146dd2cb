// Embedding lookup for sm_103a and the gradient of its table: kernels and C
// entry points.
//
// The gradient needs, for every table row, the positions that point to it.
// They are found by a stable radix sort of the token numbers (least
// significant digit first, so equal tokens keep ascending positions): the sums
// then run over contiguous lists in a fixed order, without atomics on values.
#include <algorithm>
#include <climits>
#include <cmath>

#include "token_device.cuh"

namespace cdg {
namespace {

constexpr int kMaxDim = 1 << 24;

// ---------------------------------------------------------------- lookup
struct EmbedArgs {
    const void *table, *tokens;
    void *out;
    long long ld_table, ld_out, count;
    int index_bytes, vocab, n;  // n accesses a row
    float scale;
};

// One access of E elements (16 bytes, one 32-bit word, or one element).
template <typename T, int E>
struct Access;
template <typename T>
struct Access<T, kPerVec<T>> {
    uint4 v;
    __device__ __forceinline__ void load(const T *p) { v = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(float *f) const
    {
        float g[kPerVec<T>];
        widen_vec<T>(v, g);
#pragma unroll
        for (int i = 0; i < kPerVec<T>; ++i) f[i] = g[i];
    }
};
template <typename T>
struct Access<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = __ldg(p); }
    __device__ __forceinline__ void get(float *f) const { f[0] = Elem<T>::get(v); }
};

template <typename T, int E>
__device__ __forceinline__ void store_elems(T *p, const float *f)
{
    if constexpr (E == 1) {
        p[0] = Elem<T>::put(f[0]);
    } else {
        float g[E];
#pragma unroll
        for (int i = 0; i < E; ++i) g[i] = f[i];
        *reinterpret_cast<uint4 *>(p) = narrow_vec<T>(g);
    }
}

// Thread (x, y): row blockIdx.x * blockDim.y + y, accesses x + k * blockDim.x
// of the UNROLL * blockDim.x that blockIdx.y takes.
template <typename T, int E, int UNROLL>
__global__ void __launch_bounds__(256) embed_kernel(const EmbedArgs p)
{
    const long long i = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (i >= p.count) return;
    const int t = token_at(p.tokens, p.index_bytes, i, p.vocab);
    const T *src = static_cast<const T *>(p.table) + static_cast<long long>(max(t, 0)) * p.ld_table;
    T *dst = static_cast<T *>(p.out) + i * p.ld_out;
    const int a0 = blockIdx.y * (blockDim.x * UNROLL) + threadIdx.x;
    Access<T, E> x[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int a = a0 + u * blockDim.x;
        if (a < p.n && t >= 0) x[u].load(src + static_cast<long long>(a) * E);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int a = a0 + u * blockDim.x;
        if (a >= p.n) break;
        float f[E];
        if (t >= 0) {
            x[u].get(f);
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] *= p.scale;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = 0.0f;
        }
        store_elems<T, E>(dst + static_cast<long long>(a) * E, f);
    }
}

template <typename T, int E, int UNROLL>
void launch_embed(const EmbedArgs &a, cudaStream_t s)
{
    int tx = 8;
    while (tx < 256 && tx * UNROLL < a.n) tx *= 2;
    const dim3 block(tx, 256 / tx);
    const dim3 grid(static_cast<unsigned>((a.count + block.y - 1) / block.y), (a.n + tx * UNROLL - 1) / (tx * UNROLL));
    embed_kernel<T, E, UNROLL><<<grid, block, 0, s>>>(a);
}

template <typename T>
void launch_embed(EmbedArgs a, int dim, int sms, cudaStream_t s)
{
    const bool vec = dim % kPerVec<T> == 0 && a.ld_table % kPerVec<T> == 0 && a.ld_out % kPerVec<T> == 0 &&
                     aligned_to(a.table, 16) && aligned_to(a.out, 16);
    a.n = vec ? dim / kPerVec<T> : dim;
    // few accesses: one a thread, spread over the SMs
    const bool few = a.count * a.n < 1024ll * sms;
    if (vec && few) launch_embed<T, kPerVec<T>, 1>(a, s);
    else if (vec) launch_embed<T, kPerVec<T>, 4>(a, s);
    else if (few) launch_embed<T, 1, 1>(a, s);
    else launch_embed<T, 1, 8>(a, s);
}

// ---------------------------------------------------------------- sort
// Up to kRankMax tokens: every token's place is the number of keys before it,
// counted directly (one launch, N^2 comparisons).  Above: a radix sort of
// digits of up to 9 bits, two launches a digit.
constexpr int kRankMax = 8192;
constexpr int kSortThreads = 256, kMaxBins = 512, kWarps = kSortThreads / 32;

struct SortPass {
    const void *tokens;       // first pass: the token list; else NULL
    const int *keys, *order;  // later passes: the previous pass's output
    int *keys_out, *order_out;
    int *hist;                // [tiles][bins]
    int index_bytes, count, vocab, shift, bins, tiles;
};

// Key i: the token number, or vocab (sorted last) where there is no token.
__device__ __forceinline__ int sort_key(const SortPass &p, int i)
{
    if (!p.tokens) return p.keys[i];
    const int t = token_at(p.tokens, p.index_bytes, i, p.vocab);
    return t < 0 ? p.vocab : t;
}

// Eight lanes a token, 32 tokens a CTA; the keys in shared memory.
__global__ void __launch_bounds__(kSortThreads) sort_rank_kernel(const SortPass p)
{
    extern __shared__ int4 keys4[];
    int *keys = reinterpret_cast<int *>(keys4);
    const int n4 = (p.count + 3) / 4;
    for (int i = threadIdx.x; i < 4 * n4; i += kSortThreads) keys[i] = i < p.count ? sort_key(p, i) : INT_MAX;
    __syncthreads();
    const int i = blockIdx.x * 32 + threadIdx.x / 8, sub = threadIdx.x % 8;
    const int key = i < p.count ? keys[i] : 0;
    int before = 0;
    // keys before i count when equal, keys after it do not
#pragma unroll 4
    for (int q = sub; q < n4; q += 8) {
        const int4 k = keys4[q];
        const int d = i - 4 * q;
        before += (k.x < key + (d > 0)) + (k.y < key + (d > 1)) + (k.z < key + (d > 2)) + (k.w < key + (d > 3));
    }
    before += __shfl_xor_sync(0xFFFFFFFFu, before, 1);
    before += __shfl_xor_sync(0xFFFFFFFFu, before, 2);
    before += __shfl_xor_sync(0xFFFFFFFFu, before, 4);
    if (sub == 0 && i < p.count) {
        p.keys_out[before] = key;
        p.order_out[before] = i;
    }
}

// ROUNDS keys a thread: tiles of ROUNDS * kSortThreads keys.
template <int ROUNDS>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortPass p)
{
    __shared__ int h[kMaxBins];
    for (int d = threadIdx.x; d < p.bins; d += kSortThreads) h[d] = 0;
    __syncthreads();
    const int i0 = blockIdx.x * (ROUNDS * kSortThreads) + threadIdx.x;
    int key[ROUNDS];
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) {
        const int i = i0 + k * kSortThreads;
        key[k] = i < p.count ? sort_key(p, i) : -1;
    }
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k)
        if (key[k] >= 0) atomicAdd(&h[(key[k] >> p.shift) & (p.bins - 1)], 1);
    __syncthreads();
    for (int d = threadIdx.x; d < p.bins; d += kSortThreads) p.hist[static_cast<long long>(blockIdx.x) * p.bins + d] = h[d];
}

// Places a tile's keys: digit d of tile t starts after all smaller digits and
// after digit d of the tiles before t.  Warp w takes the tile's w-th run of 32 *
// ROUNDS keys, 32 at a time, in order: the sort is stable.
template <int ROUNDS>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const SortPass p)
{
    __shared__ int start[kMaxBins];
    __shared__ int cnt[kWarps][kMaxBins];
    __shared__ int wsum[kWarps];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int i0 = (blockIdx.x * kWarps + warp) * (32 * ROUNDS);
    int key[ROUNDS], rank[ROUNDS];
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) {
        const int i = i0 + k * 32 + lane;
        key[k] = i < p.count ? sort_key(p, i) : -1;
    }
    // totals and this tile's prefix, two digits a thread
    const int d0 = 2 * tid, d1 = d0 + 1;
    int tot0 = 0, tot1 = 0, before0 = 0, before1 = 0;
    if (d0 < p.bins) {
#pragma unroll 8
        for (int t = 0; t < p.tiles; ++t) {
            const int2 h = __ldg(reinterpret_cast<const int2 *>(p.hist + static_cast<long long>(t) * p.bins + d0));
            const bool prior = t < static_cast<int>(blockIdx.x);
            before0 += prior ? h.x : 0;
            before1 += prior ? h.y : 0;
            tot0 += h.x;
            tot1 += h.y;
        }
    }
    int run = tot0 + tot1;  // inclusive scan over threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, run, o);
        if (lane >= o) run += up;
    }
    if (lane == 31) wsum[warp] = run;
    for (int x = tid; x < kWarps * kMaxBins; x += kSortThreads) (&cnt[0][0])[x] = 0;
    __syncthreads();
    int base = run - tot0 - tot1;
    for (int w = 0; w < warp; ++w) base += wsum[w];
    if (d0 < p.bins) {
        start[d0] = base + before0;
        start[d1] = base + tot0 + before1;
    }
    // rank of each key among its warp's keys of the same digit
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) {
        const int d = key[k] < 0 ? kMaxBins : (key[k] >> p.shift) & (p.bins - 1);
        const unsigned same = __match_any_sync(0xFFFFFFFFu, d);
        const int prior = d < kMaxBins ? cnt[warp][d] : 0;
        rank[k] = prior + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (d < kMaxBins && lane == __ffs(same) - 1) cnt[warp][d] = prior + __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // per digit: the warps' counts become their first positions
    for (int d = tid; d < p.bins; d += kSortThreads) {
        int at = start[d];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int c = cnt[w][d];
            cnt[w][d] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) {
        const int i = i0 + k * 32 + lane;
        if (i >= p.count) break;
        const int at = cnt[warp][(key[k] >> p.shift) & (p.bins - 1)] + rank[k];
        p.keys_out[at] = key[k];
        p.order_out[at] = p.tokens ? i : p.order[i];
    }
}

// ---------------------------------------------------------------- sums
// The sorted positions are cut into chunks of one size.  A chunk's CTA reads
// its rows of dout in order, several at once, and writes a token's sum where
// the token's run lies within the chunk; a run that crosses chunk borders
// leaves partial sums (fp32): the chunk's first run in slot 0 if it began
// earlier, its last run in slot 1 if it began here and goes on.  A second
// launch adds those in chunk order.  So the work is even whatever the tokens'
// frequencies, and the order of additions is fixed.
constexpr int kSumThreads = 128, kMaxChunk = 64, kRowsAtOnce = 8;

struct EmbedGradArgs {
    const void *dout;
    void *dtable;
    long long ld_dout, ld_dtable;
    const int *keys, *order;  // sorted tokens and their positions
    float *partial;           // [chunks][2][dim]
    int count, vocab, dim, accumulate;
    int chunk, chunks;        // positions a chunk, chunks
    int tx, col_tiles;        // threads across a row; column tiles
    unsigned sum_ctas, zero_ctas;
    float scale;
};

template <typename O, int E>
__device__ __forceinline__ void write_sum(const EmbedGradArgs &p, int token, int col, const float (&s)[E])
{
    O *dst = static_cast<O *>(p.dtable) + static_cast<long long>(token) * p.ld_dtable + col;
    constexpr int V = E == 1 ? 1 : kPerVec<O>;
#pragma unroll
    for (int q = 0; q < E; q += V) {
        float f[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            f[e] = s[q + e] * p.scale;
            if (p.accumulate) f[e] += Elem<O>::get(dst[q + e]);
        }
        store_elems<O, V>(dst + q, f);
    }
}

// First position with keys[i] >= v, by a warp: 32 probes a step.
__device__ __forceinline__ int warp_lower_bound(const int *keys, int count, int v, int lane)
{
    int lo = 0, n = count;  // the answer lies in [lo, lo + n]
    while (n > 0) {
        const int step = (n + 31) / 32, at = min(lo + (lane + 1) * step - 1, lo + n - 1);
        const unsigned less = __ballot_sync(0xFFFFFFFFu, __ldg(keys + at) < v);
        const int full = __popc(less);  // probes below v
        const int to = min(full * step, n);
        lo += to;
        n = min(step - 1, n - to);
        if (full == 32) n = 0;
    }
    return lo;
}

// E elements an access (16 bytes of T, or 1), K accesses a thread.
template <typename T, typename O, int E, int K>
__global__ void __launch_bounds__(kSumThreads) embed_grad_kernel(const EmbedGradArgs p)
{
    __shared__ int s_key[kSumThreads / 8][kMaxChunk + 2], s_row[kSumThreads / 8][kMaxChunk];
    // the CTAs that clear rows without a token lie evenly among the others
    const unsigned all = p.sum_ctas + p.zero_ctas;
    const unsigned z0 = static_cast<unsigned>(static_cast<unsigned long long>(blockIdx.x) * p.zero_ctas / all);
    const unsigned z1 = static_cast<unsigned>((blockIdx.x + 1ull) * p.zero_ctas / all);
    if (z1 != z0) {
        const int lane = threadIdx.x % 32, row = static_cast<int>(z0) * (kSumThreads / 32) + threadIdx.x / 32;
        if (row >= p.vocab) return;
        const int at = warp_lower_bound(p.keys, p.count, row, lane);
        if (at < p.count && __ldg(p.keys + at) == row) return;
        O *dst = static_cast<O *>(p.dtable) + static_cast<long long>(row) * p.ld_dtable;
        if constexpr (E > 1) {
            constexpr int V = kPerVec<O>;
            for (int c = lane; c < p.dim / V; c += 32) reinterpret_cast<uint4 *>(dst)[c] = make_uint4(0, 0, 0, 0);
        } else {
            for (int c = lane; c < p.dim; c += 32) dst[c] = Elem<O>::put(0.0f);
        }
        return;
    }
    const unsigned b = blockIdx.x - z0;
    const int ty = kSumThreads / p.tx, x = threadIdx.x % p.tx, y = threadIdx.x / p.tx;
    const int tile = static_cast<int>(b % p.col_tiles);
    const long long c = static_cast<long long>(b / p.col_tiles) * ty + y;
    const bool real = c < p.chunks;
    const int i0 = real ? static_cast<int>(c) * p.chunk : 0, n = real ? min(p.chunk, p.count - i0) : 0;
    // keys with one neighbour on either side (-1 outside the list)
    for (int q = x; q < n + 2; q += p.tx) {
        const int i = i0 + q - 1;
        s_key[y][q] = real && i >= 0 && i < p.count ? __ldg(p.keys + i) : -1;
    }
    for (int q = x; q < n; q += p.tx) s_row[y][q] = __ldg(p.order + i0 + q);
    __syncthreads();
    if (!real) return;
    const int *key = s_key[y] + 1;
    const int col0 = tile * p.tx * E * K + x * E;
    if (col0 >= p.dim) return;
    const T *src = static_cast<const T *>(p.dout) + col0;

    float acc[K][E];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[k][e] = 0.0f;
    bool began = key[-1] == key[0];  // the run began in an earlier chunk
    for (int q0 = 0; q0 < n; q0 += kRowsAtOnce) {
        if (key[q0] == p.vocab) break;  // no tokens from here on
        Access<T, E> v[kRowsAtOnce][K];
#pragma unroll
        for (int r = 0; r < kRowsAtOnce; ++r)
            if (q0 + r < n && key[q0 + r] < p.vocab) {
                const T *row = src + static_cast<long long>(s_row[y][q0 + r]) * p.ld_dout;
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (k == 0 || col0 + k * p.tx * E < p.dim) v[r][k].load(row + k * p.tx * E);
            }
#pragma unroll
        for (int r = 0; r < kRowsAtOnce; ++r) {
            const int q = q0 + r;
            if (q >= n || key[q] == p.vocab) break;
            const bool ends = key[q + 1] != key[q], last = q == n - 1;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float f[E];
                v[r][k].get(f);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[k][e] += f[e];
            }
            if (!ends && !last) continue;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int col = col0 + k * p.tx * E;
                if (k > 0 && col >= p.dim) break;
                if (ends && !began) {
                    write_sum<O, E>(p, key[q], col, acc[k]);
                } else {
                    float *out = p.partial + (2 * c + (began ? 0 : 1)) * p.dim + col;
#pragma unroll
                    for (int e = 0; e < E; ++e) out[e] = acc[k][e];
                }
#pragma unroll
                for (int e = 0; e < E; ++e) acc[k][e] = 0.0f;
            }
            began = false;
        }
    }
}

// Runs that cross chunk borders: the chunk where such a run begins adds its
// slot 1 and the following chunks' slots 0, in order.
template <typename O>
__global__ void __launch_bounds__(kSumThreads) embed_grad_join_kernel(const EmbedGradArgs p)
{
    const int c = blockIdx.x;
    const int end = min((c + 1) * p.chunk, p.count);  // first position after the chunk
    if (end >= p.count) return;
    const int v = __ldg(p.keys + end - 1);
    if (v == p.vocab || __ldg(p.keys + end) != v) return;            // its last run ends here
    const int first = c * p.chunk;
    if (first > 0 && __ldg(p.keys + first - 1) == v) return;         // and it began here
    const int run_end = warp_lower_bound(p.keys, p.count, v + 1, threadIdx.x % 32);
    const int chunks = (run_end - 1) / p.chunk - c;                  // chunks that follow
    for (int col = blockIdx.y * kSumThreads + threadIdx.x; col < p.dim; col += gridDim.y * kSumThreads) {
        const float *part = p.partial + 2ll * c * p.dim + col;
        float s[1] = {part[p.dim]};
#pragma unroll 8
        for (int k = 1; k <= chunks; ++k) s[0] += part[2ll * k * p.dim];
        write_sum<O, 1>(p, v, col, s);
    }
}

// Workspace: keys and order twice (the passes alternate), digit counts,
// partial sums.
struct GradLayout {
    size_t keys[2], order[2], hist, partial, bytes;
    int rounds, tiles, passes, digit, chunk, chunks;
};
GradLayout grad_layout(long long count, int vocab, int dim)
{
    GradLayout l;
    int bits = 1;
    while ((1ll << bits) <= vocab) ++bits;  // keys 0 .. vocab
    l.passes = (bits + 8) / 9;
    l.digit = std::max(1, (bits + l.passes - 1) / l.passes);
    l.rounds = count <= 262144 ? 4 : 16;
    l.tiles = static_cast<int>((count + l.rounds * kSortThreads - 1) / (l.rounds * kSortThreads));
    l.chunk = count * dim < (1ll << 24) ? 16 : kMaxChunk;
    l.chunks = static_cast<int>((count + l.chunk - 1) / l.chunk);
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t was = at;
        at += (n + 255) / 256 * 256;
        return was;
    };
    const bool rank = count <= kRankMax;
    for (int i = 0; i < (rank ? 1 : 2); ++i) {
        l.keys[i] = take(static_cast<size_t>(count) * 4);
        l.order[i] = take(static_cast<size_t>(count) * 4);
    }
    l.hist = take(rank ? 0 : static_cast<size_t>(l.tiles) * (1u << l.digit) * 4);
    l.partial = take(static_cast<size_t>(l.chunks) * 2 * dim * 4);
    l.bytes = at;
    return l;
}

bool grad_sizes_ok(long long count, int vocab, int dim)
{
    return count >= 0 && count < (1ll << 30) && vocab >= 1 && vocab < INT_MAX && dim >= 1 && dim <= kMaxDim;
}

template <int ROUNDS>
void launch_sort_pass(const SortPass &p, cudaStream_t s)
{
    sort_count_kernel<ROUNDS><<<p.tiles, kSortThreads, 0, s>>>(p);
    sort_place_kernel<ROUNDS><<<p.tiles, kSortThreads, 0, s>>>(p);
}

template <typename T, typename O, int E, int K>
cudaError_t launch_sums(EmbedGradArgs a, cudaStream_t s)
{
    a.tx = 8;
    while (a.tx < kSumThreads && a.tx * E * K < a.dim) a.tx *= 2;
    a.col_tiles = (a.dim + a.tx * E * K - 1) / (a.tx * E * K);
    const int ty = kSumThreads / a.tx;
    const long long sum = (a.chunks + ty - 1ll) / ty * a.col_tiles;
    const long long zero = a.accumulate ? 0 : (a.vocab + kSumThreads / 32 - 1ll) / (kSumThreads / 32);
    if (sum + zero >= (1ll << 31)) return cudaErrorInvalidConfiguration;
    a.sum_ctas = static_cast<unsigned>(sum);
    a.zero_ctas = static_cast<unsigned>(zero);
    if (sum + zero > 0) embed_grad_kernel<T, O, E, K><<<a.sum_ctas + a.zero_ctas, kSumThreads, 0, s>>>(a);
    if (a.chunks > 1)
        embed_grad_join_kernel<O><<<dim3(a.chunks, std::min(8, (a.dim + kSumThreads - 1) / kSumThreads)), kSumThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, typename O>
cudaError_t launch_sums(const EmbedGradArgs &a, cudaStream_t s)
{
    // 16-byte accesses where every row of both matrices starts on 16 bytes
    const bool vec = a.dim % kPerVec<T> == 0 && a.ld_dout % kPerVec<T> == 0 && a.ld_dtable % kPerVec<O> == 0 &&
                     aligned_to(a.dout, 16) && aligned_to(a.dtable, 16);
    return vec ? launch_sums<T, O, kPerVec<T>, 1>(a, s) : launch_sums<T, O, 1, 4>(a, s);
}

bool is_dtype(int d) { return d == CDG_F16 || d == CDG_BF16 || d == CDG_F32; }

}  // namespace
}  // namespace cdg

extern "C" {

int cdg_embed(const void *table, long long ld_table, const void *tokens, int index_bytes, long long count, int vocab,
              int dim, int dtype, float scale, void *out, long long ld_out, cdg_stream_t stream)
{
    using namespace cdg;
    if (count < 0 || vocab < 1 || dim < 1 || ld_table < dim || ld_out < dim || !is_dtype(dtype) ||
        (index_bytes != 4 && index_bytes != 8) || !std::isfinite(scale))
        return CDG_ERR_INVALID_ARG;
    if (count == 0) return CDG_OK;
    if (!table || !tokens || !out) return CDG_ERR_INVALID_ARG;
    if (count >= (1ll << 31) || dim > kMaxDim) return CDG_ERR_UNSUPPORTED;
    const int es = dtype_bytes(dtype);
    if (!aligned_to(table, es) || !aligned_to(tokens, index_bytes) || !aligned_to(out, es)) return CDG_ERR_ALIGNMENT;
    const Extent o = extent(out, matrix_bytes(count, dim, ld_out, es));
    if (overlap(o, extent(table, matrix_bytes(vocab, dim, ld_table, es))) ||
        overlap(o, extent(tokens, static_cast<size_t>(count) * index_bytes)))
        return CDG_ERR_ALIAS;
    const int sms = sm_count();
    if (sms < 1) return CDG_ERR_CUDA;
    const EmbedArgs a{table, tokens, out, ld_table, ld_out, count, index_bytes, vocab, 0, scale};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == CDG_F32) launch_embed<float>(a, dim, sms, s);
    else if (dtype == CDG_F16) launch_embed<__half>(a, dim, sms, s);
    else launch_embed<__nv_bfloat16>(a, dim, sms, s);
    return cudaGetLastError() == cudaSuccess ? CDG_OK : CDG_ERR_CUDA;
}

size_t cdg_embed_grad_workspace_bytes(long long count, int vocab, int dim)
{
    return cdg::grad_sizes_ok(count, vocab, dim) ? std::max<size_t>(16, cdg::grad_layout(count, vocab, dim).bytes) : 0;
}

int cdg_embed_grad(const void *dout, long long ld_dout, const void *tokens, int index_bytes, long long count,
                   int vocab, int dim, int dtype, float scale, void *dtable, long long ld_dtable, int out_f32,
                   int accumulate, void *workspace, cdg_stream_t stream)
{
    using namespace cdg;
    if (!grad_sizes_ok(count, vocab, dim) || ld_dout < dim || ld_dtable < dim || !is_dtype(dtype) ||
        (index_bytes != 4 && index_bytes != 8) || !std::isfinite(scale) || (out_f32 != 0 && out_f32 != 1) ||
        (accumulate != 0 && accumulate != 1) || !dtable || !workspace || (count > 0 && (!dout || !tokens)))
        return CDG_ERR_INVALID_ARG;
    const int es = dtype_bytes(dtype), os = out_f32 ? 4 : es;
    if (!aligned_to(workspace, 16) || !aligned_to(dtable, os) || !aligned_to(dout, es) || !aligned_to(tokens, index_bytes))
        return CDG_ERR_ALIGNMENT;
    const GradLayout l = grad_layout(count, vocab, dim);
    const Extent o = extent(dtable, matrix_bytes(vocab, dim, ld_dtable, os)), w = extent(workspace, std::max<size_t>(16, l.bytes));
    const Extent in[2] = {extent(dout, matrix_bytes(count, dim, ld_dout, es)),
                          extent(tokens, static_cast<size_t>(count) * index_bytes)};
    if (overlap(o, w) || overlap(o, in[0]) || overlap(o, in[1]) || overlap(w, in[0]) || overlap(w, in[1]))
        return CDG_ERR_ALIAS;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    const int *keys = reinterpret_cast<int *>(ws + l.keys[0]), *order = reinterpret_cast<int *>(ws + l.order[0]);
    SortPass p{tokens, nullptr, nullptr, reinterpret_cast<int *>(ws + l.keys[0]), reinterpret_cast<int *>(ws + l.order[0]),
               reinterpret_cast<int *>(ws + l.hist), index_bytes, static_cast<int>(count), vocab, 0, 1 << l.digit, l.tiles};
    if (count > 0 && count <= kRankMax) {
        sort_rank_kernel<<<static_cast<unsigned>((count + 31) / 32), kSortThreads, (count + 3) / 4 * 16, s>>>(p);
    } else if (count > 0) {
        for (int q = 0; q < l.passes; ++q) {
            p.tokens = q == 0 ? tokens : nullptr;
            p.keys = keys;
            p.order = order;
            p.keys_out = reinterpret_cast<int *>(ws + l.keys[q & 1]);
            p.order_out = reinterpret_cast<int *>(ws + l.order[q & 1]);
            p.shift = q * l.digit;
            if (l.rounds == 4) launch_sort_pass<4>(p, s);
            else launch_sort_pass<16>(p, s);
            keys = p.keys_out;
            order = p.order_out;
        }
    }
    if (cudaGetLastError() != cudaSuccess) return CDG_ERR_CUDA;
    EmbedGradArgs a{};
    a.dout = dout;
    a.dtable = dtable;
    a.ld_dout = ld_dout;
    a.ld_dtable = ld_dtable;
    a.keys = keys;
    a.order = order;
    a.partial = reinterpret_cast<float *>(ws + l.partial);
    a.count = static_cast<int>(count);
    a.vocab = vocab;
    a.dim = dim;
    a.accumulate = accumulate;
    a.chunk = l.chunk;
    a.chunks = l.chunks;
    a.scale = scale;
    const cudaError_t e = dtype == CDG_F32   ? launch_sums<float, float>(a, s)
                          : dtype == CDG_F16 ? (out_f32 ? launch_sums<__half, float>(a, s) : launch_sums<__half, __half>(a, s))
                          : out_f32          ? launch_sums<__nv_bfloat16, float>(a, s)
                                             : launch_sums<__nv_bfloat16, __nv_bfloat16>(a, s);
    return e == cudaSuccess ? CDG_OK : CDG_ERR_CUDA;
}

}  // extern "C"
