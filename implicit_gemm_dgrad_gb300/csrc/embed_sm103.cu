// Embedding lookup for sm_103a and the gradient of its table: kernels and C
// entry points.
//
// The lookup reads and writes every element once: DRAM-bound, less what
// repeated tokens find in L2 (32768 x 4096 fp16, text-like tokens: 61 us, 8.8
// TB/s of reads and writes; 30000 x 777 bf16, rows at every alignment: 16 us).
//
// The gradient needs, for every table row, the positions that point to it.
// They are found by a stable sort of the token numbers, so that the sums run
// over contiguous lists in a fixed order, without atomics on values.  Its cost
// beside the data: 65536 tokens x 4096 bf16 into 32768 rows read 537 MB and
// write 268 MB, 119 us at the copy rate; the call takes 170 us, of which the
// sort's four launches and the join of long runs are about 40 (the sort has 64
// tiles for 152 SMs, and each of them adds up all tiles' digit counts).
// Accumulating, it reads and writes the rows that tokens point to, here 13.6
// thousand: 190 us (floor 112).  2048 x 1000 into 10007 fp32 rows: 25 us, and 21
// accumulating.
//
// The adding up grows with the square of the tiles: 2^18 tokens x 64 take 134 us,
// 2^20 0.40 ms, 2^22 0.87, 2^24 4.4 (of which the data is 0.3).
#include <algorithm>
#include <climits>
#include <cmath>

#include "ptx.cuh"
#include "token_device.cuh"

namespace cdg {
namespace {

constexpr int kMaxDim = 1 << 24;

// Where a matrix's rows lie in 16-byte vectors: row v's first element is
// element `phase(v)` of its first vector.
struct Phase {
    uint32_t base, ld;  // elements, modulo the vector's
    template <typename T>
    static Phase of(const void *p, long long ld)
    {
        return Phase{static_cast<uint32_t>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T)),
                     static_cast<uint32_t>(ld % kPerVec<T>)};
    }
    template <typename T>
    __device__ __forceinline__ int at(uint32_t v) const { return static_cast<int>((base + v * ld) & (kPerVec<T> - 1)); }
};

// Elements [col, col + E) of a row of `cols`, of which those that exist: whole
// aligned vectors, or single elements at the row's ends.
template <typename O, int E>
__device__ __forceinline__ void store_columns(O *row, int col, int cols, const float (&f)[E])
{
    if (col >= 0 && col + E <= cols) {
        constexpr int V = kPerVec<O>;
#pragma unroll
        for (int q = 0; q < E; q += V) {
            float g[V];
#pragma unroll
            for (int e = 0; e < V; ++e) g[e] = f[q + e];
            *reinterpret_cast<uint4 *>(row + col + q) = narrow_vec<O>(g);
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (col + e >= 0 && col + e < cols) row[col + e] = Elem<O>::put(f[e]);
    }
}

// ---------------------------------------------------------------- lookup
struct EmbedArgs {
    const void *table, *tokens;
    void *out;
    long long ld_table, ld_out, count;
    int index_bytes, vocab, dim;
    Phase phase;             // of out
    const char *lo, *hi;     // the table
    float scale;
};

// Thread (x, y): row blockIdx.x * blockDim.y + y, vectors x + k * blockDim.x of
// the UNROLL * blockDim.x that blockIdx.y takes.  Vectors are aligned in out;
// ALIGNED: and in the table, else they are read from two blocks each.
template <typename T, bool ALIGNED, int UNROLL>
__global__ void __launch_bounds__(256) embed_kernel(const EmbedArgs p)
{
    constexpr int E = kPerVec<T>;
    const long long i = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (i >= p.count) return;
    const int t = token_at(p.tokens, p.index_bytes, i, p.vocab);
    const T *src = static_cast<const T *>(p.table) + static_cast<long long>(max(t, 0)) * p.ld_table;
    T *dst = static_cast<T *>(p.out) + i * p.ld_out;
    const int col0 = static_cast<int>(blockIdx.y * (blockDim.x * UNROLL) + threadIdx.x) * E -
                     (ALIGNED ? 0 : p.phase.at<T>(static_cast<uint32_t>(i)));
    Shifted<T> x[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int col = col0 + static_cast<int>(u * blockDim.x) * E;
        if (col < p.dim && t >= 0) {
            if (ALIGNED) x[u].a = __ldg(reinterpret_cast<const uint4 *>(src + col));
            else x[u].load(src + col, p.lo, p.hi, col, p.dim);
        }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int col = col0 + static_cast<int>(u * blockDim.x) * E;
        if (col >= p.dim) break;
        float f[E];
        if (t >= 0) {
            widen_vec<T>(ALIGNED ? x[u].a : x[u].get(), f);
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] *= p.scale;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = 0.0f;
        }
        store_columns<T, E>(dst, col, p.dim, f);
    }
}

template <typename T, bool ALIGNED, int UNROLL>
void launch_embed(const EmbedArgs &a, cudaStream_t s)
{
    const int n = (a.dim + kPerVec<T> - 1) / kPerVec<T> + (ALIGNED ? 0 : 1);  // vectors a row, at most
    int tx = 8;
    while (tx < 256 && tx * UNROLL < n) tx *= 2;
    const dim3 block(tx, 256 / tx);
    const dim3 grid(static_cast<unsigned>((a.count + block.y - 1) / block.y), (n + tx * UNROLL - 1) / (tx * UNROLL));
    embed_kernel<T, ALIGNED, UNROLL><<<grid, block, 0, s>>>(a);
}

template <typename T>
void launch_embed(EmbedArgs a, int sms, cudaStream_t s)
{
    const int E = kPerVec<T>;
    const bool aligned = a.dim % E == 0 && a.ld_table % E == 0 && a.ld_out % E == 0 && aligned_to(a.table, 16) &&
                         aligned_to(a.out, 16);
    a.phase = Phase::of<T>(a.out, a.ld_out);
    a.lo = static_cast<const char *>(a.table);
    a.hi = a.lo + matrix_bytes(a.vocab, a.dim, a.ld_table, sizeof(T));
    // few vectors: one a thread, spread over the SMs
    const bool few = a.count * (a.dim / E + 1) < 1024ll * sms;
    if (aligned && few) launch_embed<T, true, 1>(a, s);
    else if (aligned) launch_embed<T, true, 4>(a, s);
    else if (few) launch_embed<T, false, 1>(a, s);
    else launch_embed<T, false, 4>(a, s);
}

// ---------------------------------------------------------------- sort
// The first launch of a call begins when all work before it is done; the others
// may begin while the one before them ends, and wait.  What the call's own
// launches write (the workspace) is therefore read past L1 (__ldcg), never as
// read-only data.
//
// Up to kRankMax tokens: every token's place is the number of keys before it,
// counted directly (one launch, N^2 comparisons; 8192 tokens take 17 us longer
// that way than by the radix sort).  Above: a radix sort of
// digits of up to 9 bits, two launches a digit.
constexpr int kRankMax = 4096;
constexpr int kSortThreads = 256, kMaxBins = 512, kWarps = kSortThreads / 32;

struct SortPass {
    const void *tokens;       // first pass: the token list; else NULL
    const int *keys, *order;  // later passes: the previous pass's output
    int *keys_out, *order_out;
    int *hist;                // [tiles][bins]
    int *runs;                // the count of long runs, set to 0
    int index_bytes, count, vocab, shift, bins, tiles;
};

// Key i: the token number, or vocab (sorted last) where there is no token.
__device__ __forceinline__ int sort_key(const SortPass &p, int i)
{
    if (!p.tokens) return __ldcg(p.keys + i);
    const int t = token_at(p.tokens, p.index_bytes, i, p.vocab);
    return t < 0 ? p.vocab : t;
}

// LANES lanes a token; the keys in shared memory.
template <int LANES>
__global__ void __launch_bounds__(kSortThreads) sort_rank_kernel(const SortPass p)
{
    extern __shared__ int4 keys4[];
    int *keys = reinterpret_cast<int *>(keys4);
    const int n4 = (p.count + 3) / 4;
    grid_dep_launch_dependents();
    grid_dep_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.runs = 0;
#pragma unroll 8
    for (int i = threadIdx.x; i < 4 * n4; i += kSortThreads) keys[i] = i < p.count ? sort_key(p, i) : INT_MAX;
    __syncthreads();
    const int i = blockIdx.x * (kSortThreads / LANES) + threadIdx.x / LANES, sub = threadIdx.x % LANES;
    const int key = i < p.count ? keys[i] : 0;
    int before = 0;
    // keys before i count when equal, keys after it do not
#pragma unroll 4
    for (int q = sub; q < n4; q += LANES) {
        const int4 k = keys4[q];
        const int d = i - 4 * q;
        before += (k.x < key + (d > 0)) + (k.y < key + (d > 1)) + (k.z < key + (d > 2)) + (k.w < key + (d > 3));
    }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
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
    grid_dep_launch_dependents();
    grid_dep_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.runs = 0;
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
    grid_dep_launch_dependents();
    grid_dep_wait();
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
#pragma unroll 16
        for (int t = 0; t < p.tiles; ++t) {
            const int2 h = __ldcg(reinterpret_cast<const int2 *>(p.hist + static_cast<long long>(t) * p.bins + d0));
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
        if (static_cast<unsigned>(at) >= static_cast<unsigned>(p.count)) continue;  // tokens changed since they were counted
        p.keys_out[at] = key[k];
        p.order_out[at] = p.tokens ? i : __ldcg(p.order + i);
    }
}

// ---------------------------------------------------------------- sums
// The sorted positions are cut into chunks of one size, a team of threads
// each.  A token's run of up to a chunk's length belongs to the chunk it begins
// in, wherever it ends.  A longer run is cut at the chunk borders: each chunk
// leaves its part's sum (fp32), in slot 0 if the run began earlier, in slot 1 if
// it begins there, and a second launch adds the parts in a fixed order.  So the
// work is even whatever the tokens' frequencies, and sums do not depend on
// scheduling.
//
// A thread holds one 16-byte vector of columns (of dout's type), placed so that
// it is aligned in the row it writes; rows of dout at other alignments are read
// from two blocks.
//
// Whatever the sorted lists hold, nothing outside the tensors is touched: keys
// and positions are checked as they are read.  (A caller that changes the tokens
// while the call runs leaves lists that no sort made.)
constexpr int kSumThreads = 128, kMaxChunk = 64, kZeroRows = 4;

// A key of the list; one that is none counts as "no token".
__device__ __forceinline__ int checked_key(const int *keys, int i, int vocab)
{
    return static_cast<int>(min(static_cast<unsigned>(__ldcg(keys + i)), static_cast<unsigned>(vocab)));
}

struct EmbedGradArgs {
    const void *dout;
    void *dtable;
    long long ld_dout, ld_dtable;
    const int *keys, *order;  // sorted tokens and their positions
    float *partial;           // [chunks][2][pitch]
    int *runs;                // long runs: how many, then the chunk each begins in (in any order)
    const char *lo, *hi;      // dout
    Phase phase;              // of dtable
    int count, vocab, dim, accumulate;
    int chunk, chunks;        // positions a chunk, chunks
    int pitch;                // of partial rows: dim and a vector more
    int tx, col_tiles;        // threads across a row; column tiles
    unsigned sum_ctas, zero_ctas;
    float scale;
};

// First position with keys[i] >= v, by a warp: 32 probes a step.
__device__ __forceinline__ int warp_lower_bound(const int *keys, int count, int v, int lane)
{
    int lo = 0, n = count;  // the answer lies in [lo, lo + n]
    while (n > 0) {
        const int step = (n + 31) / 32, at = min(lo + (lane + 1) * step - 1, lo + n - 1);
        const unsigned less = __ballot_sync(0xFFFFFFFFu, __ldcg(keys + at) < v);
        const int full = __popc(less);  // probes below v
        const int to = min(full * step, n);
        lo += to;
        n = min(step - 1, n - to);
        if (full == 32) n = 0;
    }
    return lo;
}
// How many of key[a .. a + n) are v, by a warp (n <= 64).
__device__ __forceinline__ int warp_count(const int *key, int a, int n, int v, int lane)
{
    return __popc(__ballot_sync(0xFFFFFFFFu, lane < n && key[a + lane] == v)) +
           __popc(__ballot_sync(0xFFFFFFFFu, lane + 32 < n && key[a + min(lane + 32, n - 1)] == v));
}

template <typename T, typename O, bool ALIGNED, bool ACCUMULATE>
__global__ void __launch_bounds__(kSumThreads, ALIGNED && !ACCUMULATE ? 7 : 1) embed_grad_kernel(const EmbedGradArgs p)
{
    constexpr int E = kPerVec<T>, V = kPerVec<O>, ROWS = ACCUMULATE ? 4 : 8;  // rows read at once
    __shared__ int s_key[kSumThreads / 32][3 * kMaxChunk + 1], s_row[kSumThreads / 32][2 * kMaxChunk];
    grid_dep_launch_dependents();
    grid_dep_wait();
    // the CTAs that clear rows without a token lie evenly among the others
    const unsigned all = p.sum_ctas + p.zero_ctas;
    const unsigned z0 = static_cast<unsigned>(static_cast<unsigned long long>(blockIdx.x) * p.zero_ctas / all);
    const unsigned z1 = static_cast<unsigned>((blockIdx.x + 1ull) * p.zero_ctas / all);
    if (z1 != z0) {
        // a few rows a warp: the next key of the list is looked for again only after a row that has one
        const int lane = threadIdx.x % 32;
        const long long row0 = (static_cast<long long>(z0) * (kSumThreads / 32) + threadIdx.x / 32) * kZeroRows;
        int next = -1;  // the first key from the last row on
        for (int r = 0; r < kZeroRows && row0 + r < p.vocab; ++r) {
            const int row = static_cast<int>(row0) + r;
            if (next < row) {
                const int at = warp_lower_bound(p.keys, p.count, row, lane);
                next = at < p.count ? __ldcg(p.keys + at) : INT_MAX;
            }
            if (next == row) continue;
            O *dst = static_cast<O *>(p.dtable) + static_cast<long long>(row) * p.ld_dtable;
            const float zero[V] = {};
            for (int c = lane * V - p.phase.at<O>(row); c < p.dim; c += 32 * V) store_columns<O, V>(dst, c, p.dim, zero);
        }
        return;
    }
    const unsigned b = blockIdx.x - z0;
    const int ty = kSumThreads / p.tx, x = threadIdx.x % p.tx, y = threadIdx.x / p.tx;
    const int tile = static_cast<int>(b % p.col_tiles);
    const long long c = static_cast<long long>(b / p.col_tiles) * ty + y;
    const bool real = c < p.chunks;
    const int chunk = p.chunk, i0 = real ? static_cast<int>(c) * chunk : 0, n = real ? min(chunk, p.count - i0) : 0;
    // the keys from one chunk before to one after (-1 before the list, INT_MAX after it)
    for (int q = x; q < 3 * chunk + 1; q += p.tx) {
        const int i = i0 + q - chunk;
        s_key[y][q] = i < 0 ? -1 : i < p.count ? checked_key(p.keys, i, p.vocab) : INT_MAX;
    }
    for (int q = x; q < 2 * chunk; q += p.tx)
        if (i0 + q < p.count) {
            const int row = __ldcg(p.order + i0 + q);
            s_row[y][q] = static_cast<unsigned>(row) < static_cast<unsigned>(p.count) ? row : 0;
        }
    __syncthreads();
    if (!real) return;
    const int *key = s_key[y] + chunk;  // key[r]: of position i0 + r

    // ---- which positions [p0, p1) are this chunk's
    const int lane = threadIdx.x % 32, head = key[0], tail = key[n - 1];
    int p0 = 0, p1 = n;
    bool began = key[-1] == head;  // a long run's part that began in an earlier chunk
    if (began) {
        const int before = warp_count(key, -chunk, chunk, head, lane), here = warp_count(key, 0, chunk, head, lane);
        if (before + here <= chunk && key[here] != head) {  // a short run of an earlier chunk
            p0 = here;
            began = false;
        }
    }
    if (p0 < n && tail < p.vocab && key[n] == tail && !(began && tail == head)) {
        const int here = warp_count(key, 0, n, tail, lane), after = warp_count(key, n, chunk, tail, lane);
        if (here + after <= chunk) p1 = n + after;  // a short run: to its end
        else if (tile == 0 && x == 0) p.runs[1 + atomicAdd(p.runs, 1)] = static_cast<int>(c);
    }

    const int vec = (tile * p.tx + x) * E;
    if (vec >= p.pitch) return;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    for (int q0 = p0; q0 < p1; q0 += ROWS) {
        if (key[q0] >= p.vocab) break;  // no tokens from here on
        Shifted<T> v[ROWS];
        uint4 old[ACCUMULATE ? ROWS : 1][ACCUMULATE ? E / V : 1];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int q = q0 + r;
            if (q >= p1 || key[q] >= p.vocab) continue;
            const int col = ALIGNED ? vec : vec - p.phase.at<O>(key[q]);
            if (col >= p.dim) continue;
            const T *src = static_cast<const T *>(p.dout) + static_cast<long long>(s_row[y][q]) * p.ld_dout + col;
            if (ALIGNED) v[r].a = __ldg(reinterpret_cast<const uint4 *>(src));
            else v[r].load(src, p.lo, p.hi, col, p.dim);
            if (ACCUMULATE && key[q + 1] != key[q] && col >= 0 && col + E <= p.dim) {
                const uint4 *at = reinterpret_cast<const uint4 *>(static_cast<const O *>(p.dtable) +
                                                                  static_cast<long long>(key[q]) * p.ld_dtable + col);
#pragma unroll
                for (int h = 0; h < E / V; ++h) old[ACCUMULATE ? r : 0][ACCUMULATE ? h : 0] = at[h];
            }
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int q = q0 + r;
            if (q >= p1 || key[q] >= p.vocab) break;
            const int col = ALIGNED ? vec : vec - p.phase.at<O>(key[q]);
            if (col < p.dim) {
                float f[E];
                widen_vec<T>(ALIGNED ? v[r].a : v[r].get(), f);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += f[e];
            }
            const bool ends = key[q + 1] != key[q];
            if (!ends && q != p1 - 1) continue;
            if (ends && !began) {
                O *dst = static_cast<O *>(p.dtable) + static_cast<long long>(key[q]) * p.ld_dtable;
                float f[E];
#pragma unroll
                for (int e = 0; e < E; ++e) f[e] = acc[e] * p.scale;
                if (ACCUMULATE) {
                    if (col >= 0 && col + E <= p.dim) {
#pragma unroll
                        for (int h = 0; h < E / V; ++h) {
                            float g[V];
                            widen_vec<O>(old[ACCUMULATE ? r : 0][ACCUMULATE ? h : 0], g);
#pragma unroll
                            for (int e = 0; e < V; ++e) f[h * V + e] += g[e];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            if (col + e >= 0 && col + e < p.dim) f[e] += Elem<O>::get(dst[col + e]);
                    }
                }
                store_columns<O, E>(dst, col, p.dim, f);
            } else {
                float *out = p.partial + (2 * c + (began ? 0 : 1)) * p.pitch + vec;
#pragma unroll
                for (int e = 0; e < E; e += 4) *reinterpret_cast<float4 *>(out + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
            }
            began = false;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = 0.0f;
        }
    }
}

// Long runs: slot 1 of the chunk where one begins and the following chunks'
// slots 0.  Eight thread rows take every eighth part each, and their sums are
// added in order; four columns a thread.
template <typename O>
__global__ void __launch_bounds__(kSumThreads) embed_grad_join_kernel(const EmbedGradArgs p)
{
    constexpr int ROWS = 8, COLS = kSumThreads / ROWS;
    __shared__ float4 part_sum[ROWS][COLS];
    const int x = threadIdx.x % COLS, y = threadIdx.x / COLS;
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int runs = __ldcg(p.runs);
    for (int r = blockIdx.x; r < runs; r += gridDim.x) {
        const int c = __ldcg(p.runs + 1 + r);
        const int v = checked_key(p.keys, (c + 1) * p.chunk - 1, p.vocab);
        if (v >= p.vocab) continue;
        const int run_end = warp_lower_bound(p.keys, p.count, v + 1, threadIdx.x % 32);
        const int parts = (run_end - 1) / p.chunk - c + 1;
        O *dst = static_cast<O *>(p.dtable) + static_cast<long long>(v) * p.ld_dtable;
        const int shift = p.phase.at<O>(v);
        for (int q0 = blockIdx.y * COLS * 4; q0 - shift < p.dim; q0 += gridDim.y * COLS * 4) {
            const int q = q0 + 4 * x;
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (q - shift < p.dim) {
                const float *part = p.partial + 2ll * c * p.pitch + q;
#pragma unroll 8
                for (int k = y; k < parts; k += ROWS) {
                    const float4 w = __ldcg(reinterpret_cast<const float4 *>(part + (k ? 2ll * k : 1ll) * p.pitch));
                    s.x += w.x;
                    s.y += w.y;
                    s.z += w.z;
                    s.w += w.w;
                }
            }
            part_sum[y][x] = s;
            __syncthreads();
            if (y == 0) {
                float f[4] = {};
#pragma unroll
                for (int k = 0; k < ROWS; ++k) {
                    const float4 w = part_sum[k][x];
                    f[0] += w.x;
                    f[1] += w.y;
                    f[2] += w.z;
                    f[3] += w.w;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int col = q - shift + e;
                    if (col < 0 || col >= p.dim) continue;
                    const float old = p.accumulate ? Elem<O>::get(dst[col]) : 0.0f;
                    dst[col] = Elem<O>::put(fmaf(f[e], p.scale, old));
                }
            }
            __syncthreads();
        }
    }
}

// Workspace: keys and order twice (the passes alternate), digit counts,
// partial sums.
struct GradLayout {
    size_t keys[2], order[2], hist, runs, partial, bytes;
    int rounds, tiles, passes, digit, chunk, chunks, pitch;
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
    // chunks as long as leave a few hundred thousand threads (of eight columns)
    l.chunk = kMaxChunk;
    while (l.chunk > 16 && count * dim / 8 / l.chunk < 400000) l.chunk /= 2;
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
    l.runs = take((1 + static_cast<size_t>(l.chunks)) * 4);
    l.pitch = dim / 8 * 8 + 16;  // whole vectors, and one more for a row's phase
    l.partial = take(static_cast<size_t>(l.chunks) * 2 * l.pitch * 4);
    l.bytes = at;
    return l;
}

bool grad_sizes_ok(long long count, int vocab, int dim)
{
    return count >= 0 && count < (1ll << 30) && vocab >= 1 && vocab < INT_MAX && dim >= 1 && dim <= kMaxDim;
}

template <int ROUNDS>
cudaError_t launch_sort_pass(const SortPass &p, cudaStream_t s)
{
    cudaError_t e;
    if (p.tokens) {  // the call's first launch
        sort_count_kernel<ROUNDS><<<p.tiles, kSortThreads, 0, s>>>(p);
        e = cudaGetLastError();
    } else {
        e = launch_early(sort_count_kernel<ROUNDS>, dim3(p.tiles), dim3(kSortThreads), 0, s, p);
    }
    return e != cudaSuccess ? e : launch_early(sort_place_kernel<ROUNDS>, dim3(p.tiles), dim3(kSortThreads), 0, s, p);
}

cudaError_t launch_rank(const SortPass &p, cudaStream_t s)
{
    const int smem = (p.count + 3) / 4 * 16;
    // the more lanes a token the more CTAs, which all read the whole list
    if (p.count <= kRankMax / 2) sort_rank_kernel<32><<<(p.count + 7) / 8, kSortThreads, smem, s>>>(p);
    else sort_rank_kernel<8><<<(p.count + 31) / 32, kSortThreads, smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T, typename O>
cudaError_t launch_sums(EmbedGradArgs a, cudaStream_t s)
{
    constexpr int E = kPerVec<T>;
    // every row of both matrices starts on 16 bytes
    const bool aligned = a.dim % E == 0 && a.ld_dout % E == 0 && a.ld_dtable % kPerVec<O> == 0 && aligned_to(a.dout, 16) &&
                         aligned_to(a.dtable, 16);
    a.phase = Phase::of<O>(a.dtable, a.ld_dtable);
    const int n = (a.dim + E - 1) / E + (aligned ? 0 : 1);  // vectors a row, at most
    a.tx = 32;
    while (a.tx < kSumThreads && a.tx < n) a.tx *= 2;
    a.col_tiles = (n + a.tx - 1) / a.tx;
    const int ty = kSumThreads / a.tx;
    const long long sum = (a.chunks + ty - 1ll) / ty * a.col_tiles;
    const int zero_rows = kSumThreads / 32 * kZeroRows;
    const long long zero = a.accumulate ? 0 : (a.vocab + zero_rows - 1ll) / zero_rows;
    if (sum + zero >= (1ll << 31)) return cudaErrorInvalidConfiguration;
    a.sum_ctas = static_cast<unsigned>(sum);
    a.zero_ctas = static_cast<unsigned>(zero);
    const dim3 grid(a.sum_ctas + a.zero_ctas), block(kSumThreads);
    cudaError_t e = cudaSuccess;
    if (grid.x > 0)
        e = aligned ? (a.accumulate ? launch_early(embed_grad_kernel<T, O, true, true>, grid, block, 0, s, a)
                                    : launch_early(embed_grad_kernel<T, O, true, false>, grid, block, 0, s, a))
                    : (a.accumulate ? launch_early(embed_grad_kernel<T, O, false, true>, grid, block, 0, s, a)
                                    : launch_early(embed_grad_kernel<T, O, false, false>, grid, block, 0, s, a));
    if (e == cudaSuccess && a.chunks > 1)
        e = launch_early(embed_grad_join_kernel<O>, dim3(std::min(a.chunks, 128), std::min(32, (a.pitch + 63) / 64)), block, 0,
                         s, a);
    return e;
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
    EmbedArgs a{};
    a.table = table;
    a.tokens = tokens;
    a.out = out;
    a.ld_table = ld_table;
    a.ld_out = ld_out;
    a.count = count;
    a.index_bytes = index_bytes;
    a.vocab = vocab;
    a.dim = dim;
    a.scale = scale;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == CDG_F32) launch_embed<float>(a, sms, s);
    else if (dtype == CDG_F16) launch_embed<__half>(a, sms, s);
    else launch_embed<__nv_bfloat16>(a, sms, s);
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
               reinterpret_cast<int *>(ws + l.hist), reinterpret_cast<int *>(ws + l.runs), index_bytes, static_cast<int>(count), vocab, 0, 1 << l.digit, l.tiles};
    if (count > 0 && count <= kRankMax) {
        if (launch_rank(p, s) != cudaSuccess) return CDG_ERR_CUDA;
    } else if (count > 0) {
        for (int q = 0; q < l.passes; ++q) {
            p.tokens = q == 0 ? tokens : nullptr;
            p.keys = keys;
            p.order = order;
            p.keys_out = reinterpret_cast<int *>(ws + l.keys[q & 1]);
            p.order_out = reinterpret_cast<int *>(ws + l.order[q & 1]);
            p.shift = q * l.digit;
            if ((l.rounds == 4 ? launch_sort_pass<4>(p, s) : launch_sort_pass<16>(p, s)) != cudaSuccess) return CDG_ERR_CUDA;
            keys = p.keys_out;
            order = p.order_out;
        }
    }
    EmbedGradArgs a{};
    a.dout = dout;
    a.dtable = dtable;
    a.ld_dout = ld_dout;
    a.ld_dtable = ld_dtable;
    a.keys = keys;
    a.order = order;
    a.partial = reinterpret_cast<float *>(ws + l.partial);
    a.runs = reinterpret_cast<int *>(ws + l.runs);
    a.count = static_cast<int>(count);
    a.vocab = vocab;
    a.dim = dim;
    a.accumulate = accumulate;
    a.chunk = l.chunk;
    a.chunks = l.chunks;
    a.pitch = l.pitch;
    a.lo = static_cast<const char *>(dout);
    a.hi = a.lo + matrix_bytes(count, dim, ld_dout, es);
    a.scale = scale;
    const cudaError_t e = dtype == CDG_F32   ? launch_sums<float, float>(a, s)
                          : dtype == CDG_F16 ? (out_f32 ? launch_sums<__half, float>(a, s) : launch_sums<__half, __half>(a, s))
                          : out_f32          ? launch_sums<__nv_bfloat16, float>(a, s)
                                             : launch_sums<__nv_bfloat16, __nv_bfloat16>(a, s);
    return e == cudaSuccess ? CDG_OK : CDG_ERR_CUDA;
}

}  // extern "C"
