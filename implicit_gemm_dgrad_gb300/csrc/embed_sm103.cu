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
constexpr int kTile = 4096, kSortThreads = 256, kMaxBins = 512;
constexpr int kWarps = kSortThreads / 32, kPerWarpKeys = kTile / kWarps;

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

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortPass p)
{
    __shared__ int h[kMaxBins];
    for (int d = threadIdx.x; d < p.bins; d += kSortThreads) h[d] = 0;
    __syncthreads();
    const int i0 = blockIdx.x * kTile, i1 = min(i0 + kTile, p.count);
    for (int i = i0 + threadIdx.x; i < i1; i += kSortThreads) atomicAdd(&h[(sort_key(p, i) >> p.shift) & (p.bins - 1)], 1);
    __syncthreads();
    for (int d = threadIdx.x; d < p.bins; d += kSortThreads) p.hist[static_cast<long long>(blockIdx.x) * p.bins + d] = h[d];
}

// Places a tile's keys: digit d of tile t starts after all smaller digits and
// after digit d of the tiles before t.  Warp w takes keys [512 w, 512 w + 512)
// of the tile, 32 at a time, in order: the sort is stable.
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const SortPass p)
{
    __shared__ int start[kMaxBins];
    __shared__ int cnt[kWarps][kMaxBins];
    __shared__ int wsum[kWarps];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    // totals and this tile's prefix, two digits a thread
    const int d0 = 2 * tid, d1 = d0 + 1;
    int tot0 = 0, tot1 = 0, before0 = 0, before1 = 0;
    if (d0 < p.bins)
        for (int t = 0; t < p.tiles; ++t) {
            const int2 h = __ldg(reinterpret_cast<const int2 *>(p.hist + static_cast<long long>(t) * p.bins + d0));
            if (t < static_cast<int>(blockIdx.x)) {
                before0 += h.x;
                before1 += h.y;
            }
            tot0 += h.x;
            tot1 += h.y;
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
    const int i0 = blockIdx.x * kTile + warp * kPerWarpKeys;
    int key[kPerWarpKeys / 32], rank[kPerWarpKeys / 32];
#pragma unroll
    for (int k = 0; k < kPerWarpKeys / 32; ++k) {
        const int i = i0 + k * 32 + lane;
        key[k] = i < p.count ? sort_key(p, i) : -1;
    }
#pragma unroll
    for (int k = 0; k < kPerWarpKeys / 32; ++k) {
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
        for (int w = 0; w < kWarps; ++w) {
            const int c = cnt[w][d];
            cnt[w][d] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPerWarpKeys / 32; ++k) {
        const int i = i0 + k * 32 + lane;
        if (i >= p.count) break;
        const int at = cnt[warp][(key[k] >> p.shift) & (p.bins - 1)] + rank[k];
        p.keys_out[at] = key[k];
        p.order_out[at] = p.tokens ? i : p.order[i];
    }
}

// ---------------------------------------------------------------- sums
struct EmbedGradArgs {
    const void *dout;
    void *dtable;
    long long ld_dout, ld_dtable;
    const int *keys, *order;  // sorted tokens and their positions
    int count, vocab, dim, accumulate;
    float scale;
};

// First position with keys[i] >= v.
__device__ __forceinline__ int lower_bound(const int *keys, int count, int v)
{
    int lo = 0, hi = count;
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (__ldg(keys + mid) < v) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// One CTA per table row.
template <typename T, typename O>
__global__ void __launch_bounds__(256) embed_grad_kernel(const EmbedGradArgs p)
{
    const int v = blockIdx.x;
    const int a = lower_bound(p.keys, p.count, v), b = lower_bound(p.keys, p.count, v + 1);
    if (p.accumulate && a == b) return;
    O *dst = static_cast<O *>(p.dtable) + static_cast<long long>(v) * p.ld_dtable;
    for (int j = threadIdx.x; j < p.dim; j += 256) {
        float s = 0.0f;
        for (int i = a; i < b; ++i)
            s += Elem<T>::get(static_cast<const T *>(p.dout)[static_cast<long long>(__ldg(p.order + i)) * p.ld_dout + j]);
        s *= p.scale;
        if (p.accumulate) s += Elem<O>::get(dst[j]);
        dst[j] = Elem<O>::put(s);
    }
}

// Workspace: keys and order twice (the passes alternate), digit counts.
struct GradLayout {
    size_t keys[2], order[2], hist, bytes;
    int tiles, passes, digit;
};
GradLayout grad_layout(long long count, int vocab)
{
    GradLayout l;
    int bits = 1;
    while ((1ll << bits) <= vocab) ++bits;  // keys 0 .. vocab
    l.passes = (bits + 8) / 9;
    l.digit = std::max(1, (bits + l.passes - 1) / l.passes);
    l.tiles = static_cast<int>((count + kTile - 1) / kTile);
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t was = at;
        at += (n + 255) / 256 * 256;
        return was;
    };
    for (int i = 0; i < 2; ++i) {
        l.keys[i] = take(static_cast<size_t>(count) * 4);
        l.order[i] = take(static_cast<size_t>(count) * 4);
    }
    l.hist = take(static_cast<size_t>(l.tiles) * (1u << l.digit) * 4);
    l.bytes = at;
    return l;
}

bool grad_sizes_ok(long long count, int vocab, int dim)
{
    return count >= 0 && count < (1ll << 30) && vocab >= 1 && vocab < INT_MAX && dim >= 1 && dim <= kMaxDim;
}

template <typename T, typename O>
void launch_sums(const EmbedGradArgs &a, cudaStream_t s)
{
    embed_grad_kernel<T, O><<<a.vocab, 256, 0, s>>>(a);
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
    return cdg::grad_sizes_ok(count, vocab, dim) ? std::max<size_t>(16, cdg::grad_layout(count, vocab).bytes) : 0;
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
    const GradLayout l = grad_layout(count, vocab);
    const Extent o = extent(dtable, matrix_bytes(vocab, dim, ld_dtable, os)), w = extent(workspace, std::max<size_t>(16, l.bytes));
    const Extent in[2] = {extent(dout, matrix_bytes(count, dim, ld_dout, es)),
                          extent(tokens, static_cast<size_t>(count) * index_bytes)};
    if (overlap(o, w) || overlap(o, in[0]) || overlap(o, in[1]) || overlap(w, in[0]) || overlap(w, in[1]))
        return CDG_ERR_ALIAS;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    const int *keys = reinterpret_cast<int *>(ws + l.keys[0]), *order = reinterpret_cast<int *>(ws + l.order[0]);
    for (int q = 0; q < l.passes && count > 0; ++q) {
        int *ko = reinterpret_cast<int *>(ws + l.keys[q & 1]), *oo = reinterpret_cast<int *>(ws + l.order[q & 1]);
        const SortPass p{q == 0 ? tokens : nullptr, keys, order, ko, oo, reinterpret_cast<int *>(ws + l.hist), index_bytes,
                         static_cast<int>(count), vocab, q * l.digit, 1 << l.digit, l.tiles};
        sort_count_kernel<<<l.tiles, kSortThreads, 0, s>>>(p);
        sort_place_kernel<<<l.tiles, kSortThreads, 0, s>>>(p);
        keys = ko;
        order = oo;
    }
    const EmbedGradArgs a{dout, dtable, ld_dout, ld_dtable, keys, order, static_cast<int>(count), vocab, dim, accumulate,
                          scale};
    if (dtype == CDG_F32) launch_sums<float, float>(a, s);
    else if (dtype == CDG_F16) out_f32 ? launch_sums<__half, float>(a, s) : launch_sums<__half, __half>(a, s);
    else out_f32 ? launch_sums<__nv_bfloat16, float>(a, s) : launch_sums<__nv_bfloat16, __nv_bfloat16>(a, s);
    return cudaGetLastError() == cudaSuccess ? CDG_OK : CDG_ERR_CUDA;
}

}  // extern "C"
