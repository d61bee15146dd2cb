// Token log probabilities for sm_103a, and their gradient: kernels and C entry
// points.
//
// Forward.  With c = scale * log2(e), every element of a row is read once:
//
//   ref                         the largest z_j c so far (rounded)
//   s = sum 2^(z_j c - ref),   e = sum 2^(z_j c - ref) (z_j c - ref)
//
// and when a thread's group of vectors holds a larger value, s and e move to
// the new reference: with r = 2^(ref - ref'), s' = s r and
// e' = r (e + (ref - ref') s).  The reference is the rounded product itself, so
// its rounding is known: lse = scale zmax + ln2 (log2 s - (zmax c - ref)), one
// rounding of lse's size (ln2 (ref + log2 s) takes three), and the entropy is
// ln2 (log2 s - e / s).  Threads, warps and the CTAs of a cluster are joined by
// the same rule, in a fixed order.
//
// What bounds it: DRAM (one read of the logits) if the instructions an element
// takes fit beside it; at 6.8 TB/s an SM has about 11 a lane for every 16-bit
// logit.  So the sums run on fp32 pairs (one instruction for two), the largest
// and smallest of a group on packed 16-bit pairs, and only the first warp of a
// CTA joins the others' sums (all of them doing so cost 20 us of 105 at 8192 x
// 32000).  256 threads and 40 registers leave six rows in flight an SM, whose
// joins overlap the others' reads.  Measured: 8192 x 32000 bf16 85 us (6.2 TB/s),
// fp32 153 us (6.8 TB/s), 65536 x 1000 bf16 39 us; one row of 131072 3.8 us, by
// a cluster of eight CTAs that push their sums to the first one (a second
// exchange would cost another microsecond).  A row that takes the second pass
// (nothing but finite masks): one of 131072 73 us, 8192 x 32000 of them 206 us.
//
// The largest logits: each thread keeps the maximum of its elements (the
// running maximum above, needed anyway).  The k-th largest of some thread
// maxima is at most the k-th largest element, so only threads whose maximum
// reaches that bound look at their elements again (in L2) and list those that
// reach it: a few dozen, ranked by counting larger 64-bit keys (ordered value,
// then lowest number).  If more than kCand reach it (many equal values) each
// warp instead keeps an exact sorted list of its k largest keys in one scan.
// That adds 3.3 us to a single row (8 of them) and 61 us to 8192 x 32000 (20).
//
// Gradient.  One read and one write of every element, nothing joined: 8192 x
// 32000 bf16 152 us (6.9 TB/s), 6145 x 50021 (rows at every alignment) 190 us with
// the entropy's term, 182 without; 504 us where a row of the logits and its row of
// the gradient lie differently in 16 bytes, and go element by element.
#include <cmath>

#include "ptx.cuh"
#include "token_device.cuh"

namespace cdg {
namespace {

constexpr int kMaxTop = 32;
constexpr int kMaxVocab = 1 << 30;  // element numbers stay in 32 bits
constexpr int kThreads = 256;
constexpr int kCand = 1024;         // candidate keys a CTA ranks
constexpr int kMaxCluster = kThreads / 32;  // CTAs that share a row (a warp for each one's keys at the end)
constexpr int kUnroll = 4;          // 16-byte loads in flight per thread
constexpr int kCtasPerSm = 6;
constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.44269504088896341f;
constexpr float kFloor = -1000.0f;  // 2^-1000 is 0 in fp32: exponents are clamped here so that 0 * -inf does not arise
// The lowest reference.  Beyond 2^24 the rounding of z c alone is more than a
// half, beyond 2^31 more than an fp32 exponent holds: the sums of a thread that
// has met nothing but masked entries (-1e10, the type's lowest value) would be
// inf, and NaN once joined.  About this reference they are 0 instead, as they
// are beside any logit that is not as far out.  Rows whose largest logit comes
// within a factor of two of it, on either side of zero, take a second pass.
constexpr float kLowest = -16777216.0f;

struct LogprobArgs {
    const void *logits, *targets;
    long long ld, rows;
    int index_bytes, vocab, top, cluster;
    float scale, c;  // c = scale * log2(e)
    float *logp, *lse, *entropy, *top_logp;
    int *top_ids;
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// max and min that keep a NaN operand (fmaxf and fminf drop it)
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float min_nan(float a, float b)
{
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Two fp32 numbers in one register pair: one instruction for both.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A row's sums about the reference zmax c (rounded), zmax the largest logit of
// those summed.
struct Sums {
    float zmax, s, e;
};
// (__fmul_rn: a product contracted into an addition would be another reference)
__device__ __forceinline__ float reference(float zmax, float c) { return zmax == -INFINITY ? 0.0f : __fmul_rn(zmax, c); }

// Sums moved to a larger largest logit.
__device__ __forceinline__ void move_to(Sums &a, float zmax, float c)
{
    const float d = a.zmax == -INFINITY ? 0.0f : fmaxf(__fmul_rn(a.zmax, c) - __fmul_rn(zmax, c), kFloor);  // none yet: s = e = 0
    const float r = exp2_fast(d);
    a.e = r * fmaf(d, a.s, a.e);
    a.s *= r;
    a.zmax = zmax;
}

// Float order as unsigned order (-0 and +0 equal); 0 is below every number.
__device__ __forceinline__ uint32_t ordered(float f)
{
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u)
{
    return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
// Largest of the warp's (NaN stays out: it never enters a zmax).
__device__ __forceinline__ float warp_max(float z) { return unordered(__reduce_max_sync(0xFFFFFFFFu, ordered(z))); }
// The warp's sums, in every lane.
__device__ __forceinline__ Sums join_lanes(Sums a, float c)
{
    move_to(a, warp_max(a.zmax), c);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a.s += __shfl_xor_sync(0xFFFFFFFFu, a.s, o);
        a.e += __shfl_xor_sync(0xFFFFFFFFu, a.e, o);
    }
    return a;
}
// Larger key = larger value, then lower element number.  Never 0.
__device__ __forceinline__ unsigned long long make_key(float z, int j)
{
    return (static_cast<unsigned long long>(ordered(z)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(j));
}
__device__ __forceinline__ int key_index(unsigned long long k) { return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k)); }

// Element-wise largest and smallest of two words (NaN elements may be dropped).
template <typename T>
struct Words;
template <>
struct Words<float> {
    static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) { return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b))); }
    static __device__ __forceinline__ uint32_t min(uint32_t a, uint32_t b) { return __float_as_uint(fminf(__uint_as_float(a), __uint_as_float(b))); }
};
template <>
struct Words<__half> {
    static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b)
    {
        const __half2 r = __hmax2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
    static __device__ __forceinline__ uint32_t min(uint32_t a, uint32_t b)
    {
        const __half2 r = __hmin2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
};
template <>
struct Words<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b)
    {
        const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
    static __device__ __forceinline__ uint32_t min(uint32_t a, uint32_t b)
    {
        const __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
};
template <typename T>
__device__ __forceinline__ float max_word(uint32_t w)
{
    float f[2];
    widen<T>(w, f);
    return sizeof(T) == 4 ? f[0] : fmaxf(f[0], f[1]);
}
template <typename T>
__device__ __forceinline__ float min_word(uint32_t w)
{
    float f[2];
    widen<T>(w, f);
    return sizeof(T) == 4 ? f[0] : fminf(f[0], f[1]);
}

// The part of a row that this CTA reads: 16-byte vectors from an aligned
// address, and up to one vector's worth of single elements before the first
// (CTA 0 of the row) and after the last (its last CTA).
template <typename T>
struct Slice {
    const T *row;
    int v0, nv;      // vectors: element numbers v0 + i * kPerVec
    int head, tail0, tail;

    __device__ __forceinline__ Slice(const T *r, int vocab, int rank, int nrank) : row(r)
    {
        constexpr int E = kPerVec<T>;
        const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(r) & 15u) / sizeof(T));
        const int h = min(mis ? E - mis : 0, vocab);
        const int all = (vocab - h) / E;
        const int a = static_cast<int>(static_cast<long long>(all) * rank / nrank);
        const int b = static_cast<int>(static_cast<long long>(all) * (rank + 1) / nrank);
        v0 = h + a * E;
        nv = b - a;
        head = rank == 0 ? h : 0;
        tail0 = h + all * E;
        tail = rank == nrank - 1 ? vocab - tail0 : 0;
    }
    __device__ __forceinline__ uint4 vec(int i) const
    {
        return __ldg(reinterpret_cast<const uint4 *>(row + v0) + i);
    }
    // number of the single element thread t holds, or -1
    __device__ __forceinline__ int single(int t) const
    {
        if (t < head) return t;
        t -= kPerVec<T>;
        return t >= 0 && t < tail ? tail0 + t : -1;
    }
};

// A thread's running sums while it reads: s and e as two numbers each (even
// and odd elements), about ref, the larger of kLowest and zmax c.
struct Run {
    float ref, zmax;
    f32x2 s, e;
};

// The reference moves up to y.
__device__ __forceinline__ void raise(Run &a, float y)
{
    if (y > a.ref) {  // (false for NaN)
        const float d = fmaxf(a.ref - y, kFloor), r = exp2_fast(d);
        const f32x2 rr = pack2(r, r);
        a.e = mul2(rr, fma2(pack2(d, d), a.s, a.e));
        a.s = mul2(rr, a.s);
        a.ref = y;
    }
}
// Two logits.  CLAMP: one may lie far below the reference, or be -inf.
template <bool CLAMP>
__device__ __forceinline__ void add(Run &a, float z0, float z1, f32x2 c, f32x2 minus_ref)
{
    f32x2 u = fma2(pack2(z0, z1), c, minus_ref);
    float u0, u1;
    unpack2(u, u0, u1);
    if (CLAMP) {
        u0 = max_nan(u0, kFloor);
        u1 = max_nan(u1, kFloor);
        u = pack2(u0, u1);
    }
    const f32x2 w = pack2(exp2_fast(u0), exp2_fast(u1));
    a.s = add2(a.s, w);
    a.e = fma2(w, u, a.e);
}
template <typename T, bool CLAMP, int N>
__device__ __forceinline__ void add_all(Run &a, const uint4 (&v)[N], float c)
{
    const f32x2 cc = pack2(c, c), minus = pack2(-a.ref, -a.ref);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float f[kPerVec<T>];
        widen_vec<T>(v[i], f);
#pragma unroll
        for (int j = 0; j < kPerVec<T>; j += 2) add<CLAMP>(a, f[j], f[j + 1], cc, minus);
    }
}
// Returns the largest of the group.
template <typename T, int N>
__device__ __forceinline__ float add_group(Run &a, const uint4 (&v)[N], float c)
{
    using W = Words<T>;
    uint32_t hi = W::max(W::max(v[0].x, v[0].y), W::max(v[0].z, v[0].w));
#pragma unroll
    for (int i = 1; i < N; ++i) hi = W::max(hi, W::max(W::max(v[i].x, v[i].y), W::max(v[i].z, v[i].w)));
    const float g = max_word<T>(hi);
    a.zmax = fmaxf(a.zmax, g);
    raise(a, __fmul_rn(g, c));
    if constexpr (sizeof(T) == 2) {
        // the smallest of the group costs half an instruction an element, the clamp a whole one
        uint32_t lo = W::min(W::min(v[0].x, v[0].y), W::min(v[0].z, v[0].w));
#pragma unroll
        for (int i = 1; i < N; ++i) lo = W::min(lo, W::min(W::min(v[i].x, v[i].y), W::min(v[i].z, v[i].w)));
        if (fmaf(min_word<T>(lo), c, -a.ref) > kFloor) {
            add_all<T, false>(a, v, c);
            return g;
        }
    }
    add_all<T, true>(a, v, c);
    return g;
}

// Insert warp-uniform key x into the warp's descending list (lane l holds its
// l-th largest key).
__device__ __forceinline__ void list_insert(unsigned long long &mine, unsigned long long x, int lane)
{
    const unsigned larger = __ballot_sync(0xFFFFFFFFu, mine > x);
    const int pos = __popc(larger);
    const unsigned long long up = __shfl_up_sync(0xFFFFFFFFu, mine, 1);
    if (lane == pos) mine = x;
    else if (lane > pos) mine = up;
}

// keys[0..n) -> the min(n, k) largest in out, descending.  Returns that count.
template <int TEAM>
__device__ __forceinline__ int rank_keys(const unsigned long long *keys, int n, int k, unsigned long long *out, int tid)
{
    for (int i = tid; i < n; i += TEAM) {
        const unsigned long long x = keys[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) rank += keys[j] > x;
        if (rank < k) out[rank] = x;
    }
    return min(n, k);
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// How many of the descending keys[0..n) are larger than x (n <= 32).
__device__ __forceinline__ int count_larger(const unsigned long long *keys, int n, unsigned long long x)
{
    int at = 0;
#pragma unroll
    for (int step = 32; step; step >>= 1)
        if (at + step <= n && keys[at + step - 1] > x) at += step;
    return at;
}

// TEAM threads a row: a warp each of eight rows, or the CTA, which a cluster of
// CTAs may share the row with.  TOP: alternatives are wanted.
template <typename T, int TEAM, bool TOP>
__global__ void __launch_bounds__(kThreads, TEAM == 32 ? 4 : kCtasPerSm) logprobs_kernel(const LogprobArgs p)
{
    constexpr bool WARP = TEAM == 32;
    constexpr int W = TEAM / 32, TEAMS = kThreads / TEAM, CAND = kCand / TEAMS;
    constexpr int PER_WARP = kMaxTop / W;  // thread maxima each warp offers
    __shared__ Sums part[W];
    __shared__ unsigned long long s_cand[TEAMS][CAND], s_best[TEAMS][kMaxTop];
    __shared__ uint32_t offer[kMaxTop];
    __shared__ int s_ncand[TEAMS];
    // what the cluster's other CTAs leave with the first one
    __shared__ Sums from_sums[kMaxCluster];
    __shared__ unsigned long long from_keys[kMaxCluster][kMaxTop];
    __shared__ int from_count[kMaxCluster];

    const int lane = threadIdx.x % 32, tid = threadIdx.x % TEAM, warp = tid / 32, team = threadIdx.x / TEAM;
    const int rank = !WARP && p.cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const long long i = WARP ? static_cast<long long>(blockIdx.x) * TEAMS + team : blockIdx.x / p.cluster;
    if (!WARP && p.cluster > 1) cluster_arrive();  // every CTA of the cluster has started before one writes to the first
    if (WARP && i >= p.rows) return;
    auto sync = [] {
        if (WARP) __syncwarp();
        else __syncthreads();
    };
    unsigned long long *const cand = s_cand[team], *const best = s_best[team];
    int *const ncand = s_ncand + team;
    const Slice<T> sl(static_cast<const T *>(p.logits) + i * p.ld, p.vocab, rank, WARP ? 1 : p.cluster);

    const int single = sl.single(tid);
    const auto vec_at = [&](int v) { return sl.vec(v + tid); };

    // ---- one pass: sums and the thread's maximum
    Run run{kLowest, -INFINITY, 0ull, 0ull};
    uint4 x[kUnroll];
    // TOP: the group of vectors that holds the thread's largest logit, and the largest of its other groups
    float top_group = -INFINITY, other_groups = -INFINITY;
    int top_at = 0;
    auto note = [&](float g, int at) {
        if (!TOP) return;
        if (g > top_group) {
            other_groups = top_group;
            top_group = g;
            top_at = at;
        } else {
            other_groups = fmaxf(other_groups, g);
        }
    };
    int v = 0;
    for (; v + kUnroll * TEAM <= sl.nv; v += kUnroll * TEAM) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) x[u] = vec_at(v + u * TEAM);
        note(add_group<T, kUnroll>(run, x, p.c), v);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        if (v + u * TEAM + tid < sl.nv) x[u] = vec_at(v + u * TEAM);
    if (single >= 0) {
        const float z = Elem<T>::get(sl.row[single]);
        run.zmax = fmaxf(run.zmax, z);
        raise(run, __fmul_rn(z, p.c));
        add<true>(run, z, -INFINITY, pack2(p.c, p.c), pack2(-run.ref, -run.ref));
    }
    float last = -INFINITY;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        if (v + u * TEAM + tid < sl.nv) {
            const uint4 y[1] = {x[u]};
            last = fmaxf(last, add_group<T, 1>(run, y, p.c));
        }
    note(last, v);
    // the target's logit, on its way while the sums are joined
    int target = -1;
    float z_target = 0.0f;
    if (tid == 0 && rank == 0 && p.logp) {
        target = token_at(p.targets, p.index_bytes, i, p.vocab);
        if (target >= 0) z_target = Elem<T>::get(sl.row[target]);
    }
    // no element at all in this thread: below every element
    const uint32_t omax = single >= 0 || tid < sl.nv ? ordered(run.zmax) : 0u;

    // ---- join the team: the CTA's sums end in its first warp
    float s0, s1, e0, e1;
    unpack2(run.s, s0, s1);
    unpack2(run.e, e0, e1);
    Sums all = join_lanes(Sums{run.zmax, s0 + s1, e0 + e1}, p.c);
    uint32_t mo = omax;  // lane l: one of 32 thread maxima
    if (TOP && tid == 0) *ncand = 0;
    if (!WARP) {
        if (lane == 0) part[warp] = all;
        if (TOP) {
            // a round more than gives `top` offers: the bound is closer, and fewer candidates reach it
            const int rounds = min(PER_WARP, (p.top + W - 1) / W + 1);
            uint32_t m = omax;
            for (int r = 0; r < PER_WARP; ++r) {
                uint32_t g = 0u;
                if (r < rounds) {
                    g = __reduce_max_sync(0xFFFFFFFFu, m);
                    const unsigned holders = __ballot_sync(0xFFFFFFFFu, m == g);
                    if (lane == __ffs(holders) - 1) m = 0u;
                }
                if (lane == 0) offer[warp * PER_WARP + r] = g;
            }
        }
        __syncthreads();
        if (warp == 0) all = join_lanes(lane < W ? part[lane] : Sums{-INFINITY, 0.0f, 0.0f}, p.c);
        if (TOP) mo = offer[lane];
    } else if (TOP) {
        __syncwarp();
    }

    // ---- the team's largest logits
    int nbest = 0;
    if constexpr (TOP) {
        int larger = 0;
#pragma unroll
        for (int l = 0; l < 32; ++l) {
            const uint32_t o = __shfl_sync(0xFFFFFFFFu, mo, l);
            larger += o > mo || (o == mo && l < lane);
        }
        const int at = __ffs(__ballot_sync(0xFFFFFFFFu, larger == p.top - 1)) - 1;
        const uint32_t bound = __shfl_sync(0xFFFFFFFFu, mo, at);
        if (omax >= bound && omax) {
            auto offer_one = [&](float z, int j) {
                if (ordered(z) >= bound) {
                    const int n = atomicAdd(ncand, 1);
                    if (n < CAND) cand[n] = make_key(z, j);
                }
            };
            if (single >= 0) offer_one(Elem<T>::get(sl.row[single]), single);
            const volatile int *listed = ncand;
            // mostly one group of the thread reaches the bound; (a row of less than a full group is still in x)
            const bool one = ordered(other_groups) < bound;
            for (int w = one ? top_at : 0; w < sl.nv && *listed <= CAND; w += kUnroll * TEAM) {
                if (sl.nv >= kUnroll * TEAM) {
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u)
                        if (w + u * TEAM + tid < sl.nv) x[u] = vec_at(w + u * TEAM);
                }
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int q = w + u * TEAM + tid;
                    if (q >= sl.nv) break;
                    const uint32_t hi = Words<T>::max(Words<T>::max(x[u].x, x[u].y), Words<T>::max(x[u].z, x[u].w));
                    if (ordered(max_word<T>(hi)) < bound) continue;
                    float f[kPerVec<T>];
                    widen_vec<T>(x[u], f);
#pragma unroll
                    for (int e = 0; e < kPerVec<T>; ++e) offer_one(f[e], sl.v0 + q * kPerVec<T> + e);
                }
                if (one) break;
            }
        }
        sync();
        int n = *ncand;
        if (n > CAND) {
            // many equal values: exact lists, one per warp (keys start at 0: below every key)
            sync();
            unsigned long long list = 0;
            auto offer_all = [&](unsigned long long key) {
                unsigned b = __ballot_sync(0xFFFFFFFFu, key > __shfl_sync(0xFFFFFFFFu, list, p.top - 1));
                while (b) {
                    const int l = __ffs(b) - 1;
                    b &= b - 1;
                    const unsigned long long y = __shfl_sync(0xFFFFFFFFu, key, l);
                    if (y > __shfl_sync(0xFFFFFFFFu, list, p.top - 1)) list_insert(list, y, lane);
                }
            };
            offer_all(single >= 0 ? make_key(Elem<T>::get(sl.row[single]), single) : 0ull);
            for (int u0 = warp * 32; u0 < sl.nv; u0 += TEAM) {
                const int u = u0 + lane;
                float f[kPerVec<T>];
                const bool real = u < sl.nv;
                widen_vec<T>(real ? sl.vec(u) : make_uint4(0u, 0u, 0u, 0u), f);
#pragma unroll
                for (int e = 0; e < kPerVec<T>; ++e)
                    offer_all(real ? make_key(f[e], sl.v0 + u * kPerVec<T> + e) : 0ull);
            }
            if (lane < p.top) cand[warp * p.top + lane] = list;
            n = W * p.top;
            sync();
        }
        nbest = rank_keys<TEAM>(cand, n, p.top, best, tid);
        sync();
    }

    // ---- join the row's CTAs: the others leave their sums and keys with the first
    if (!WARP && p.cluster > 1) {
        cluster_wait();
        if (rank) {
            if (tid == 0) {
                const uint32_t to = mapa_shared(smem_u32(&from_sums[rank]), 0);
                st_cluster_u32(to, __float_as_uint(all.zmax));
                st_cluster_u32(to + 4, __float_as_uint(all.s));
                st_cluster_u32(to + 8, __float_as_uint(all.e));
                st_cluster_u32(mapa_shared(smem_u32(&from_count[rank]), 0), static_cast<uint32_t>(nbest));
            }
            if (tid < nbest) st_cluster_u64(mapa_shared(smem_u32(&from_keys[rank][tid]), 0), best[tid]);
            __syncwarp();
            cluster_arrive();
            return;
        }
        if (tid == 0) from_sums[0] = all;
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (warp == 0) all = join_lanes(lane < p.cluster ? from_sums[lane] : Sums{-INFINITY, 0.0f, 0.0f}, p.c);
        if (TOP) {
            // a list a warp, a key a lane: its rank is its own place and what the other lists hold above it (counting
            // over all keys instead took 1.3 thousand cycles longer)
            if (tid < nbest) from_keys[0][tid] = best[tid];
            if (tid == 0) from_count[0] = nbest;
            __syncthreads();
            if (warp < p.cluster && lane < from_count[warp]) {
                const unsigned long long key = from_keys[warp][lane];
                int place = lane;
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q)  // independent searches, side by side
                    place += count_larger(from_keys[q], q < p.cluster && q != warp ? from_count[q] : 0, key);
                if (place < p.top) best[place] = key;
            }
            __syncthreads();
        }
    }

    if (warp != 0) return;  // the first warp of the team has the sums and writes the row's answers

    // The largest logit is finite, its product with c far from zero or infinite
    // (e.g. a row masked with -1e9 or the type's lowest value): sums about the logit
    // itself, in a second pass by this warp alone.
    const bool extreme = fabsf(all.zmax) < INFINITY && !(fabsf(all.zmax * p.c) < -kLowest / 2);
    if (extreme) {
        all.s = all.e = 0.0f;
        for (int j = lane; j < p.vocab; j += 32) {
            // (not times c, which passes fp32 for the largest scales)
            const float u = max_nan((Elem<T>::get(sl.row[j]) - all.zmax) * p.scale * kLog2e, kFloor), w = exp2_fast(u);
            all.s += w;
            all.e = fmaf(w, u, all.e);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            all.s += __shfl_xor_sync(0xFFFFFFFFu, all.s, o);
            all.e += __shfl_xor_sync(0xFFFFFFFFu, all.e, o);
        }
    }
    const float ref = reference(all.zmax, p.c);

    const float logs = log2f(all.s);
    // log of the sum of exp(scale (z - zmax)): the reference's own rounding, zmax c - ref, comes off
    const float spread = kLn2 * (extreme ? logs : logs - fmaf(all.zmax, p.c, -ref));
    const bool none = all.zmax == -INFINITY && all.s == 0.0f;  // nothing but -inf
    const bool bad = isnan(all.s);
    const float lse = fmaf(all.zmax, p.scale, spread);
    // scale (z - zmax) rather than z c - ref: a product with c can pass fp32 where the answer does not
    auto logp_of = [&](float z) {
        if (none) return -INFINITY;
        const float d = z - all.zmax;
        return d == -INFINITY && z > -INFINITY ? fmaf(z, p.scale, -lse)  // further apart than fp32 reaches
                                               : fmaf(d, p.scale, -spread);
    };
    if (tid == 0) {
        if (p.lse) p.lse[i] = none ? -INFINITY : lse;
        if (p.entropy) p.entropy[i] = none ? 0.0f : kLn2 * (logs - all.e / all.s);
        if (p.logp) p.logp[i] = target >= 0 ? logp_of(z_target) : 0.0f;
    }
    if (TOP && tid < p.top) {
        const unsigned long long key = best[tid];
        const float z = unordered(static_cast<uint32_t>(key >> 32));
        p.top_ids[i * p.top + tid] = bad ? -1 : key_index(key);
        p.top_logp[i * p.top + tid] = bad ? NAN : logp_of(z);
    }
}

// ---------------------------------------------------------------- gradient
struct LogprobGradArgs {
    const void *logits, *targets;
    long long ld, ld_d;
    long long rows;
    int index_bytes, vocab, chunks;
    float scale;
    const float *lse, *entropy, *g_logp, *g_entropy;
    void *dlogits;
};

// One element: t = scale z - lse (= log p), q = scale z - (lse - H) (= log p +
// H, which cancel where p is largest: lse - H as a sum of two floats),
// d = -scale (g + h q) p, and + scale g at the target.
//
// A row far from zero (nothing left but masks of -1e10) has an lse whose rounding
// alone is a large number: p would be inf, and a gradient of zero NaN.  FAR rows
// hold log p to at most 0 (on every row it cost 8 us of 152 at 8192 x 32000).
struct GradRow {
    float scale, lse, lse_h, lse_h_lo, H, h, g;  // lse - H = lse_h + lse_h_lo
    template <bool FAR = false>
    __device__ __forceinline__ float at(float z) const
    {
        float t = max_nan(fmaf(z, scale, -lse), kFloor);  // p = 0 there, and its weight stays finite
        float q = fmaxf(fmaf(z, scale, -lse_h) - lse_h_lo, kFloor);
        if (FAR) {
            t = min_nan(t, 0.0f);
            q = fminf(q, H);
        }
        const float p = exp2_fast(t * kLog2e);
        return -scale * fmaf(h, q, g) * p;
    }
};

constexpr int kGradThreads = 256;

// TX threads take one chunk of a row, TX * kUnroll vectors; a CTA several rows
// where a row is short.
template <typename T, int TX>
__global__ void __launch_bounds__(kGradThreads) logprobs_grad_kernel(const LogprobGradArgs p)
{
    constexpr int E = kPerVec<T>;
    const int tid = threadIdx.x % TX;
    const long long group = blockIdx.x / p.chunks, i = group * (kGradThreads / TX) + threadIdx.x / TX;
    const int chunk = static_cast<int>(blockIdx.x - group * p.chunks);
    if (i >= p.rows) return;
    const T *z = static_cast<const T *>(p.logits) + i * p.ld;
    T *d = static_cast<T *>(p.dlogits) + i * p.ld_d;
    const int t = token_at(p.targets, p.index_bytes, i, p.vocab);
    const float lse = __ldg(p.lse + i);
    const bool none = lse == -INFINITY;  // a row of -inf: zero gradient
    const float g = t >= 0 && !none ? __ldg(p.g_logp + i) : 0.0f;
    const float h = p.g_entropy && !none ? __ldg(p.g_entropy + i) : 0.0f;
    const float H = p.g_entropy && !none ? __ldg(p.entropy + i) : 0.0f;
    // two-sum of lse and -H (Knuth): the rounding error of lse - H, exactly
    const float lh = lse - H, back = lh - lse, lo = (lse - (lh - back)) + (-H - back);
    const bool far = !none && !(fabsf(lse) < 1048576.0f);  // from 2^20 on lse is off by up to 1/16; NaN too
    const GradRow f{p.scale, none ? 0.0f : lse, none ? 0.0f : lh, none ? 0.0f : lo, H, h, g};
    auto put = [&](int j, float r) {
        if (j == t) r = fmaf(p.scale, g, r);
        d[j] = Elem<T>::put(r);
    };
    auto one = [&](int j) { put(j, f.at(Elem<T>::get(z[j]))); };

    const uint32_t za = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z)) & 15u;
    const uint32_t da = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(d)) & 15u;
    if (za != da || far) {  // element by element (two rows that never align together)
        const int n = TX * kUnroll * E, j0 = chunk * n, j1 = min(j0 + n, p.vocab);
        if (far) {
            for (int j = j0 + tid; j < j1; j += TX) put(j, f.at<true>(Elem<T>::get(z[j])));
        } else {
#pragma unroll 4
            for (int j = j0 + tid; j < j1; j += TX) one(j);
        }
        return;
    }
    const int head = min(za ? static_cast<int>((16u - za) / sizeof(T)) : 0, p.vocab);
    const int nv = (p.vocab - head) / E;
    if (chunk == 0) {
        const int rest = head + nv * E;
        if (tid < head) one(tid);
        else if (tid >= 8 && tid - 8 < p.vocab - rest) one(rest + tid - 8);
    }
    const uint4 *zv = reinterpret_cast<const uint4 *>(z + head);
    uint4 *dv = reinterpret_cast<uint4 *>(d + head);
    const int v0 = chunk * TX * kUnroll + tid;
    uint4 x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        if (v0 + u * TX < nv) x[u] = zv[v0 + u * TX];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int v = v0 + u * TX;
        if (v >= nv) break;
        float y[E];
        widen_vec<T>(x[u], y);
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = f.at(y[e]);
        const int at = t - head - v * E;
        if (t >= 0 && at >= 0 && at < E) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e == at) y[e] = fmaf(p.scale, g, y[e]);
        }
        dv[v] = narrow_vec<T>(y);
    }
}

// Up to this vocabulary a warp takes a row, if there are more rows than run at
// once with a CTA each (65536 x 1000: 39 us against 172, with 5 alternatives 82
// against 369).  Fewer rows get a CTA each, which ends the longer of them sooner
// (256 x 4096 with 5 alternatives: 5.1 us against 7.2; 256 x 1000: 4.6 against
// 4.3).
constexpr int kWarpVocab = 4096;

template <typename T, bool TOP>
cudaError_t launch_logprobs(const LogprobArgs &a, int sms, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    if (a.vocab <= kWarpVocab && a.rows > static_cast<long long>(kCtasPerSm) * sms) {
        cfg.gridDim = dim3(static_cast<unsigned>((a.rows + kThreads / 32 - 1) / (kThreads / 32)));
        return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, 32, TOP>, a);
    }
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows * a.cluster));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, kThreads, TOP>, a);
}

template <typename T>
cudaError_t launch_logprobs(const LogprobArgs &a, int sms, cudaStream_t s)
{
    return a.top ? launch_logprobs<T, true>(a, sms, s) : launch_logprobs<T, false>(a, sms, s);
}

template <typename T>
void launch_grad(const LogprobGradArgs &a, int tx, unsigned grid, cudaStream_t s)
{
    if (tx == 32) logprobs_grad_kernel<T, 32><<<grid, kGradThreads, 0, s>>>(a);
    else if (tx == 64) logprobs_grad_kernel<T, 64><<<grid, kGradThreads, 0, s>>>(a);
    else if (tx == 128) logprobs_grad_kernel<T, 128><<<grid, kGradThreads, 0, s>>>(a);
    else logprobs_grad_kernel<T, kGradThreads><<<grid, kGradThreads, 0, s>>>(a);
}

bool bad_common(const void *logits, long long ld, int index_bytes, long long rows, int vocab, int dtype, float scale)
{
    return rows < 0 || vocab < 1 || ld < vocab || (dtype != CDG_F16 && dtype != CDG_BF16 && dtype != CDG_F32) ||
           (index_bytes != 4 && index_bytes != 8) || !(scale > 0.0f) || !std::isfinite(scale) || (rows > 0 && !logits);
}

}  // namespace
}  // namespace cdg

extern "C" {

int cdg_token_logprobs(const void *logits, long long ld, const void *targets, int index_bytes, long long rows,
                       int vocab, int dtype, float scale, int top, float *logp, float *lse, float *entropy,
                       int *top_ids, float *top_logp, cdg_stream_t stream)
{
    using namespace cdg;
    if (bad_common(logits, ld, index_bytes, rows, vocab, dtype, scale) || top < 0 || top > kMaxTop || top > vocab)
        return CDG_ERR_INVALID_ARG;
    if (rows == 0) return CDG_OK;
    if (!targets != !logp || (top > 0) != (top_ids != nullptr) || (top > 0) != (top_logp != nullptr) ||
        (!logp && !lse && !entropy && !top))
        return CDG_ERR_INVALID_ARG;
    if (rows > (1ll << 31) / kMaxCluster - 1 || vocab > kMaxVocab) return CDG_ERR_UNSUPPORTED;
    const int es = dtype_bytes(dtype);
    if (!aligned_to(logits, es) || !aligned_to(targets, index_bytes) || !aligned_to(logp, 4) || !aligned_to(lse, 4) ||
        !aligned_to(entropy, 4) || !aligned_to(top_ids, 4) || !aligned_to(top_logp, 4))
        return CDG_ERR_ALIGNMENT;
    const size_t n = static_cast<size_t>(rows);
    const Extent in[2] = {extent(logits, matrix_bytes(rows, vocab, ld, es)), extent(targets, n * index_bytes)};
    const Extent out[5] = {extent(logp, n * 4), extent(lse, n * 4), extent(entropy, n * 4), extent(top_ids, n * top * 4),
                           extent(top_logp, n * top * 4)};
    for (int i = 0; i < 5; ++i) {
        for (const Extent &e : in)
            if (overlap(out[i], e)) return CDG_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return CDG_ERR_ALIAS;
    }
    const int sms = sm_count();
    if (sms < 1) return CDG_ERR_CUDA;
    LogprobArgs a{logits, targets, ld, rows, index_bytes, vocab, top, 1, scale,
                  static_cast<float>(static_cast<double>(scale) * 1.4426950408889634), logp, lse, entropy, top_logp,
                  top_ids};
    // CTAs a row: while there are fewer rows than SMs, split a row over a cluster
    while (a.cluster < kMaxCluster && rows * a.cluster * 2 <= 2ll * sms && vocab / (2 * a.cluster) >= 4096) a.cluster *= 2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == CDG_F32   ? launch_logprobs<float>(a, sms, s)
                          : dtype == CDG_F16 ? launch_logprobs<__half>(a, sms, s)
                                             : launch_logprobs<__nv_bfloat16>(a, sms, s);
    return e == cudaSuccess ? CDG_OK : CDG_ERR_CUDA;
}

int cdg_token_logprobs_grad(const void *logits, long long ld, const void *targets, int index_bytes, long long rows,
                            int vocab, int dtype, float scale, const float *lse, const float *entropy,
                            const float *g_logp, const float *g_entropy, void *dlogits, long long ld_d,
                            cdg_stream_t stream)
{
    using namespace cdg;
    if (bad_common(logits, ld, index_bytes, rows, vocab, dtype, scale) || ld_d < vocab) return CDG_ERR_INVALID_ARG;
    if (rows == 0) return CDG_OK;
    if (!targets || !lse || !g_logp || !dlogits || (g_entropy && !entropy)) return CDG_ERR_INVALID_ARG;
    const int es = dtype_bytes(dtype);
    int tx = 32;
    while (tx < kGradThreads && static_cast<long long>(tx) * kUnroll * (16 / es) < vocab) tx *= 2;
    const int per = tx * kUnroll * (16 / es), ty = kGradThreads / tx;
    const int chunks = (vocab - 1) / per + 1;
    const long long groups = (rows - 1) / ty + 1;
    if (rows > ((1ll << 31) - 1) / chunks || vocab > kMaxVocab) return CDG_ERR_UNSUPPORTED;
    if (!aligned_to(logits, es) || !aligned_to(targets, index_bytes) || !aligned_to(lse, 4) || !aligned_to(entropy, 4) ||
        !aligned_to(g_logp, 4) || !aligned_to(g_entropy, 4) || !aligned_to(dlogits, es))
        return CDG_ERR_ALIGNMENT;
    const size_t n = static_cast<size_t>(rows);
    const Extent out = extent(dlogits, matrix_bytes(rows, vocab, ld_d, es));
    const Extent in[5] = {extent(targets, n * index_bytes), extent(lse, n * 4), extent(entropy, n * 4),
                          extent(g_logp, n * 4), extent(g_entropy, n * 4)};
    for (const Extent &e : in)
        if (overlap(out, e)) return CDG_ERR_ALIAS;
    if (!(dlogits == logits && ld == ld_d) && overlap(out, extent(logits, matrix_bytes(rows, vocab, ld, es))))
        return CDG_ERR_ALIAS;
    const LogprobGradArgs a{logits, targets, ld, ld_d, rows, index_bytes, vocab, chunks, scale, lse, entropy, g_logp,
                            g_entropy, dlogits};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = static_cast<unsigned>(groups * chunks);
    if (dtype == CDG_F32) launch_grad<float>(a, tx, grid, s);
    else if (dtype == CDG_F16) launch_grad<__half>(a, tx, grid, s);
    else launch_grad<__nv_bfloat16>(a, tx, grid, s);
    return cudaGetLastError() == cudaSuccess ? CDG_OK : CDG_ERR_CUDA;
}

}  // extern "C"
