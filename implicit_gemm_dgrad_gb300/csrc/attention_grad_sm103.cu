// The attention's gradient for sm_103a.  With p = exp(s - lse) recomputed from
// the forward's lse, D_i = do_i . o_i, dp = do v^T and ds = p (dp - D):
//
//   dv = p^T do,   dk = scale ds^T q,   dq = scale ds k
//
// Three kernels: the rows' statistics (- lse log2 e and D), then dk and dv by
// CTAs of 128 keys, then dq by CTAs of 128 queries.  The second and the third
// both compute s and dp, so the gradient takes seven products of a pair of
// tiles rather than five; but each of its sums belongs to one CTA, stays in
// tensor memory from the first step to the last and is added in a fixed order
// (no atomics, no fp32 copy of dq in memory), and p and ds go back to tensor
// memory as the 16-bit A operand of the next product, never to shared memory.
// For dk and dv the scores are computed transposed (a thread a key, columns
// queries), so that P^T and dS^T lie as those products need them.
//
// p and ds are rounded to 16 bits as operands of the products that sum them; fp16's
// at a power of two times their value (DsScale).
//
// Each kernel's warps (640 threads): 0-15 compute (128 rows x 32 columns a
// warpgroup), 16 loads by TMA, 17 issues MMAs, 18 fetches the queries'
// statistics of a step (dk and dv), 19 items.  The two phases of a step, p and ds, each
// overlap two products of the tensor cores: dk and dv run
//   p(i) | dS^T(i-1) Q, dP^T(i)      then      ds(i) | P^T(i) dO, S^T(i+1)
//
// Measured (GB300, 8192 causal tokens, 16 heads of 128 over 4, bf16): 647 us, 1060
// TFLOP/s of the five products that the gradient needs, 1490 of the seven made, call after
// call, where the power limit lowers the SM clock (609 us for ten; dk and dv 3.0 thousand
// cycles a step for products of 2.05, dq 2.3 for 1.54); packed documents 474 us (454); fp16
// 660 for ten, 2 % more than bf16 at the same clock.  A step's phases wait for one another: scores complete, p of all
// sixteen warps 1.4 thousand cycles, two products 1.3.  Eight warps of 64 columns
// took 725 us where sixteen of 32 took 663.
#include <algorithm>

#include "attention_device.cuh"

namespace cdg {
namespace {

constexpr int kWarpLoad = 16, kWarpMma = 17, kWarpStats = 18;
constexpr int kSlots = 2;  // steps of each streamed operand in shared memory

// (- lse log2 e, D) of every row and head; a row that saw nothing (lse = -inf)
// gets -inf there, so that every p of it is 0.  16 lanes take kStatRows tokens of
// a head, all of whose loads are in flight together.
//
// fp16: the largest sizes beside them (CatParams::sizes), and those of v's rows by CTAs of their
// own, from which dS's power of two comes (DsScale).  Rows that are not finite, or in
// no sequence, have none.
constexpr int kStatRows = 4;
constexpr int kStatThreads = 256, kStatGroups = kStatThreads / 16;
constexpr int kSizeCtas = 304;  // fp16, of each side: two on each of 152 SMs

__device__ __forceinline__ uint32_t finite_size(float v) { return isfinite(v) ? __float_as_uint(fabsf(v)) : 0u; }
__device__ __forceinline__ uint4 larger(uint4 a, uint4 b) { return make_uint4(max(a.x, b.x), max(a.y, b.y), max(a.z, b.z), 0u); }
// (sizes are not negative: their bits compare as they do)
__device__ __forceinline__ uint4 warp_largest(uint4 v)
{
    return make_uint4(__reduce_max_sync(0xFFFFFFFFu, v.x), __reduce_max_sync(0xFFFFFFFFu, v.y), __reduce_max_sync(0xFFFFFFFFu, v.z), 0u);
}

// The sum over 16 lanes of 8 products each.
__device__ __forceinline__ float dot16(const float (&x)[8], const float (&y)[8])
{
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(x[e], y[e], sum);
#pragma unroll
    for (int d = 8; d; d /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    return sum;
}

template <bool BF16>
__global__ void __launch_bounds__(kStatThreads) attention_stats_kernel(const __grid_constant__ CatParams p)
{
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    grid_dep_launch_dependents();
    grid_dep_wait();
    const bool of_v = !BF16 && static_cast<int>(blockIdx.x) >= p.stat_ctas;
    const int cta = of_v ? blockIdx.x - p.stat_ctas : blockIdx.x, ctas = of_v ? p.size_ctas : p.stat_ctas;
    const int tokens = of_v ? p.k_tokens : p.q_tokens, heads = of_v ? p.kv_heads : p.heads, lane = threadIdx.x & 15;
    int lo = 0, hi = 0;  // the rows that sequences hold
    if (!BF16) {
        const void *offsets = of_v ? p.k_offsets : p.q_offsets;
        lo = offset_at(offsets, p.index_bytes, 0, tokens);
        hi = offset_at(offsets, p.index_bytes, p.sequences, tokens);
    }
    uint4 top = make_uint4(0, 0, 0, 0);
    const long long groups = (tokens + kStatRows - 1ll) / kStatRows * heads;
    // (a warp's two groups go round together)
    for (long long g0 = static_cast<long long>(cta) * kStatGroups + threadIdx.x / 32 * 2; g0 < groups; g0 += static_cast<long long>(ctas) * kStatGroups) {
        const long long g = g0 + ((threadIdx.x >> 4) & 1), block = g / heads, token = block * kStatRows;
        const int head = static_cast<int>(g - block * heads);
        const long long col = static_cast<long long>(head) * p.dim + 8 * lane;
        uint4 a[kStatRows], b[kStatRows];
        float x[8], y[8];
        if (of_v) {
#pragma unroll
            for (int r = 0; r < kStatRows; ++r)
                a[r] = token + r >= lo && token + r < hi && 8 * lane < p.dim
                           ? ld_written(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.v_in) + (token + r) * p.ld_v + col))
                           : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < kStatRows; ++r) {
                widen_vec<T>(a[r], x);
                top.y = max(top.y, finite_size(dot16(x, x)));
            }
            continue;
        }
#pragma unroll
        for (int r = 0; r < kStatRows; ++r) {
            const bool in = token + r < tokens && 8 * lane < p.dim;
            a[r] = in ? ld_written(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.d_o) + (token + r) * p.ld_do + col)) : make_uint4(0, 0, 0, 0);
            b[r] = in ? ld_written(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.o_in) + (token + r) * p.ld_oi + col)) : make_uint4(0, 0, 0, 0);
        }
        float mine = 0.0f, square = 0.0f;  // lane r: row r's sums
#pragma unroll
        for (int r = 0; r < kStatRows; ++r) {
            widen_vec<T>(a[r], x);
            widen_vec<T>(b[r], y);
            const float sum = dot16(x, y);
            if (lane == r) mine = sum;
            if (!BF16) {
                const float sq = dot16(x, x);
                if (lane == r) square = sq;
            }
        }
        if (lane < kStatRows && token + lane < tokens) {
            const long long at = static_cast<long long>(head) * p.q_tokens + token + lane;
            const float lse = ld_written(p.lse_in + at);
            p.stats[at] = make_float2(lse == -INFINITY ? -INFINITY : -lse * 1.4426950408889634f, mine);
            if (!BF16 && token + lane >= lo && token + lane < hi) top = larger(top, make_uint4(finite_size(square), 0u, finite_size(mine), 0u));
        }
    }
    if constexpr (!BF16) {
        __shared__ uint4 red[kStatThreads / 32];
        top = warp_largest(top);
        if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = top;
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int w = 1; w < kStatThreads / 32; ++w) top = larger(top, red[w]);
            p.sizes[blockIdx.x] = top;
        }
    }
}

// fp16 holds p of 1 / n of many keys, and ds, which is smaller still, below its smallest normal
// number (2^-14), where its steps are 2^-24.  Both are therefore rounded at a power of
// two times their value, exactly undone where the sums are stored: p at 2^11 (dk and dv's
// alone: dq's stays fp32), ds at the 2^k >= 1 that brings max |do| max |v| + max |do o|, which
// |dp - D| is never above, to between 2^10 and 2^11.  With the forward's lse p is at most 1; the
// 2^5 that is left is for an lse that is not.  bf16 has fp32's range, and scales nothing.
constexpr int kPScale = 11;
template <bool BF16>
struct DsScale {
    float up = 1.0f, down = 1.0f;  // 2^k, 2^-k
    // (a converged warp, in fp16; each warp that needs it reads the sizes for itself, beneath the first loads)
    __device__ __forceinline__ explicit DsScale(const CatParams &p)
    {
        if constexpr (!BF16) {
            uint4 v = make_uint4(0, 0, 0, 0);
            for (int i = threadIdx.x & 31; i < p.stat_ctas + p.size_ctas; i += 32) v = larger(v, ld_written(p.sizes + i));
            v = warp_largest(v);
            const float bound = sqrtf(__uint_as_float(v.x)) * sqrtf(__uint_as_float(v.y)) + __uint_as_float(v.z);
            const int k = bound > 0.0f ? max(0, kPScale - 1 - ilogbf(bound)) : 0;
            up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);  // (fp16's smallest numbers: k is below 64)
            down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
        }
    }
};

constexpr int kWarpItems = 19;

struct GradBars {
    uint32_t own_full0, own_empty0;  // [2]: the item's own tiles (K and V, or Q and dO)
    uint32_t full_a0, empty_a0;      // [kSlots]: the streamed operand of the scores (Q, or K)
    uint32_t full_b0, empty_b0;      // [kSlots]: the streamed operand of dP (dO, or V)
    uint32_t st_full0, st_empty0;    // [kSlots]: statistics
    uint32_t s_full, s_read, dp_full, ds_ready, out_full, out_empty, drain;
};

struct GradSmem {
    uint32_t own, ring_a, ring_b, stats, tile_bytes;
    GradBars B;
    ItemBars I;
    uint32_t *tmem_slot;
    volatile uint32_t *abort_flag, *slot_parity;  // parity of each slot's last load: a, b, then the own tiles'
};
constexpr int kGradTail = kItemBytes + 512;

template <int SLICES>
__device__ __forceinline__ GradSmem grad_layout(uint8_t *smem_raw, int item_warps)
{
    GradSmem S;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    S.tile_bytes = kSliceBytes * SLICES;
    S.own = base;
    S.ring_a = base + 2 * S.tile_bytes;
    S.ring_b = S.ring_a + kSlots * S.tile_bytes;
    S.stats = S.ring_b + kSlots * S.tile_bytes;  // kSlots x 128 shifts, then 128 sums
    const uint32_t items = S.stats + kSlots * CAT_TILE * 8;
    S.I = init_items(smem_raw + (items - raw), items, item_warps);
    uint32_t at = items + kItemBytes;
    auto take = [&](int n) {
        const uint32_t was = at;
        at += 8 * n;
        return was;
    };
    S.B.own_full0 = take(2);
    S.B.own_empty0 = take(2);
    S.B.full_a0 = take(kSlots);
    S.B.empty_a0 = take(kSlots);
    S.B.full_b0 = take(kSlots);
    S.B.empty_b0 = take(kSlots);
    S.B.st_full0 = take(kSlots);
    S.B.st_empty0 = take(kSlots);
    S.B.s_full = take(1);
    S.B.s_read = take(1);
    S.B.dp_full = take(1);
    S.B.ds_ready = take(1);
    S.B.out_full = take(1);
    S.B.out_empty = take(1);
    S.B.drain = take(1);
    S.tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + (at - raw));
    S.abort_flag = S.tmem_slot + 1;
    S.slot_parity = S.tmem_slot + 2;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(S.B.own_full0 + 8u * s, 1);
            mbar_init(S.B.own_empty0 + 8u * s, 1);
        }
        for (int s = 0; s < kSlots; ++s) {
            for (uint32_t b : {S.B.full_a0, S.B.empty_a0, S.B.full_b0, S.B.empty_b0}) mbar_init(b + 8u * s, 1);
            mbar_init(S.B.st_full0 + 8u * s, 32);
            mbar_init(S.B.st_empty0 + 8u * s, 16);
        }
        for (uint32_t b : {S.B.s_full, S.B.dp_full, S.B.out_full, S.B.drain}) mbar_init(b, 1);
        for (uint32_t b : {S.B.s_read, S.B.ds_ready, S.B.out_empty}) mbar_init(b, 16);
        for (int s = 0; s < 2 * kSlots + 2; ++s) S.slot_parity[s] = 0u;
        *S.abort_flag = 0u;
        fence_mbar_init();
    }
    return S;
}

// After all roles: on an abort the latest load of every used slot lands before the CTA exits.
__device__ __forceinline__ void grad_end(const CatParams &p, const GradSmem &S, uint32_t tmem)
{
    __syncthreads();
    if (*S.abort_flag && threadIdx.x == 0) {
        volatile uint32_t no_abort = 0;
        const Ctl drain_ctl{&no_abort, p.status};
        for (int s = 0; s < 2 * kSlots + 2; ++s) {
            const uint32_t v = S.slot_parity[s];
            const uint32_t bar = s >= 2 * kSlots ? S.B.own_full0 + 8u * (s - 2 * kSlots)
                                 : s < kSlots    ? S.B.full_a0 + 8u * s
                                                 : S.B.full_b0 + 8u * (s - kSlots);
            if (v & 2u) wait_bar(bar, v & 1u, drain_ctl);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x / 32 == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

__device__ __forceinline__ void drain_mmas(const CatParams &p, const GradSmem &S, uint32_t leader)
{
    mma_commit(leader, S.B.drain);
    volatile uint32_t no_abort = 0;
    wait_bar(S.B.drain, 0, Ctl{&no_abort, p.status});
}

// The loads of one item: its own two tiles, and pairs of streamed tiles.
// where(n, head, token): of the n-th pair.  items, steps: what came before.
template <typename At>
__device__ __forceinline__ bool run_grad_loads(const CatParams &p, const GradSmem &S, Ctl ctl, bool leader, int count,
                                               const CUtensorMap &own_a, const CUtensorMap &own_b, int own_head, int own_token,
                                               const CUtensorMap &map_a, const CUtensorMap &map_b, uint32_t &items, uint32_t &steps,
                                               At where)
{
    for (int n = 0; n < count; ++n, ++steps) {
        const uint32_t slot = steps % kSlots, parity = (steps / kSlots) & 1u;
        int head, token;
        where(n, head, token);
        for (int b = 0; b < 2; ++b) {
            if (n == 0) {  // (the scores' operands first)
                if (!wait_bar(S.B.own_empty0 + 8u * b, (items & 1u) ^ 1u, ctl)) return false;
                if (leader) {
                    S.slot_parity[2 * kSlots + b] = (items & 1u) | 2u;
                    mbar_arrive_expect_tx(S.B.own_full0 + 8u * b, S.tile_bytes);
                    load_tile(S.own + b * S.tile_bytes, b ? own_b : own_a, S.B.own_full0 + 8u * b, p.slices, own_head, own_token);
                }
                __syncwarp();
            }
            if (!wait_bar((b ? S.B.empty_b0 : S.B.empty_a0) + 8u * slot, parity ^ 1u, ctl)) return false;
            if (leader) {
                const uint32_t bar = (b ? S.B.full_b0 : S.B.full_a0) + 8u * slot;
                S.slot_parity[b * kSlots + slot] = parity | 2u;
                mbar_arrive_expect_tx(bar, S.tile_bytes);
                load_tile((b ? S.ring_b : S.ring_a) + slot * S.tile_bytes, b ? map_b : map_a, bar, p.slices, head, token);
            }
            __syncwarp();
        }
    }
    if (count > 0) ++items;
    return true;
}

// Columns of tensor memory: scores, dP, and the sums (dV and dK, or dQ).
constexpr uint32_t kS = 0, kDP = 128, kSum = 256;

// ------------------------------------------------------------------ dk, dv

// An item of dk and dv: 128 keys, and its part of the steps of their group's query
// heads over the query tiles that see some of them.
template <bool SPLIT>
struct KeyTile {
    int j0;              // first key of the tile, in its sequence
    int lo, count;       // first query tile and their number, for each head
    int kv_head, part;
    int begin, end;      // the part's steps: of head n / count, query tile lo + n % count
    __device__ __forceinline__ KeyTile(const CatParams &p, const Item &item)
    {
        const Place &at = item.at;
        kv_head = SPLIT ? item.head / p.k_splits : item.head;
        part = SPLIT ? item.head - kv_head * p.k_splits : 0;
        // (a sequence's first keys, which under a causal mask most queries see, come first)
        j0 = at.tile * CAT_TILE;
        const int off = at.kl - at.ql, j1 = min(j0 + CAT_TILE, at.kl);
        const int first = p.causal ? max(0, j0 - off) : 0, last = p.window ? min(at.ql, j1 - 1 - off + p.window) : at.ql;
        lo = first / CAT_TILE;
        count = last > first ? (last + CAT_TILE - 1) / CAT_TILE - lo : 0;
        begin = 0;
        end = count * p.group;
        if (SPLIT) take_part(begin, end, part, p.k_splits);
    }
    __device__ __forceinline__ int steps() const { return end - begin; }
    __device__ __forceinline__ void where(const CatParams &p, int n, int &head, int &tile) const
    {
        if (SPLIT) n += begin;
        const int h = n / count;
        head = kv_head * p.group + h;
        tile = lo + n - h * count;
    }
};

// Four numbers of shared memory that the whole warp reads.
__device__ __forceinline__ void ld_shared_4(uint32_t at, float (&v)[4])
{
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(at));
}

// Zeroes the columns past [lo, hi).
__device__ __forceinline__ void hide(float (&s)[32], int lo, int hi)
{
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (e < lo || e >= hi) s[e] = 0.0f;
}

template <bool BF16>
__device__ __forceinline__ void put_rounded(uint32_t taddr, const float (&s)[32])
{
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = round2<BF16>(s[2 * e], s[2 * e + 1]);
    tmem_st_16(taddr, w);
    tmem_st_wait();
}

template <bool BF16, bool SPLIT>
__device__ __forceinline__ bool compute_dkv(const CatParams &p, const GradSmem &S, Ctl ctl, uint32_t tmem, const Place &at,
                                            const KeyTile<SPLIT> &kt, const DsScale<BF16> &scale, uint32_t &done, uint32_t &items)
{
    const int warp = threadIdx.x / 32, part = warp / 4, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t s_col = tmem + lanes + kS + 32u * part, dp_col = tmem + lanes + kDP + 32u * part;
    // (p is at 2^kPScale in fp16)
    const float of_p = BF16 ? 1.0f : scale.up * (1.0f / (1 << kPScale)), p_down = BF16 ? 1.0f : 1.0f / (1 << kPScale);
    const f32x2 c2 = pack2(p.scale_log2, p.scale_log2), of_p2 = pack2(of_p, of_p);
    const int off = at.kl - at.ql, j = kt.j0 + row;
    const int steps = kt.steps();
    int tile = kt.count > 0 ? kt.lo + kt.begin % kt.count : 0;
    for (int n = 0; n < steps; ++n, ++done) {
        const uint32_t slot = done % kSlots;
        const uint32_t stats = S.stats + slot * 2 * CAT_TILE * 4 + part * 32 * 4;
        const int i0 = tile * CAT_TILE;
        if (++tile == kt.lo + kt.count) tile = kt.lo;
        // columns [lo, hi) of this part see the key
        const bool whole = (!p.causal || kt.j0 + CAT_TILE - 1 <= i0 + off) && (!p.window || kt.j0 > i0 + CAT_TILE - 1 + off - p.window);
        const int lo = p.causal ? j - off - i0 - 32 * part : 0, hi = p.window ? j - off - i0 - 32 * part + p.window : 32;
        if (!wait_bar(S.B.st_full0 + 8u * slot, (done / kSlots) & 1u, ctl) || !wait_bar(S.B.s_full, done & 1u, ctl)) return false;
        tc_fence_after();
        float s[32];
        tmem_ld_32(s_col, s);
        tmem_wait(s);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            float shift[4];
            ld_shared_4(stats + e * 4u, shift);
#pragma unroll
            for (int f = 0; f < 4; f += 2) {
                float a, b;
                unpack2(fma2(pack2(s[e + f], s[e + f + 1]), c2, pack2(shift[f], shift[f + 1])), a, b);
                s[e + f] = exp2_approx(a);
                s[e + f + 1] = exp2_approx(b);
            }
        }
        if (!whole) hide(s, lo, hi);
        put_rounded<BF16>(s_col, s);
        warp_arrive(S.B.s_read);
        if (!wait_bar(S.B.dp_full, done & 1u, ctl)) return false;
        tc_fence_after();
        float dp[32];
        tmem_ld_32(dp_col, dp);
        tmem_wait(dp);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            float d[4];
            ld_shared_4(stats + (CAT_TILE + e) * 4u, d);
#pragma unroll
            for (int f = 0; f < 4; f += 2)
                unpack2(mul2(pack2(s[e + f], s[e + f + 1]), fma2(pack2(dp[e + f], dp[e + f + 1]), of_p2, pack2(d[f], d[f + 1]))),
                        dp[e + f], dp[e + f + 1]);
        }
        if (!whole) hide(dp, lo, hi);  // (dP of an unseen pair may be anything)
        put_rounded<BF16>(dp_col, dp);
        warp_arrive(S.B.ds_ready);
        if ((threadIdx.x & 31) == 0) mbar_arrive(S.B.st_empty0 + 8u * slot);
    }
    // the first two warpgroups store dv, the others dk, half of the columns each
    const long long token = at.k0 + j, first = token - (threadIdx.x & 31);
    const bool is_dk = part >= 2;
    const int c0 = 32 * p.slices * (part & 1), c1 = min(p.dim, c0 + 32 * p.slices), rows = at.kl - (j & ~31);
    const long long ld = SPLIT ? static_cast<long long>(p.kv_heads) * p.dim : is_dk ? p.ld_dk : p.ld_dv;
    uint16_t *out = static_cast<uint16_t *>(is_dk ? p.dk : p.dv) + first * ld + static_cast<long long>(kt.kv_head) * p.dim;
    float *sum = p.k_partial + ((2ll * kt.part + is_dk) * p.k_tokens + first) * ld + static_cast<long long>(kt.kv_head) * p.dim;
    if (steps > 0) {
        if (!wait_bar(S.B.out_full, items & 1u, ctl)) return false;
        ++items;
        tc_fence_after();
        const uint32_t taddr = tmem + lanes + kSum + 64u * p.slices * is_dk;
        const float down = is_dk ? scale.down : p_down;
        if (SPLIT) store_rows_f32(taddr, c0, c1, down, sum, ld, rows);
        else store_rows<BF16>(taddr, c0, c1, is_dk ? p.scale * down : down, out, ld, rows);
        warp_arrive(S.B.out_empty);
    } else if (j < at.kl) {
        const int lane = threadIdx.x & 31;
        if (SPLIT)
            for (int c = c0; c < c1; c += 4) *reinterpret_cast<float4 *>(sum + lane * ld + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        else
            zero_row(out + lane * ld, c0, c1);
    }
    return true;
}

template <bool BF16, int SLICES, bool SPLIT>
__global__ void __launch_bounds__(CAT_GRAD_THREADS, 1) attention_dkv_kernel(const __grid_constant__ CatParams p)
{
    constexpr uint32_t tile_bytes = kSliceBytes * SLICES;
    extern __shared__ uint8_t smem_raw[];
    const GradSmem S = grad_layout<SLICES>(smem_raw, 19);
    const int warp = threadIdx.x / 32;
    grid_dep_wait();
    // dq needs the statistics alone: its CTAs may start as soon as all of these have
    grid_dep_launch_dependents();
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(S.tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *S.tmem_slot;
    const Ctl ctl{S.abort_flag, p.status};
    Item item;
    uint32_t done = 0, items = 0;  // steps, and items that had some
    if (warp == kWarpItems) {
        run_items(p, S.I, ctl, CAT_TILE, true, p.kv_heads * p.k_splits);
    } else if (warp == kWarpLoad) {
        const bool leader = elect_one_sync();
        for (int n = 0; next_item(S.I, ctl, n, item); ++n) {
            const KeyTile<SPLIT> kt(p, item);
            if (!run_grad_loads(p, S, ctl, leader, kt.steps(), p.tmK, p.tmV, kt.kv_head, item.at.k0 + kt.j0, p.tmQ, p.tmDO, items, done,
                                [&](int k, int &head, int &token) {
                                    int tile;
                                    kt.where(p, k, head, tile);
                                    token = item.at.q0 + tile * CAT_TILE;
                                }))
                break;
            if (leader) mbar_arrive(S.I.go);
            __syncwarp();
        }
    } else if (warp == kWarpStats) {
        const int lane = threadIdx.x & 31;
        // as the computing warps add them: fp16's p and ds are scaled
        const float p_up = BF16 ? 0.0f : kPScale, minus = BF16 ? -1.0f : DsScale<BF16>(p).up * (-1.0f / (1 << kPScale));
        bool ok = true;
        for (int n = 0; ok && next_item(S.I, ctl, n, item); ++n) {
            const KeyTile<SPLIT> kt(p, item);
            for (int k = 0; k < kt.steps(); ++k, ++done) {
                const uint32_t slot = done % kSlots;
                int head, tile;
                kt.where(p, k, head, tile);
                ok = wait_bar(S.B.st_empty0 + 8u * slot, ((done / kSlots) & 1u) ^ 1u, ctl);
                if (!ok) break;
                const float2 *src = p.stats + static_cast<long long>(head) * p.q_tokens + item.at.q0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = 32 * e + lane, i = tile * CAT_TILE + c;
                    const float2 v = i < item.at.ql ? ld_written(src + i) : make_float2(-INFINITY, 0.0f);
                    st_shared_f32(S.stats + (slot * 2 * CAT_TILE + c) * 4u, BF16 ? v.x : v.x + p_up);
                    st_shared_f32(S.stats + ((slot * 2 + 1) * CAT_TILE + c) * 4u, v.y * minus);
                }
                mbar_arrive(S.B.st_full0 + 8u * slot);
            }
        }
    } else if (warp == kWarpMma) {
        const uint32_t leader = elect_one_sync();
        const uint32_t tm = uniform(tmem), s = tm + kS, dp = tm + kDP, dv = tm + kSum, dk = dv + 64u * SLICES;
        bool ok = true;
        for (int n = 0; ok && next_item(S.I, ctl, n, item); ++n) {
            const KeyTile<SPLIT> kt(p, item);
            const int total = uniform(kt.steps()), count = uniform(kt.count), begin = uniform(kt.begin);
            const int rest = uniform(item.at.ql - kt.lo * CAT_TILE);
            if (total == 0) continue;
            // waits for the k-th streamed tile; rows behind the sequence's end become zeros
            auto filled = [&](uint32_t full0, uint32_t ring, int k, uint32_t step) {
                if (!wait_bar(full0 + 8u * (step % kSlots), (step / kSlots) & 1u, ctl)) return false;
                tc_fence_after();
                const int valid = rest - (begin + k) % count * CAT_TILE;
                if (valid < CAT_TILE) zero_rows(ring + (step % kSlots) * tile_bytes, SLICES, valid);
                return true;
            };
            auto scores = [&](int k) {
                const uint32_t step = done + k;
                if (!filled(S.B.full_a0, S.ring_a, k, step)) return false;
                issue_qk<SLICES>(leader, s, S.own, S.ring_a + (step % kSlots) * tile_bytes, p.idesc_qk, p.ksteps);
                mma_commit(leader, S.B.s_full);
                if (k + 1 == total) mma_commit(leader, S.B.own_empty0);
                return true;
            };
            auto dps = [&](int k) {
                const uint32_t step = done + k;
                if (!filled(S.B.full_b0, S.ring_b, k, step)) return false;
                issue_qk<SLICES>(leader, dp, S.own + tile_bytes, S.ring_b + (step % kSlots) * tile_bytes, p.idesc_qk, p.ksteps);
                mma_commit(leader, S.B.dp_full);
                if (k + 1 == total) mma_commit(leader, S.B.own_empty0 + 8u);
                return true;
            };
            ok = wait_bar(S.B.own_full0, items & 1u, ctl) && scores(0) && wait_bar(S.B.own_full0 + 8u, items & 1u, ctl) && dps(0);
            for (int k = 0; ok && k < total; ++k) {
                const bool next = k + 1 < total;
                const uint32_t step = done + k, slot = step % kSlots;
                ok = wait_bar(S.B.s_read, step & 1u, ctl);
                // the item before has left the sums
                if (ok && k == 0) ok = wait_bar(S.B.out_empty, (items & 1u) ^ 1u, ctl);
                if (!ok) break;
                tc_fence_after();
                issue_pv<32>(leader, dv, s, S.ring_b + slot * tile_bytes, p.idesc_pv, k != 0);
                mma_commit(leader, S.B.empty_b0 + 8u * slot);
                ok = (!next || scores(k + 1)) && wait_bar(S.B.ds_ready, step & 1u, ctl);
                if (!ok) break;
                tc_fence_after();
                issue_pv<32>(leader, dk, dp, S.ring_a + slot * tile_bytes, p.idesc_pv, k != 0);
                mma_commit(leader, S.B.empty_a0 + 8u * slot);
                if (!next) mma_commit(leader, S.B.out_full);
                else ok = dps(k + 1);
            }
            done += total;
            ++items;
        }
        drain_mmas(p, S, leader);
    } else if (warp < 16) {
        const DsScale<BF16> scale(p);
        for (int n = 0; next_item(S.I, ctl, n, item); ++n)
            if (!compute_dkv<BF16, SPLIT>(p, S, ctl, tmem, item.at, KeyTile<SPLIT>(p, item), scale, done, items)) break;
    }
    grad_end(p, S, tmem);
}

// ------------------------------------------------------------------ dq

// An item of dq: 128 queries from i0 of a head, its part [lo, hi) of the steps of keys.
template <bool SPLIT>
struct QueryTile {
    int i0, lo, hi, head, part;
    __device__ __forceinline__ QueryTile(const CatParams &p, const Item &item)
    {
        const Place &at = item.at;
        head = SPLIT ? item.head / p.q_splits : item.head;
        part = SPLIT ? item.head - head * p.q_splits : 0;
        // a sequence's last queries first: under a causal mask they see most keys
        i0 = ((at.ql + CAT_TILE - 1) / CAT_TILE - 1 - at.tile) * CAT_TILE;
        key_steps(p, at, i0, min(i0 + CAT_TILE, at.ql), lo, hi);
        if (SPLIT) take_part(lo, hi, part, p.q_splits);
    }
};

template <bool BF16, bool SPLIT>
__device__ __forceinline__ bool compute_dq(const CatParams &p, const GradSmem &S, Ctl ctl, uint32_t tmem, const Place &at,
                                           const QueryTile<SPLIT> &qt, const DsScale<BF16> &scale, uint32_t &done, uint32_t &items)
{
    const int i0 = qt.i0, head = qt.head, lo = qt.lo, hi = qt.hi;
    const int warp = threadIdx.x / 32, part = warp / 4, row = threadIdx.x & 127, i = i0 + row;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t s_col = tmem + lanes + kS + 32u * part, dp_col = tmem + lanes + kDP + 32u * part;
    const f32x2 c2 = pack2(p.scale_log2, p.scale_log2);
    const int r_first = i0 + at.kl - at.ql, r = r_first + row;
    const long long token = at.q0 + i;
    const bool valid = i < at.ql;
    const float2 st = valid ? ld_written(p.stats + static_cast<long long>(head) * p.q_tokens + token) : make_float2(-INFINITY, 0.0f);
    const float d = -st.y * scale.up;
    const f32x2 shift = pack2(st.x, st.x), minus_d = pack2(d, d), up2 = pack2(scale.up, scale.up);
    for (int j = lo; j < hi; ++j, ++done) {
        const int k0 = j * CAT_TILE;
        const bool whole = k0 + CAT_TILE <= at.kl && (!p.causal || k0 + CAT_TILE - 1 <= r_first) &&
                           (!p.window || k0 > r_first + CAT_TILE - 1 - p.window);
        if (!wait_bar(S.B.s_full, done & 1u, ctl)) return false;
        tc_fence_after();
        float s[32];
        tmem_ld_32(s_col, s);
        tmem_wait(s);
        warp_arrive(S.B.s_read);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            float a, b;
            unpack2(fma2(pack2(s[e], s[e + 1]), c2, shift), a, b);
            s[e] = exp2_approx(a);
            s[e + 1] = exp2_approx(b);
        }
        if (!wait_bar(S.B.dp_full, done & 1u, ctl)) return false;
        tc_fence_after();
        float dp[32];
        tmem_ld_32(dp_col, dp);
        tmem_wait(dp);
#pragma unroll
        for (int e = 0; e < 32; e += 2)
            unpack2(mul2(pack2(s[e], s[e + 1]), fma2(pack2(dp[e], dp[e + 1]), up2, minus_d)), dp[e], dp[e + 1]);
        if (!whole)  // (scores and dP of an unseen pair may be anything)
            hide(dp, p.window ? r - p.window + 1 - k0 - 32 * part : 0, min(at.kl, p.causal ? r + 1 : at.kl) - k0 - 32 * part);
        put_rounded<BF16>(dp_col, dp);
        warp_arrive(S.B.ds_ready);
    }
    uint16_t *out = static_cast<uint16_t *>(p.dq) + (token - (threadIdx.x & 31)) * p.ld_dq + static_cast<long long>(head) * p.dim;
    const long long width = static_cast<long long>(p.heads) * p.dim;
    float *sum = p.q_partial + (static_cast<long long>(qt.part) * p.q_tokens + token - (threadIdx.x & 31)) * width + static_cast<long long>(head) * p.dim;
    const int c0 = 32 * part, c1 = min(p.dim, c0 + 32);
    if (hi > lo) {
        if (!wait_bar(S.B.out_full, items & 1u, ctl)) return false;
        ++items;
        tc_fence_after();
        const int rows = at.ql - (i & ~31);
        if (SPLIT) store_rows_f32(tmem + lanes + kSum, c0, c1, scale.down, sum, width, rows);
        else store_rows<BF16>(tmem + lanes + kSum, c0, c1, p.scale * scale.down, out, p.ld_dq, rows);
        warp_arrive(S.B.out_empty);
    } else if (valid) {
        const int lane = threadIdx.x & 31;
        if (SPLIT)
            for (int c = c0; c < c1; c += 4) *reinterpret_cast<float4 *>(sum + lane * width + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        else
            zero_row(out + lane * p.ld_dq, c0, c1);
    }
    return true;
}

template <bool BF16, int SLICES, bool SPLIT>
__global__ void __launch_bounds__(CAT_GRAD_THREADS, 1) attention_dq_kernel(const __grid_constant__ CatParams p)
{
    constexpr uint32_t tile_bytes = kSliceBytes * SLICES;
    extern __shared__ uint8_t smem_raw[];
    const GradSmem S = grad_layout<SLICES>(smem_raw, 18);
    const int warp = threadIdx.x / 32;
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(S.tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *S.tmem_slot;
    const Ctl ctl{S.abort_flag, p.status};
    Item item;
    uint32_t done = 0, items = 0;  // steps, and items that had some
    if (warp == kWarpItems) {
        run_items(p, S.I, ctl, CAT_TILE, false, p.heads * p.q_splits);
    } else if (warp == kWarpLoad) {
        const bool leader = elect_one_sync();
        for (int n = 0; next_item(S.I, ctl, n, item); ++n) {
            const QueryTile<SPLIT> qt(p, item);
            if (!run_grad_loads(p, S, ctl, leader, qt.hi - qt.lo, p.tmQ, p.tmDO, qt.head, item.at.q0 + qt.i0, p.tmK, p.tmV, items, done,
                                [&](int k, int &head, int &token) {
                                    head = qt.head / p.group;
                                    token = item.at.k0 + (qt.lo + k) * CAT_TILE;
                                }))
                break;
            if (leader) mbar_arrive(S.I.go);
            __syncwarp();
        }
    } else if (warp == kWarpMma) {
        const uint32_t leader = elect_one_sync();
        const uint32_t tm = uniform(tmem), s = tm + kS, dp = tm + kDP, dq = tm + kSum;
        bool ok = true;
        for (int n = 0; ok && next_item(S.I, ctl, n, item); ++n) {
            const QueryTile<SPLIT> qt(p, item);
            const int total = uniform(qt.hi - qt.lo), rest = uniform(item.at.kl - qt.lo * CAT_TILE);
            if (total <= 0) continue;
            auto scores = [&](int k) {
                const uint32_t step = done + k, slot = step % kSlots;
                if (!wait_bar(S.B.full_a0 + 8u * slot, (step / kSlots) & 1u, ctl)) return false;
                tc_fence_after();
                // keys behind the sequence's end become zeros: dS K sums over them
                if (rest - k * CAT_TILE < CAT_TILE) zero_rows(S.ring_a + slot * tile_bytes, SLICES, rest - k * CAT_TILE);
                issue_qk<SLICES>(leader, s, S.own, S.ring_a + slot * tile_bytes, p.idesc_qk, p.ksteps);
                mma_commit(leader, S.B.s_full);
                if (k + 1 == total) mma_commit(leader, S.B.own_empty0);
                return true;
            };
            auto dps = [&](int k) {
                const uint32_t step = done + k, slot = step % kSlots;
                if (!wait_bar(S.B.full_b0 + 8u * slot, (step / kSlots) & 1u, ctl)) return false;
                tc_fence_after();
                issue_qk<SLICES>(leader, dp, S.own + tile_bytes, S.ring_b + slot * tile_bytes, p.idesc_qk, p.ksteps);
                mma_commit(leader, S.B.dp_full);
                mma_commit(leader, S.B.empty_b0 + 8u * slot);
                if (k + 1 == total) mma_commit(leader, S.B.own_empty0 + 8u);
                return true;
            };
            ok = wait_bar(S.B.own_full0, items & 1u, ctl) && scores(0) && wait_bar(S.B.own_full0 + 8u, items & 1u, ctl) && dps(0);
            for (int k = 0; ok && k < total; ++k) {
                const bool next = k + 1 < total;
                const uint32_t step = done + k, slot = step % kSlots;
                ok = wait_bar(S.B.s_read, step & 1u, ctl);
                if (!ok) break;
                tc_fence_after();
                ok = (!next || scores(k + 1)) && wait_bar(S.B.ds_ready, step & 1u, ctl);
                // the item before has left the sums
                if (ok && k == 0) ok = wait_bar(S.B.out_empty, (items & 1u) ^ 1u, ctl);
                if (!ok) break;
                tc_fence_after();
                issue_pv<32>(leader, dq, dp, S.ring_a + slot * tile_bytes, p.idesc_pv, k != 0);
                mma_commit(leader, S.B.empty_a0 + 8u * slot);
                if (!next) mma_commit(leader, S.B.out_full);
                else ok = dps(k + 1);
            }
            done += total;
            ++items;
        }
        drain_mmas(p, S, leader);
    } else if (warp < 16) {
        const DsScale<BF16> scale(p);
        for (int n = 0; next_item(S.I, ctl, n, item); ++n) {
            const QueryTile<SPLIT> qt(p, item);
            if (!compute_dq<BF16, SPLIT>(p, S, ctl, tmem, item.at, qt, scale, done, items)) break;
        }
    }
    grad_end(p, S, tmem);
    // This kernel began without waiting for the one before it (the statistics that
    // both need were complete before either began); what follows waits for this one alone.
    grid_dep_wait();
}

// Sums of the parts of up to 16 rows of one head, added in order, times f, to 16-bit rows.
template <bool BF16>
__device__ __forceinline__ void join_rows(const float *src, long long width, long long part, int parts, float f, uint16_t *out,
                                          long long ld, int rows, int dim)
{
    const int vecs = dim / 4;
    for (int i = threadIdx.x; i < rows * vecs; i += 128) {
        const int r = i / vecs, c = (i - r * vecs) * 4;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int s = 0; s < parts; ++s) {
            const float4 u = ld_written(reinterpret_cast<const float4 *>(src + s * part + r * width + c));
            v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        *reinterpret_cast<uint2 *>(out + r * ld + c) = make_uint2(round2<BF16>(v.x * f, v.y * f), round2<BF16>(v.z * f, v.w * f));
    }
}

// CTAs [0, key_items): dk and dv of 16 keys and a head; the others: dq of 16 queries and a head.
template <bool BF16>
__global__ void __launch_bounds__(128) attention_grad_join_kernel(const __grid_constant__ CatParams p, unsigned key_items)
{
    grid_dep_launch_dependents();
    grid_dep_wait();
    if (blockIdx.x < key_items) {
        const int head = static_cast<int>(blockIdx.x % p.kv_heads);
        const Place at = find_tile(p, blockIdx.x / p.kv_heads, CAT_JOIN_ROWS, true);
        if (at.tile < 0) return;
        const int rows = min(CAT_JOIN_ROWS, at.kl - at.tile * CAT_JOIN_ROWS);
        const long long width = static_cast<long long>(p.kv_heads) * p.dim, token = at.k0 + at.tile * CAT_JOIN_ROWS, kind = p.k_tokens * width,
                        col = static_cast<long long>(head) * p.dim;
        const float *src = p.k_partial + token * width + col;
        join_rows<BF16>(src, width, 2 * kind, p.k_splits, 1.0f, static_cast<uint16_t *>(p.dv) + token * p.ld_dv + col, p.ld_dv, rows, p.dim);
        join_rows<BF16>(src + kind, width, 2 * kind, p.k_splits, p.scale, static_cast<uint16_t *>(p.dk) + token * p.ld_dk + col, p.ld_dk, rows,
                        p.dim);
    } else {
        const unsigned item = blockIdx.x - key_items;
        const int head = static_cast<int>(item % p.heads);
        const Place at = find_tile(p, item / p.heads, CAT_JOIN_ROWS, false);
        if (at.tile < 0) return;
        const long long width = static_cast<long long>(p.heads) * p.dim, token = at.q0 + at.tile * CAT_JOIN_ROWS, col = static_cast<long long>(head) * p.dim;
        join_rows<BF16>(p.q_partial + token * width + col, width, p.q_tokens * width, p.q_splits, p.scale,
                        static_cast<uint16_t *>(p.dq) + token * p.ld_dq + col, p.ld_dq, min(CAT_JOIN_ROWS, at.ql - at.tile * CAT_JOIN_ROWS), p.dim);
    }
}

}  // namespace
}  // namespace cdg

size_t cat_smem_grad(int slices) { return 1024 + (2 + 2 * cdg::kSlots) * cdg::kSliceBytes * slices + cdg::kSlots * CAT_TILE * 8 + cdg::kGradTail; }

namespace {
typedef void (*Kernel)(CatParams);
template <int SLICES, bool SPLIT>
Kernel dkv_kernel(int bf16) { return bf16 ? cdg::attention_dkv_kernel<true, SLICES, SPLIT> : cdg::attention_dkv_kernel<false, SLICES, SPLIT>; }
Kernel dkv_kernel(int slices, int bf16, int split)
{
    return slices == 2 ? (split ? dkv_kernel<2, true>(bf16) : dkv_kernel<2, false>(bf16))
                       : (split ? dkv_kernel<1, true>(bf16) : dkv_kernel<1, false>(bf16));
}
template <int SLICES, bool SPLIT>
Kernel dq_kernel(int bf16) { return bf16 ? cdg::attention_dq_kernel<true, SLICES, SPLIT> : cdg::attention_dq_kernel<false, SLICES, SPLIT>; }
Kernel dq_kernel(int slices, int bf16, int split)
{
    return slices == 2 ? (split ? dq_kernel<2, true>(bf16) : dq_kernel<2, false>(bf16))
                       : (split ? dq_kernel<1, true>(bf16) : dq_kernel<1, false>(bf16));
}
}  // namespace

long long cat_stat_ctas(long long tokens, int heads, int bf16)
{
    const long long n = ((tokens + cdg::kStatRows - 1) / cdg::kStatRows * heads + cdg::kStatGroups - 1) / cdg::kStatGroups;
    return bf16 ? n : std::min<long long>(n, cdg::kSizeCtas);
}

cudaError_t cat_launch_stats(const CatParams &p, int bf16, cudaStream_t s)
{
    using namespace cdg;
    const dim3 grid(static_cast<unsigned>(p.stat_ctas + p.size_ctas)), block(kStatThreads);
    return bf16 ? launch_early(attention_stats_kernel<true>, grid, block, 0, s, p)
                : launch_early(attention_stats_kernel<false>, grid, block, 0, s, p);
}

cudaError_t cat_launch_dkv(const CatParams &p, int bf16, long long items, cudaStream_t s)
{
    using namespace cdg;
    const dim3 grid(static_cast<unsigned>(items * p.k_splits)), block(CAT_GRAD_THREADS);
    const int smem = static_cast<int>(cat_smem_grad(p.slices));
    const Kernel k = dkv_kernel(p.slices, bf16, p.k_splits > 1);
    return launch_early(k, grid, block, smem, s, p);
}

cudaError_t cat_launch_grad_join(const CatParams &p, int bf16, long long key_items, long long query_items, cudaStream_t s)
{
    using namespace cdg;
    const unsigned keys = p.k_splits > 1 ? static_cast<unsigned>(key_items) : 0u, queries = p.q_splits > 1 ? static_cast<unsigned>(query_items) : 0u;
    if (keys + queries == 0) return cudaSuccess;
    return bf16 ? launch_early(attention_grad_join_kernel<true>, dim3(keys + queries), dim3(128), 0, s, p, keys)
                : launch_early(attention_grad_join_kernel<false>, dim3(keys + queries), dim3(128), 0, s, p, keys);
}

// After cat_launch_dkv on the same stream, beside whose end it begins; without
// keys there is no such launch, and this one waits for all before it.
cudaError_t cat_launch_dq(const CatParams &p, int bf16, long long items, cudaStream_t s)
{
    using namespace cdg;
    const dim3 grid(static_cast<unsigned>(items * p.q_splits)), block(CAT_GRAD_THREADS);
    const int smem = static_cast<int>(cat_smem_grad(p.slices));
    const Kernel k = dq_kernel(p.slices, bf16, p.q_splits > 1);
    if (p.k_tokens > 0) return launch_early(k, grid, block, smem, s, p);
    k<<<grid, block, smem, s>>>(p);
    return cudaGetLastError();
}

cudaError_t cat_prepare_grad()
{
    for (int i = 0; i < 16; ++i) {
        const int slices = 1 + (i & 1), bf16 = i >> 1 & 1, split = i >> 2 & 1;
        const cudaError_t e = cudaFuncSetAttribute(i & 8 ? dkv_kernel(slices, bf16, split) : dq_kernel(slices, bf16, split),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, CDG_MAX_DYN_SMEM);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}
