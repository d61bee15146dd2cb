// Attention over packed sequences for sm_103a: o = softmax(scale q k^T) v over
// the keys that each query sees, and the log of each row's sum (lse) for the
// gradient (attention_grad_sm103.cu).
//
// A CTA takes 256 queries of a head, as two MMA tiles of 128, through the keys
// in steps of 128.  Scores S = Q K^T go to tensor memory; a warpgroup a tile
// turns them into P = 2^(S c - m c), c = scale log2(e), in registers (a thread
// a row) and puts P back over S as the 16-bit A operand of O += P V, whose
// sums stay in tensor memory.  m follows the running maximum only when it grows
// by more than 2^8 (P is at most 256 then, far inside both 16-bit types' range),
// so that O is rarely rescaled; the row sum is of the unrounded fp32 P, and O /
// sum is the same for any m.
//
// While one tile's warpgroup works on its scores, the tensor cores run the
// other tile's P V and its next Q K^T: S0 S1 O0 O1 fill tensor memory.
//
// Roles (384 threads): warps 0-3 and 4-7 the tiles' softmax, warp 8 TMA loads
// (Q once an item, K and V steps through a ring), warp 9 MMA issue, warp 10 items.
//
// Measured (GB300, 8192 causal tokens, 16 heads of 128 over 4, bf16): 198 us, 1390
// TFLOP/s call after call, where the power limit lowers the SM clock (189 us for ten at 2.07
// GHz); packed documents of 1 to 4096 tokens 150 us, 1100 (145); 8192 x 8192 heads of 64
// 814 TFLOP/s.  A step of a pair of tiles takes 2.6 thousand cycles, its products
// 2.05: what bounds it is the chain of one tile, scores -> softmax (1.1 thousand
// cycles) -> P V -> next scores, which the other tile's products do not quite cover.
#include "attention_device.cuh"

namespace cdg {
namespace {

constexpr int kStages = 4;  // ring slots of one K or V step

constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpItems = 10;

struct FwdBars {
    uint32_t full0, empty0;       // [kStages]
    uint32_t q_full0, q_empty0;   // [2], as all of these: a tile's Q
    uint32_t s_full0, p_ready0, o_full0, o_empty0;
    uint32_t drain;
};

struct Range {
    int lo, hi;
};

// An item's 256 queries of one head: two tiles from query i0, and the steps of
// keys that each of them and both together see (SPLIT: of those, its part).
template <bool SPLIT>
struct Steps {
    int i0;
    Range tile[2], all;
    int head, part;
    __device__ __forceinline__ Steps(const CatParams &p, const Item &item)
    {
        const Place &at = item.at;
        head = SPLIT ? item.head / p.q_splits : item.head;
        part = SPLIT ? item.head - head * p.q_splits : 0;
        // a sequence's last tiles first: under a causal mask they are the longest
        i0 = ((at.ql + 2 * CAT_TILE - 1) / (2 * CAT_TILE) - 1 - at.tile) * 2 * CAT_TILE;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int a = i0 + t * CAT_TILE;
            if (a < at.ql) key_steps(p, at, a, min(a + CAT_TILE, at.ql), tile[t].lo, tile[t].hi);
            else tile[t] = Range{0, 0};
        }
        const bool some0 = tile[0].hi > tile[0].lo, some1 = tile[1].hi > tile[1].lo;
        all.lo = some0 && some1 ? min(tile[0].lo, tile[1].lo) : some0 ? tile[0].lo : tile[1].lo;
        all.hi = some0 && some1 ? max(tile[0].hi, tile[1].hi) : some0 ? tile[0].hi : tile[1].hi;
        if (SPLIT) {
            take_part(all.lo, all.hi, part, p.q_splits);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                tile[t] = Range{max(tile[t].lo, all.lo), min(tile[t].hi, all.hi)};
                if (tile[t].hi <= tile[t].lo) tile[t] = Range{all.lo, all.lo};
            }
        }
    }
};

// Scores past [lo, hi) are not seen.
__device__ __forceinline__ void hide(float (&s)[32], int lo, int hi)
{
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (e < lo || e >= hi) s[e] = -INFINITY;
}

// One tile's softmax over one item.  steps, items: what this tile has done before.
template <bool BF16, bool SPLIT>
__device__ __forceinline__ bool run_softmax(const CatParams &p, const FwdBars &B, Ctl ctl, uint32_t tmem, const Place &at,
                                            int head, int part, int i0, int t, Range range, uint32_t &steps, uint32_t &items)
{
    const int warp = threadIdx.x / 32, row = threadIdx.x & 127, i = i0 + row;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t s_col = tmem + lanes + 128u * t, o_col = tmem + lanes + 256u + 64u * p.slices * t;
    const float c = p.scale_log2;
    const f32x2 c2 = pack2(c, c);
    const int r = i + at.kl - at.ql;  // the last key that a causal query sees
    float m = -INFINITY, l = 0.0f;
    for (int j = range.lo; j < range.hi; ++j) {
        // columns [lo, hi) of this step are seen; most steps are seen whole
        const int k0 = j * CAT_TILE, r_first = i0 + at.kl - at.ql;
        const bool whole = k0 + CAT_TILE <= at.kl && (!p.causal || k0 + CAT_TILE - 1 <= r_first) &&
                           (!p.window || k0 > r_first + 127 - p.window);
        const int hi = min(at.kl, p.causal ? r + 1 : at.kl) - k0, lo = p.window ? r - p.window + 1 - k0 : 0;
        if (!wait_bar(B.s_full0 + 8u * t, steps & 1u, ctl)) return false;
        ++steps;
        tc_fence_after();
        if (j == range.lo) {  // (the maximum alone)
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float s[32];
                tmem_ld_32(s_col + 32u * q, s);
                tmem_wait(s);
                if (!whole) hide(s, lo - 32 * q, hi - 32 * q);
#pragma unroll
                for (int e = 0; e < 32; e += 2) mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], s[e], s[e + 1]);
            }
            m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        }
        // One pass makes P about the m of the steps before and finds the step's own
        // maximum beside it; where that has grown too far, m moves up and the pass is
        // made again.
        uint32_t w[4][16];
        f32x2 sum[2];
        for (;;) {
            const float mc = m == -INFINITY ? 0.0f : __fmul_rn(m, c);
            const f32x2 shift = pack2(-mc, -mc);
            float mx[2] = {-INFINITY, -INFINITY};
            sum[0] = sum[1] = pack2(0.0f, 0.0f);
            auto exponentials = [&](float(&v)[32], int q) {
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    mx[(e >> 1) & 1] = max3(mx[(e >> 1) & 1], v[e], v[e + 1]);
                    float a, b;
                    unpack2(fma2(pack2(v[e], v[e + 1]), c2, shift), a, b);
                    a = exp2_approx(a);
                    b = exp2_approx(b);
                    sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pack2(a, b));
                    w[q][e / 2] = round2<BF16>(a, b);
                }
            };
            // (the last quarter is loaded into the first one's registers)
            float s[3][32];
#pragma unroll
            for (int q = 0; q < 3; ++q) tmem_ld_32(s_col + 32u * q, s[q]);
#pragma unroll
            for (int q = 0; q < 3; ++q) tmem_wait(s[q]);
            if (!whole) {
#pragma unroll
                for (int q = 0; q < 3; ++q) hide(s[q], lo - 32 * q, hi - 32 * q);
            }
            exponentials(s[0], 0);
            tmem_ld_32(s_col + 96u, s[0]);
            exponentials(s[1], 1);
            exponentials(s[2], 2);
            tmem_wait(s[0]);
            if (!whole) hide(s[0], lo - 96, hi - 96);
            exponentials(s[0], 3);
            const float top = fmaxf(mx[0], mx[1]);
            const bool grow = (top - m) * c > 8.0f;  // (false where both are -inf)
            if (!__any_sync(0xFFFFFFFFu, grow)) break;
            // S of this step is complete, so the P V of the step before is: O may be rescaled
            const float f = grow ? exp2_approx((m - top) * c) : 1.0f;
            l *= f;
            if (grow) m = top;
            if (j > range.lo) {
#pragma unroll 1
                for (int c0 = 0; c0 < 64 * p.slices; c0 += 8) tmem_scale_8(o_col + c0, f);
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_st_16(s_col + 16u * q, w[q]);
        float a, b;
        unpack2(add2(sum[0], sum[1]), a, b);
        l += a + b;
        tmem_st_wait();
        warp_arrive(B.p_ready0 + 8u * t);
    }
    const bool valid = i < at.ql;
    const long long token = at.q0 + i, first = token - (threadIdx.x & 31), width = static_cast<long long>(p.heads) * p.dim;
    // a row that sees nothing (l = 0, m = -inf) answers 0 and -inf
    const bool none = m == -INFINITY && l == 0.0f;
    float *lse = SPLIT ? p.lse_partial + static_cast<long long>(part) * p.heads * p.q_tokens : p.lse;
    if (valid)
        lse[static_cast<long long>(head) * p.q_tokens + token] =
            none ? -INFINITY : (__fmul_rn(m, c) + log2f(l)) * 0.6931471805599453f;
    uint16_t *out = static_cast<uint16_t *>(p.o) + first * p.ld_o + static_cast<long long>(head) * p.dim;
    if (range.hi > range.lo) {
        if (!wait_bar(B.o_full0 + 8u * t, items & 1u, ctl)) return false;
        ++items;
        tc_fence_after();
        const float f = none ? 0.0f : 1.0f / l;
        const int rows = at.ql - (i & ~31);
        if (SPLIT)
            store_rows_f32(o_col, 0, p.dim, f, p.q_partial + (static_cast<long long>(part) * p.q_tokens + first) * width + static_cast<long long>(head) * p.dim, width, rows);
        else
            store_rows<BF16>(o_col, 0, p.dim, f, out, p.ld_o, rows);
        warp_arrive(B.o_empty0 + 8u * t);
    } else if (valid && !SPLIT) {
        zero_row(out + (threadIdx.x & 31) * p.ld_o, 0, p.dim);
    }
    return true;
}

template <bool BF16, int SLICES, bool SPLIT>
__global__ void __launch_bounds__(CAT_THREADS, 1) attention_kernel(const __grid_constant__ CatParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    constexpr uint32_t tile_bytes = kSliceBytes * SLICES;
    // shared memory: Q tiles | ring | items | mbarriers, flags
    const uint32_t q_smem = base, ring = base + 2 * tile_bytes, items_at = ring + kStages * tile_bytes, bars = items_at + kItemBytes;
    const FwdBars B{bars, bars + 8 * kStages, bars + 16 * kStages, bars + 16 * kStages + 16, bars + 16 * kStages + 32,
                    bars + 16 * kStages + 48, bars + 16 * kStages + 64, bars + 16 * kStages + 80, bars + 16 * kStages + 96};
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + (bars - raw) + 16 * kStages + 104);
    volatile uint32_t *abort_flag = tmem_slot + 1;
    volatile uint32_t *slot_parity = tmem_slot + 2;  // of each ring slot's last load, and of the Q tiles'
    const int warp = threadIdx.x / 32;
    grid_dep_launch_dependents();
    const ItemBars I = init_items(smem_raw + (items_at - raw), items_at, 10);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(B.full0 + 8u * s, 1);
            mbar_init(B.empty0 + 8u * s, 1);
        }
        for (int s = 0; s < kStages + 2; ++s) slot_parity[s] = 0u;
        for (int t = 0; t < 2; ++t) {
            for (uint32_t b : {B.q_full0, B.q_empty0, B.s_full0, B.o_full0}) mbar_init(b + 8u * t, 1);
            mbar_init(B.p_ready0 + 8u * t, 4);
            mbar_init(B.o_empty0 + 8u * t, 4);
        }
        mbar_init(B.drain, 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    grid_dep_wait();
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Ctl ctl{abort_flag, p.status};
    if (warp == kWarpItems) {
        run_items(p, I, ctl, 2 * CAT_TILE, false, p.heads * p.q_splits);
    } else if (warp == kWarpLoad) {
        const bool leader = elect_one_sync();
        Item item;
        uint32_t q_loads[2] = {0, 0};
        int stage = 0;
        uint32_t parity = 0;
        bool ok = true;
        for (int n = 0; ok && next_item(I, ctl, n, item); ++n) {
            const Steps<SPLIT> st(p, item);
            auto load_q = [&](int t) {
                if (st.tile[t].hi <= st.tile[t].lo) return true;
                if (!wait_bar(B.q_empty0 + 8u * t, (q_loads[t] & 1u) ^ 1u, ctl)) return false;
                if (leader) {
                    slot_parity[kStages + t] = (q_loads[t] & 1u) | 2u;
                    mbar_arrive_expect_tx(B.q_full0 + 8u * t, tile_bytes);
                    load_tile(q_smem + t * tile_bytes, p.tmQ, B.q_full0 + 8u * t, SLICES, st.head, item.at.q0 + st.i0 + t * CAT_TILE);
                }
                __syncwarp();
                ++q_loads[t];
                return true;
            };
            ok = load_q(0);
            for (int k = 0; ok && k < 2 * (st.all.hi - st.all.lo); ++k) {
                if (!wait_bar(B.empty0 + 8u * stage, parity ^ 1u, ctl)) {
                    ok = false;
                    break;
                }
                if (leader) {
                    slot_parity[stage] = parity | 2u;
                    mbar_arrive_expect_tx(B.full0 + 8u * stage, tile_bytes);
                    load_tile(ring + stage * tile_bytes, k & 1 ? p.tmV : p.tmK, B.full0 + 8u * stage, SLICES, st.head / p.group,
                              item.at.k0 + (st.all.lo + k / 2) * CAT_TILE);
                }
                __syncwarp();
                if (++stage == kStages) {
                    stage = 0;
                    parity ^= 1u;
                }
                if (k == 0) ok = load_q(1);
            }
            if (leader) mbar_arrive(I.go);
            __syncwarp();
        }
    } else if (warp == kWarpMma) {
        const uint32_t leader = elect_one_sync();
        const uint32_t tm = uniform(tmem), o_cols = 64u * SLICES;
        auto scores = [&](int t, int slot) {
            issue_qk<SLICES>(leader, tm + 128u * t, q_smem + t * tile_bytes, ring + slot * tile_bytes, p.idesc_qk, p.ksteps);
            mma_commit(leader, B.s_full0 + 8u * t);
        };
        uint32_t loads = 0;                  // of the ring, so far
        uint32_t done0 = 0, done1 = 0;       // steps of each tile
        uint32_t items0 = 0, items1 = 0;     // items of each tile
        bool ok = true;
        Item item;
        for (int n = 0; ok && next_item(I, ctl, n, item); ++n) {
            const Steps<SPLIT> st(p, item);
            const int lo = st.all.lo, steps = uniform(st.all.hi - lo), kl = uniform(item.at.kl - lo * CAT_TILE);
            if (steps <= 0) continue;
            // each tile's steps [first, end), counted from lo
            const int first0 = uniform(st.tile[0].lo - lo), end0 = uniform(st.tile[0].hi - lo);
            const int first1 = uniform(st.tile[1].lo - lo), end1 = uniform(st.tile[1].hi - lo);
            ok = wait_bar(B.full0 + 8u * (loads % kStages), (loads / kStages) & 1u, ctl);
            if (ok && first0 < end0) ok = wait_bar(B.q_full0, items0 & 1u, ctl);
            if (!ok) break;
            tc_fence_after();
            if (first0 < end0 && first0 == 0) {
                scores(0, loads % kStages);
                if (end0 == 1) mma_commit(leader, B.q_empty0);
            }
            if (first1 < end1) ok = wait_bar(B.q_full0 + 8u, items1 & 1u, ctl);
            if (!ok) break;
            tc_fence_after();
            if (first1 < end1 && first1 == 0) {
                scores(1, loads % kStages);
                if (end1 == 1) mma_commit(leader, B.q_empty0 + 8u);
            }
            mma_commit(leader, B.empty0 + 8u * (loads % kStages));
            ++loads;
            // the ring goes on with this step's V, then the next one's K
            for (int j = 0; ok && j < steps; ++j) {
                const bool next = j + 1 < steps;
                const uint32_t v_slot = loads % kStages, k_slot = (loads + 1) % kStages;
                ok = wait_bar(B.full0 + 8u * v_slot, (loads / kStages) & 1u, ctl) &&
                     (!next || wait_bar(B.full0 + 8u * k_slot, ((loads + 1) / kStages) & 1u, ctl));
                if (!ok) break;
                tc_fence_after();
                const int valid = kl - j * CAT_TILE;
                if (valid < CAT_TILE) zero_rows(ring + v_slot * tile_bytes, SLICES, valid);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int first = t ? first1 : first0, end = t ? end1 : end0;
                    uint32_t &done = t ? done1 : done0, &its = t ? items1 : items0;
                    if (j >= first && j < end) {
                        ok = wait_bar(B.p_ready0 + 8u * t, done & 1u, ctl);
                        // the item before has left O
                        if (ok && j == first) ok = wait_bar(B.o_empty0 + 8u * t, (its & 1u) ^ 1u, ctl);
                        if (!ok) break;
                        ++done;
                        tc_fence_after();
                        issue_pv<128>(leader, tm + 256u + o_cols * t, tm + 128u * t, ring + v_slot * tile_bytes, p.idesc_pv, j != first);
                        if (j + 1 == end) {
                            mma_commit(leader, B.o_full0 + 8u * t);
                            ++its;
                        }
                    }
                    if (next && j + 1 >= first && j + 1 < end) {
                        scores(t, k_slot);
                        if (j + 2 == end) mma_commit(leader, B.q_empty0 + 8u * t);
                    }
                }
                if (!ok) break;
                mma_commit(leader, B.empty0 + 8u * v_slot);
                if (next) mma_commit(leader, B.empty0 + 8u * k_slot);
                loads += next ? 2 : 1;
            }
        }
        mma_commit(leader, B.drain);
        volatile uint32_t no_abort = 0;
        wait_bar(B.drain, 0, Ctl{&no_abort, p.status});
    } else if (warp < 8) {
        const int t = warp / 4;
        uint32_t steps = 0, items = 0;
        Item item;
        for (int n = 0; next_item(I, ctl, n, item); ++n) {
            const Steps<SPLIT> st(p, item);
            if (st.i0 + t * CAT_TILE < item.at.ql &&
                !run_softmax<BF16, SPLIT>(p, B, ctl, tmem, item.at, st.head, st.part, st.i0 + t * CAT_TILE, t, t ? st.tile[1] : st.tile[0], steps,
                                   items))
                break;
        }
    }
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) {
        // let the latest load of every used slot land before the CTA exits
        volatile uint32_t no_abort = 0;
        const Ctl drain_ctl{&no_abort, p.status};
        for (int s = 0; s < kStages + 2; ++s) {
            const uint32_t v = slot_parity[s];
            if (v & 2u) wait_bar(s < kStages ? B.full0 + 8u * s : B.q_full0 + 8u * (s - kStages), v & 1u, drain_ctl);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// o and lse of 16 queries and a head from their parts': lse = log sum exp(lse_s),
// o = sum exp(lse_s - lse) o_s.  A part that saw nothing (-inf) has left its o
// unwritten: it is loaded, so that all loads are in flight together, and not used.
template <bool BF16>
__global__ void __launch_bounds__(128) attention_join_kernel(const __grid_constant__ CatParams p)
{
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int head = static_cast<int>(blockIdx.x % p.heads);
    const Place at = find_tile(p, blockIdx.x / p.heads, CAT_JOIN_ROWS, false);
    if (at.tile < 0) return;
    const int rows = min(CAT_JOIN_ROWS, at.ql - at.tile * CAT_JOIN_ROWS), vecs = p.dim / 4;
    const long long width = static_cast<long long>(p.heads) * p.dim, part = p.q_tokens * width, lse_part = static_cast<long long>(p.heads) * p.q_tokens;
    for (int i = threadIdx.x; i < rows * vecs; i += 128) {
        const int r = i / vecs, c = (i - r * vecs) * 4;
        const long long token = at.q0 + at.tile * CAT_JOIN_ROWS + r;
        const float *lse = p.lse_partial + static_cast<long long>(head) * p.q_tokens + token;
        const float *src = p.q_partial + token * width + static_cast<long long>(head) * p.dim + c;
        float top = -INFINITY;
#pragma unroll 8
        for (int s = 0; s < p.q_splits; ++s) top = fmaxf(top, ld_written(lse + s * lse_part));
        const float ref = top == -INFINITY ? 0.0f : top;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float total = 0.0f;
#pragma unroll 4
        for (int s = 0; s < p.q_splits; ++s) {
            const float l = ld_written(lse + s * lse_part);
            const float4 u = ld_written(reinterpret_cast<const float4 *>(src + s * part));
            const bool seen = l != -INFINITY;
            const float w = expf(l - ref);
            total += w;
            v.x = seen ? fmaf(w, u.x, v.x) : v.x;
            v.y = seen ? fmaf(w, u.y, v.y) : v.y;
            v.z = seen ? fmaf(w, u.z, v.z) : v.z;
            v.w = seen ? fmaf(w, u.w, v.w) : v.w;
        }
        const float f = total == 0.0f ? 0.0f : 1.0f / total;
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + token * p.ld_o + static_cast<long long>(head) * p.dim + c) =
            make_uint2(round2<BF16>(v.x * f, v.y * f), round2<BF16>(v.z * f, v.w * f));
        if (c == 0) p.lse[static_cast<long long>(head) * p.q_tokens + token] = total == 0.0f ? -INFINITY : top + logf(total);
    }
}

}  // namespace
}  // namespace cdg

size_t cat_smem_forward(int slices) { return 1024 + (2 + cdg::kStages) * cdg::kSliceBytes * slices + cdg::kItemBytes + 256; }

namespace {
typedef void (*Kernel)(CatParams);
template <int SLICES, bool SPLIT>
Kernel forward_kernel(int bf16) { return bf16 ? cdg::attention_kernel<true, SLICES, SPLIT> : cdg::attention_kernel<false, SLICES, SPLIT>; }
Kernel forward_kernel(int slices, int bf16, int split)
{
    return slices == 2 ? (split ? forward_kernel<2, true>(bf16) : forward_kernel<2, false>(bf16))
                       : (split ? forward_kernel<1, true>(bf16) : forward_kernel<1, false>(bf16));
}
}  // namespace

cudaError_t cat_launch_forward(const CatParams &p, int bf16, long long items, long long join_items, cudaStream_t s)
{
    using namespace cdg;
    const dim3 grid(static_cast<unsigned>(items * p.q_splits)), block(CAT_THREADS);
    const int smem = static_cast<int>(cat_smem_forward(p.slices));
    void (*k)(CatParams) = forward_kernel(p.slices, bf16, p.q_splits > 1);
    const cudaError_t e = launch_early(k, grid, block, smem, s, p);
    if (e != cudaSuccess || p.q_splits == 1) return e;
    const dim3 tiles(static_cast<unsigned>(join_items));
    return bf16 ? launch_early(attention_join_kernel<true>, tiles, dim3(128), 0, s, p)
                : launch_early(attention_join_kernel<false>, tiles, dim3(128), 0, s, p);
}

cudaError_t cat_prepare_forward()
{
    for (int i = 0; i < 8; ++i) {
        const cudaError_t e = cudaFuncSetAttribute(forward_kernel(1 + (i & 1), i >> 1 & 1, i >> 2), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   CDG_MAX_DYN_SMEM);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}
