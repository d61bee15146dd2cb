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
// (Q once, K and V steps through a ring), warp 9 MMA issue.
#include "attention_device.cuh"

namespace cdg {
namespace {

constexpr int kStages = 4;  // ring slots of one K or V step

struct FwdBars {
    uint32_t q_full, full0, empty0, s_full0, p_ready0, o_full0, drain;
};

struct Range {
    int lo, hi;
    __device__ __forceinline__ bool has(int j) const { return j >= lo && j < hi; }
};

template <bool BF16>
__device__ __forceinline__ void run_softmax(const CatParams &p, const FwdBars &B, Ctl ctl, uint32_t tmem, const Place &at,
                                            int head, int i0, int t, Range range)
{
    const int warp = threadIdx.x / 32, row = threadIdx.x & 127, i = i0 + row;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t s_col = tmem + lanes + 128u * t, o_col = tmem + lanes + 256u + 64u * p.slices * t;
    const float c = p.scale_log2;
    const f32x2 c2 = pack2(c, c);
    const int r = i + at.kl - at.ql;  // the last key that a causal query sees
    const bool valid = i < at.ql;
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int j = range.lo; j < range.hi; ++j) {
        const int n = j - range.lo;
        if (!wait_bar(B.s_full0 + 8u * t, n & 1, ctl)) {
            ok = false;
            break;
        }
        tc_fence_after();
        float s[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld_32(s_col + 32u * q, s[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_wait(s[q]);
        // columns [lo, hi) of this step are seen; most steps are seen whole
        const int k0 = j * CAT_TILE, r_first = i0 + at.kl - at.ql;
        const bool whole = k0 + CAT_TILE <= at.kl && (!p.causal || k0 + CAT_TILE - 1 <= r_first) &&
                           (!p.window || k0 > r_first + 127 - p.window);
        if (!whole) {
            const int hi = min(at.kl, p.causal ? r + 1 : at.kl) - k0, lo = p.window ? r - p.window + 1 - k0 : 0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (32 * q + e < lo || 32 * q + e >= hi) s[q][e] = -INFINITY;
        }
        float mx[4] = {s[0][0], s[1][0], s[2][0], s[3][0]};
#pragma unroll
        for (int e = 1; e < 32; ++e)
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = fmaxf(mx[q], s[q][e]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (n == 0) {
            m = top;
        } else {
            const bool grow = (top - m) * c > 8.0f;  // (false where both are -inf)
            if (__any_sync(0xFFFFFFFFu, grow)) {
                // S of this step is complete, so the P V of the step before is: O may be rescaled
                const float f = grow ? exp2_approx((m - top) * c) : 1.0f;
                l *= f;
                if (grow) m = top;
#pragma unroll 1
                for (int c0 = 0; c0 < 64 * p.slices; c0 += 8) tmem_scale_8(o_col + c0, f);
            }
        }
        const float mc = m == -INFINITY ? 0.0f : __fmul_rn(m, c);
        const f32x2 shift = pack2(-mc, -mc);
        f32x2 sum = pack2(0.0f, 0.0f), sum_b = sum;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                float a, b;
                unpack2(fma2(pack2(s[q][e], s[q][e + 1]), c2, shift), a, b);
                a = exp2_approx(a);
                b = exp2_approx(b);
                if (e & 2) sum_b = add2(sum_b, pack2(a, b));
                else sum = add2(sum, pack2(a, b));
                w[e / 2] = round2<BF16>(a, b);
            }
            tmem_st_16(s_col + 16u * q, w);
        }
        float a, b;
        unpack2(add2(sum, sum_b), a, b);
        l += a + b;
        tmem_st_wait();
        warp_arrive(B.p_ready0 + 8u * t);
    }
    if (ok && range.hi > range.lo) ok = wait_bar(B.o_full0 + 8u * t, 0, ctl);
    if (!ok) return;
    tc_fence_after();
    const long long token = at.q0 + i;
    uint16_t *out = static_cast<uint16_t *>(p.o) + token * p.ld_o + static_cast<long long>(head) * p.dim;
    // a row that sees nothing (l = 0, m = -inf) answers 0 and -inf
    const bool none = m == -INFINITY && l == 0.0f;
    if (range.hi > range.lo) {
        store_row<BF16>(o_col, 0, p.dim, none ? 0.0f : 1.0f / l, out, valid);
    } else if (valid) {
        zero_row(out, 0, p.dim);
    }
    if (valid)
        p.lse[static_cast<long long>(head) * p.q_tokens + token] =
            none ? -INFINITY : (__fmul_rn(m, c) + log2f(l)) * 0.6931471805599453f;
}

template <bool BF16>
__global__ void __launch_bounds__(CAT_THREADS, 1) attention_kernel(const __grid_constant__ CatParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t tile_bytes = kSliceBytes * p.slices;
    // shared memory: Q tiles | ring | mbarriers, flags
    const uint32_t q_smem = base, ring = base + 2 * tile_bytes, bars = ring + kStages * tile_bytes;
    const FwdBars B{bars, bars + 8, bars + 8 + 8 * kStages, bars + 8 + 16 * kStages, bars + 24 + 16 * kStages,
                    bars + 40 + 16 * kStages, bars + 56 + 16 * kStages};
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + (bars - raw) + 64 + 16 * kStages);
    volatile uint32_t *abort_flag = tmem_slot + 1;
    volatile uint32_t *slot_parity = tmem_slot + 2;  // of each ring slot's last load, and of Q's
    const int warp = threadIdx.x / 32;
    grid_dep_launch_dependents();
    if (threadIdx.x == 0) {
        mbar_init(B.q_full, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(B.full0 + 8u * s, 1);
            mbar_init(B.empty0 + 8u * s, 1);
        }
        for (int s = 0; s <= kStages; ++s) slot_parity[s] = 0u;
        for (int t = 0; t < 2; ++t) {
            mbar_init(B.s_full0 + 8u * t, 1);
            mbar_init(B.p_ready0 + 8u * t, 4);
            mbar_init(B.o_full0 + 8u * t, 1);
        }
        mbar_init(B.drain, 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    grid_dep_wait();
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    const int head = static_cast<int>(blockIdx.x % p.heads);
    Place at = find_tile(p, blockIdx.x / p.heads, 2 * CAT_TILE, false);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Ctl ctl{abort_flag, p.status};
    if (at.tile >= 0) {
        // a sequence's last tiles first: under a causal mask they are the longest
        const int i0 = ((at.ql + 2 * CAT_TILE - 1) / (2 * CAT_TILE) - 1 - at.tile) * 2 * CAT_TILE;
        Range range[2];
        for (int t = 0; t < 2; ++t) {
            const int a = i0 + t * CAT_TILE;
            if (a < at.ql) key_steps(p, at, a, min(a + CAT_TILE, at.ql), range[t].lo, range[t].hi);
            else range[t] = Range{0, 0};
        }
        const bool some0 = range[0].hi > range[0].lo, some1 = range[1].hi > range[1].lo;
        const int lo = some0 && some1 ? min(range[0].lo, range[1].lo) : some0 ? range[0].lo : range[1].lo;
        const int hi = some0 && some1 ? max(range[0].hi, range[1].hi) : some0 ? range[0].hi : range[1].hi;
        const int kv_head = head / p.group;
        if (warp == 8) {
            const bool leader = elect_one_sync();
            if (leader && lo < hi) {
                for (int t = 0; t < 2; ++t)
                    if (range[t].hi > range[t].lo) {
                        if (!slot_parity[kStages]) {
                            slot_parity[kStages] = 2u;
                            mbar_arrive_expect_tx(B.q_full, (some0 + some1) * tile_bytes);
                        }
                        load_tile(q_smem + t * tile_bytes, p.tmQ, B.q_full, p.slices, head, at.q0 + i0 + t * CAT_TILE);
                    }
            }
            int stage = 0;
            uint32_t parity = 0;
            bool ok = true;
            for (int n = 0; ok && n < 2 * (hi - lo); ++n) {
                if (!wait_bar(B.empty0 + 8u * stage, parity ^ 1u, ctl)) {
                    ok = false;
                    break;
                }
                if (leader) {
                    slot_parity[stage] = parity | 2u;
                    mbar_arrive_expect_tx(B.full0 + 8u * stage, tile_bytes);
                    load_tile(ring + stage * tile_bytes, n & 1 ? p.tmV : p.tmK, B.full0 + 8u * stage, p.slices, kv_head,
                              at.k0 + (lo + n / 2) * CAT_TILE);
                }
                __syncwarp();
                if (++stage == kStages) {
                    stage = 0;
                    parity ^= 1u;
                }
            }
        } else if (warp == 9) {
            const bool leader = elect_one_sync();
            const uint32_t o_cols = 64u * p.slices;
            // the n-th load of the ring: step lo + n / 2, K (even) or V (odd)
            auto slot = [&](int n) { return ring + (n % kStages) * tile_bytes; };
            auto filled = [&](int n) { return wait_bar(B.full0 + 8u * (n % kStages), (n / kStages) & 1, ctl); };
            auto scores = [&](int t, int n) {
                issue_qk(tmem + 128u * t, q_smem + t * tile_bytes, slot(n), p.idesc_qk, p.ksteps);
                umma_commit(B.s_full0 + 8u * t);
            };
            bool ok = lo < hi && wait_bar(B.q_full, 0, ctl) && filled(0);
            if (ok) {
                tc_fence_after();
                if (leader) {
                    for (int t = 0; t < 2; ++t)
                        if (range[t].has(lo)) scores(t, 0);
                    umma_commit(B.empty0);
                }
                __syncwarp();
            }
            for (int j = lo; ok && j < hi; ++j) {
                const int nv = 2 * (j - lo) + 1, nk = nv + 1;
                const bool next = j + 1 < hi;
                ok = filled(nv) && (!next || filled(nk));
                if (!ok) break;
                tc_fence_after();
                const int valid = at.kl - j * CAT_TILE;
                if (valid < CAT_TILE) zero_rows(slot(nv), p.slices, valid);
                for (int t = 0; t < 2; ++t) {
                    if (range[t].has(j)) {
                        const int n = j - range[t].lo;
                        ok = wait_bar(B.p_ready0 + 8u * t, n & 1, ctl);
                        if (!ok) break;
                        tc_fence_after();
                        if (leader) {
                            const uint32_t a = tmem + 128u * t;
                            issue_pv<128>(tmem + 256u + o_cols * t, a, slot(nv), p.idesc_pv, n != 0);
                            if (j + 1 == range[t].hi) umma_commit(B.o_full0 + 8u * t);
                        }
                        __syncwarp();
                    }
                    if (next && leader && range[t].has(j + 1)) scores(t, nk);
                    __syncwarp();
                }
                if (!ok) break;
                if (leader) {
                    umma_commit(B.empty0 + 8u * (nv % kStages));
                    if (next) umma_commit(B.empty0 + 8u * (nk % kStages));
                }
                __syncwarp();
            }
            if (leader) umma_commit(B.drain);
            __syncwarp();
            volatile uint32_t no_abort = 0;
            wait_bar(B.drain, 0, Ctl{&no_abort, p.status});
        } else if (warp < 8) {
            const int t = warp / 4;
            if (i0 + t * CAT_TILE < at.ql) run_softmax<BF16>(p, B, ctl, tmem, at, head, i0 + t * CAT_TILE, t, range[t]);
        }
    }
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) {
        // let the latest load of every used slot land before the CTA exits
        volatile uint32_t no_abort = 0;
        const Ctl drain_ctl{&no_abort, p.status};
        for (int s = 0; s <= kStages; ++s) {
            const uint32_t v = slot_parity[s];
            if (v & 2u) wait_bar(s == kStages ? B.q_full : B.full0 + 8u * s, v & 1u, drain_ctl);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace
}  // namespace cdg

size_t cat_smem_forward(int slices) { return 1024 + (2 + cdg::kStages) * cdg::kSliceBytes * slices + 256; }

cudaError_t cat_launch_forward(const CatParams &p, int bf16, long long items, cudaStream_t s)
{
    using namespace cdg;
    const dim3 grid(static_cast<unsigned>(items)), block(CAT_THREADS);
    const int smem = static_cast<int>(cat_smem_forward(p.slices));
    return bf16 ? launch_early(attention_kernel<true>, grid, block, smem, s, p)
                : launch_early(attention_kernel<false>, grid, block, smem, s, p);
}

cudaError_t cat_prepare_forward()
{
    cudaError_t e = cudaFuncSetAttribute(cdg::attention_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, CDG_MAX_DYN_SMEM);
    return e != cudaSuccess ? e
                            : cudaFuncSetAttribute(cdg::attention_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   CDG_MAX_DYN_SMEM);
}
