// Shared by the attention's kernels (attention_sm103.cu, attention_grad_sm103.cu):
// which sequence and tile a CTA works on, what a query sees, and the small
// pieces of the tensor-memory pipelines.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attention_params.h"
#include "ptx.cuh"
#include "token_device.cuh"
#include "wait.cuh"

namespace cdg {

constexpr uint32_t kSliceBytes = CAT_TILE * 128;  // 64 columns x 128 rows of 16-bit values: 16 KB

// 2^x to about two units in the last place, 0 below 2^-126.
__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Two fp32 values rounded to the 16-bit type, the first in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t round2(float a, float b)
{
    if (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Loads of what an overlapping launch writes (statistics, parts, the forward's o and
// lse): past L1, and kept behind this kernel's wait, which read-only loads are not.
__device__ __forceinline__ float ld_written(const float *p)
{
    float v;
    asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_written(const float2 *p)
{
    float2 v;
    asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_written(const float4 *p)
{
    float4 v;
    asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint4 ld_written(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// 32 TMEM lanes x 32 columns into registers; the values are there after tmem_wait.
__device__ __forceinline__ void tmem_ld_32(uint32_t taddr, float (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr)
        : "memory");
}
// Waits for this thread's loads; tied to the registers, so that no use of them moves above it.
__device__ __forceinline__ void tmem_wait(float (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                   "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
                   "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]),
                   "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]),
                   "+f"(r[30]), "+f"(r[31])
                 :
                 : "memory");
}
// Eight columns of tensor memory times f.
__device__ __forceinline__ void tmem_scale_8(uint32_t taddr, float f)
{
    float r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                 : "r"(taddr)
                 : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7])
                 :
                 : "memory");
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] *= f;
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "f"(r[0]),
                 "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Shared-memory matrix descriptor of an MN-major operand in 128-byte-swizzled
// atoms (64 columns x 8 rows, 1 KB), slices of 64 columns kSliceBytes apart:
// the same tile that sdesc_k128_sw128 reads K-major.
__device__ __forceinline__ uint64_t sdesc_mn_slices(uint32_t saddr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((kSliceBytes >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// A value that is the same in all lanes of the (converged) warp, in a form that
// the compiler knows to be: what is computed from it, the descriptors of MMAs
// above all, then lives in uniform registers, where the instruction wants it.
__device__ __forceinline__ int uniform(int v) { return static_cast<int>(__reduce_or_sync(0xFFFFFFFFu, static_cast<unsigned>(v))); }

// MMAs and commits under a predicate instead of a branch: the whole warp runs
// the code around them, one lane issues.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t leader, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(leader)
        : "memory");
}

// D (128 x 128) = A B^T over the head's width, both K-major tiles of 64-column slices.
template <int SLICES>
__device__ __forceinline__ void issue_qk(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, int ksteps)
{
    const uint64_t ad = sdesc_k128_sw128(a), bd = sdesc_k128_sw128(b);
#pragma unroll
    for (int k = 0; k < 4 * SLICES; ++k) {
        const uint32_t at = (k >> 2) * (kSliceBytes >> 4) + 2u * (k & 3);
        if (k < ksteps) mma_ss(leader, d, ad + at, bd + at, idesc, k != 0);
    }
}

// D (128 x dim) (+)= A B over 128 rows of the MN-major tile B, A in tensor
// memory: 16-bit values, CHUNK of them (CHUNK / 2 columns) from every CHUNK-th
// column of fp32 scores that they were made from.
template <int CHUNK>
__device__ __forceinline__ void issue_pv(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add)
{
    const uint64_t bd = sdesc_mn_slices(b);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        mma_ts(leader, d, a + (16 * k / CHUNK) * CHUNK + 8u * (k % (CHUNK / 16)), bd + 128u * k, idesc, add || k != 0);
}

// ---------------------------------------------------------------- sequences

__device__ __forceinline__ int offset_at(const void *offsets, int index_bytes, int i, int tokens)
{
    if (!offsets) return i == 0 ? 0 : tokens;
    const long long t = index_bytes == 8 ? __ldg(static_cast<const long long *>(offsets) + i)
                                         : static_cast<long long>(__ldg(static_cast<const int *>(offsets) + i));
    return static_cast<int>(t < 0 ? 0 : t > tokens ? tokens : t);
}

// A CTA's sequence and tile of `rows` queries (or keys): sequences' tiles are
// counted in order.  Any offsets stay inside the tensors: they are cut to
// [0, tokens], and a sequence that ends before it begins is empty.
struct Place {
    int q0, ql, k0, kl;  // first row and length of the queries and of the keys
    int tile;            // of this sequence; -1: no such tile
};
// Where the search for a tile left off: items of one CTA come in ascending order,
// and the next one's search goes on there (a search from the first one would read all
// offsets before it for every item).  One that finds no tile leaves the end of the
// list, so that the items after it, which have none either, are searched for no more:
// a launch has a CTA for every tile that its sequences could have, and of a list that ends in
// 4095 empty sequences most have none (8192 tokens, 16 heads: 19.4 ms with a
// search for each, 0.44 ms so; 0.19 without the empty ones).
struct Scan {
    int sequence = 0;
    long long before = 0;  // tiles of the sequences before it
};
__device__ __forceinline__ Place find_tile(const CatParams &p, long long item, int rows, bool of_keys, Scan &scan)
{
    const int lane = threadIdx.x & 31;
    if (item < scan.before) scan = Scan{};
    long long before = scan.before;
    for (int s0 = scan.sequence; s0 < p.sequences; s0 += 32) {
        const int s = s0 + lane;
        int q0 = 0, ql = 0, k0 = 0, kl = 0;
        if (s < p.sequences) {
            q0 = offset_at(p.q_offsets, p.index_bytes, s, p.q_tokens);
            ql = max(0, offset_at(p.q_offsets, p.index_bytes, s + 1, p.q_tokens) - q0);
            k0 = offset_at(p.k_offsets, p.index_bytes, s, p.k_tokens);
            kl = max(0, offset_at(p.k_offsets, p.index_bytes, s + 1, p.k_tokens) - k0);
        }
        const int n = ((of_keys ? kl : ql) + rows - 1) / rows;
        int upto = n;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
            if (lane >= d) upto += v;
        }
        const unsigned here = __ballot_sync(0xFFFFFFFFu, before + upto > item);
        if (here) {
            const int w = __ffs(here) - 1;
            Place r;
            r.q0 = __shfl_sync(0xFFFFFFFFu, q0, w);
            r.ql = __shfl_sync(0xFFFFFFFFu, ql, w);
            r.k0 = __shfl_sync(0xFFFFFFFFu, k0, w);
            r.kl = __shfl_sync(0xFFFFFFFFu, kl, w);
            scan.sequence = s0;
            scan.before = before;
            r.tile = static_cast<int>(item - before) - (__shfl_sync(0xFFFFFFFFu, upto, w) - __shfl_sync(0xFFFFFFFFu, n, w));
            return r;
        }
        before += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    scan.sequence = p.sequences;
    scan.before = before;
    return Place{0, 0, 0, 0, -1};
}
__device__ __forceinline__ Place find_tile(const CatParams &p, long long item, int rows, bool of_keys)
{
    Scan scan;
    return find_tile(p, item, rows, of_keys, scan);
}

// ---------------------------------------------------------------- work items
// A launch has a CTA for every item it could have; those that run take over,
// one by one, the items of CTAs that have not started yet (the hardware hands
// out their numbers in order), so that barriers, tensor memory and the loads of
// the next item are set up while the last one ends.  One warp fetches items and
// finds their tiles ahead of the others, into two slots of shared memory; it asks
// for an item once the loads of the one before have all been issued (sooner, and
// CTAs in long items would keep others' work to themselves).
struct Item {
    int head;
    Place at;
};
struct ItemBars {
    uint32_t full0, empty0, reply_full, go, reply;  // reply: 16 bytes, 16-byte aligned
    volatile int *slots;                        // [2][8]: 1 if there is an item, head, q0, ql, k0, kl, tile
};
constexpr int kItemBytes = 8 * 6 + 16 + 64;  // barriers, reply, slots

// Waits for the next item, or for one to be taken up, last as long as an item does: millions of
// steps of a very long sequence, or a list of a million offsets.  What goes wrong
// inside an item ends these waits too, through the abort flag.
__device__ __forceinline__ Ctl across_items(Ctl ctl)
{
    ctl.limit = 600000000000ull;
    return ctl;
}

__device__ __forceinline__ void run_items(const CatParams &p, const ItemBars &I, Ctl ctl, int rows, bool of_keys, int heads)
{
    const int lane = threadIdx.x & 31;
    long long item = blockIdx.x;
    int n = 0;
    Scan scan;
    const Ctl patient = across_items(ctl);
    for (uint32_t asked = 0;; ++asked) {
        const Place at = find_tile(p, item / heads, rows, of_keys, scan);
        if (at.tile >= 0) {
            if (!wait_bar(I.empty0 + 8u * (n & 1), ((n >> 1) & 1) ^ 1u, patient)) return;
            if (lane == 0) {
                volatile int *v = I.slots + 8 * (n & 1);
                v[0] = 1; v[1] = static_cast<int>(item % heads);
                v[2] = at.q0; v[3] = at.ql; v[4] = at.k0; v[5] = at.kl; v[6] = at.tile;
                mbar_arrive(I.full0 + 8u * (n & 1));
            }
            __syncwarp();
            if (!wait_bar(I.go, n & 1, patient)) return;
            ++n;
        }
        if (lane == 0) {
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(I.reply_full, 16);
            asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(I.reply),
                         "r"(I.reply_full)
                         : "memory");
        }
        __syncwarp();
        if (!wait_bar(I.reply_full, asked & 1u, ctl)) return;
        uint32_t x, more;
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t.reg .b32 y, z;\n\t"
            "ld.shared.b128 r, [%2];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
            "selp.u32 %1, 1, 0, p;\n\t"
            "mov.u32 %0, 0;\n\t"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, _}, r;\n\t}"
            : "=&r"(x), "=&r"(more)
            : "r"(I.reply)
            : "memory");
        __syncwarp();
        if (!more) break;
        item = x;
    }
    if (!wait_bar(I.empty0 + 8u * (n & 1), ((n >> 1) & 1) ^ 1u, patient)) return;
    if (lane == 0) {
        I.slots[8 * (n & 1)] = 0;
        mbar_arrive(I.full0 + 8u * (n & 1));
    }
}

// The n-th item, for one of the warps that work on items; false after the last.
__device__ __forceinline__ bool next_item(const ItemBars &I, Ctl ctl, int n, Item &item)
{
    if (!wait_bar(I.full0 + 8u * (n & 1), (n >> 1) & 1, across_items(ctl))) return false;
    volatile int *v = I.slots + 8 * (n & 1);
    const int some = v[0];
    item.head = v[1];
    item.at = Place{v[2], v[3], v[4], v[5], v[6]};
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(I.empty0 + 8u * (n & 1));
    return some != 0;
}

// Lays out and initialises the barriers at `at` (16-byte aligned); `warps` work on items.
__device__ __forceinline__ ItemBars init_items(uint8_t *generic, uint32_t at, int warps)
{
    const ItemBars I{at, at + 16, at + 32, at + 40, at + 48, reinterpret_cast<volatile int *>(generic + 64)};
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(I.full0 + 8u * s, 1);
            mbar_init(I.empty0 + 8u * s, warps);
        }
        mbar_init(I.reply_full, 1);
        mbar_init(I.go, 1);
    }
    return I;
}

// Key steps [lo, hi) that some query of [i0, i1) sees.
__device__ __forceinline__ void key_steps(const CatParams &p, const Place &at, int i0, int i1, int &lo, int &hi)
{
    const int off = at.kl - at.ql;
    const int end = p.causal ? min(at.kl, i1 + off) : at.kl;
    const int first = p.window ? max(0, i0 + off - p.window + 1) : 0;
    lo = first / CAT_TILE;
    hi = end > first ? (end + CAT_TILE - 1) / CAT_TILE : lo;
}

// Part `part` of `parts` of the steps [lo, hi).
__device__ __forceinline__ void take_part(int &lo, int &hi, int part, int parts)
{
    const int first = lo, n = hi - lo;
    lo = first + static_cast<int>(static_cast<long long>(n) * part / parts);
    hi = first + static_cast<int>(static_cast<long long>(n) * (part + 1) / parts);
}

// ---------------------------------------------------------------- pieces

// Zeroes rows [valid, 128) of a tile (this warp alone), for the async proxy to see.
// What lies behind a sequence's end is another's, and may be NaN: as an operand that
// is summed over its rows it has to be zero.
__device__ __forceinline__ void zero_rows(uint32_t tile, int slices, int valid)
{
    const int lane = threadIdx.x & 31;
    for (int s = 0; s < slices; ++s)
        for (uint32_t at = static_cast<uint32_t>(valid) * 128u + lane * 16u; at < kSliceBytes; at += 512u)
            st_shared_v4(tile + s * kSliceBytes + at, 0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    __syncwarp();
}

__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap &map, uint32_t bar, int slices, int head, int token)
{
    for (int s = 0; s < slices; ++s)
        tma_load_3d(dst + s * kSliceBytes, reinterpret_cast<uint64_t>(&map), bar, 64 * s, head, token);
}

// One lane of a converged warp arrives for it, after all lanes' work on tensor memory.
__device__ __forceinline__ void warp_arrive(uint32_t bar)
{
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Four lanes' four 16-byte pieces transposed: piece i of lane j goes to piece j of lane i.
__device__ __forceinline__ void transpose_pieces(uint32_t (&w)[4][4])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d <= 2; d *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!(i & d)) {
                const bool high = lane & d;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t give = high ? w[i][e] : w[i + d][e];
                    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, give, d);
                    if (high) w[i][e] = got;
                    else w[i + d][e] = got;
                }
            }
}

// Columns [c0, c1) of 32 rows of fp32 sums in tensor memory (both multiples of 8;
// taddr the warp's first column), times the rows' f, to 16-bit values: lane i's
// row at out + i * ld (elements), rows [0, rows) of the warp.  After the exchange
// a store writes 64 bytes of a row.
template <bool BF16>
__device__ __forceinline__ void store_rows(uint32_t taddr, int c0, int c1, float f, uint16_t *out, long long ld, int rows)
{
    const int lane = threadIdx.x & 31;
    for (; c0 < c1; c0 += 32) {
        float v[32];
        tmem_ld_32(taddr + c0, v);
        tmem_wait(v);
        uint32_t w[4][4];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e >> 2][e & 3] = round2<BF16>(v[2 * e] * f, v[2 * e + 1] * f);
        transpose_pieces(w);
        const int col = c0 + 8 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = (lane & ~3) + i;
            if (row < rows && col < c1) *reinterpret_cast<uint4 *>(out + row * ld + col) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
        }
    }
}
// The same, as fp32.
__device__ __forceinline__ void store_rows_f32(uint32_t taddr, int c0, int c1, float f, float *out, long long ld, int rows)
{
    const int lane = threadIdx.x & 31;
    for (; c0 < c1; c0 += 32) {
        float v[32];
        tmem_ld_32(taddr + c0, v);
        tmem_wait(v);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t w[4][4];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e >> 2][e & 3] = __float_as_uint(v[16 * half + e] * f);
            transpose_pieces(w);
            const int col = c0 + 16 * half + 4 * (lane & 3);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = (lane & ~3) + i;
                if (row < rows && col < c1) *reinterpret_cast<uint4 *>(out + row * ld + col) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
            }
        }
    }
}
__device__ __forceinline__ void zero_row(void *out, int c0, int c1)
{
    for (; c0 < c1; c0 += 8) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + c0) = make_uint4(0, 0, 0, 0);
}

}  // namespace cdg
