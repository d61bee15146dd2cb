// Newton-Schulz orthogonalisation for sm_103a: the kernels behind
// cdg_muon_orthogonalize and cdg_muon_step.
//
//   X <- a X + B X,   B = b A + c A^2,   A = X X^T      (X is m x n, m <= n)
//
// Every product runs on the tensor cores with fp16 operands and fp32 sums.
// What fp16 keeps of each is chosen by its effect on the result (relative
// Frobenius error after five steps, 64-bit simulation over Gaussian, low-rank
// and decaying spectra):
//   - X, rounded once to fp16, loses what lies below its largest singular
//     values and the iteration amplifies that (5e-3 on a low-rank U): the
//     linear term a X takes X as a sum of two fp16 parts, the products the
//     high part;
//   - B is dominated by its diagonal: kept in fp32 apart and applied row-wise
//     (1.5e-3 -> 8e-4 on a Gaussian U);
//   - A and the rest of B are rounded once to fp16, times 1024.
// Where that is not enough -- fp32 gradients, and small matrices, whose few
// directions do not average the rounding -- every operand is two fp16 parts
// (22 bits) and a product three: high x high, high x low, low x high.  The
// result then has fp32 accuracy.
// X starts as U times a power of two, exact for fp16 and bf16 gradients; the
// rest of the division by |U|_F goes into the first step's factors.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "muon_params.h"
#include "token_device.cuh"
#include "wait.cuh"

namespace cdg {
namespace {

// MN-major operand in 128-byte-swizzled atoms (64 columns x 8 rows, 1 KB):
// leading offset = bytes between 64-column slices, stride offset = bytes
// between groups of 8 rows along the reduction.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t slice_bytes)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((slice_bytes >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

__device__ __forceinline__ float half_bits(uint16_t v) { return __half2float(__ushort_as_half(v)); }
__device__ __forceinline__ uint16_t to_half_bits(float v) { return __half_as_ushort(__float2half_rn(v)); }

// ---------------------------------------------------------------- norm and first X
// U at element e of matrix b: U itself, or from G and the new momentum.
template <typename T>
__device__ __forceinline__ float update_at(const CmuPrepare &p, long long e)
{
    const float g = Elem<T>::get(static_cast<const T *>(p.u)[e]);
    if (p.nesterov < 0) return g;
    const float m = p.m_out[e];
    return p.nesterov ? fmaf(p.momentum, m, g) : m;
}

template <typename T>
__global__ void __launch_bounds__(256) norm_kernel(const CmuPrepare p)
{
    __shared__ float part[8];
    const long long per = static_cast<long long>(p.rows) * p.cols, base = blockIdx.y * per;
    float s = 0.0f;
    for (long long e = blockIdx.x * 256ll + threadIdx.x; e < per; e += gridDim.x * 256ll) {
        if (p.nesterov >= 0)
            p.m_out[base + e] = fmaf(p.momentum, p.m_in[base + e], Elem<T>::get(static_cast<const T *>(p.u)[base + e]));
        const float u = update_at<T>(p, base + e);
        s = fmaf(u, u, s);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        float t = 0.0f;
        for (int w = 0; w < 8; ++w) t += part[w];
        p.partial[blockIdx.y * CMU_MAX_PARTIALS + blockIdx.x] = t;
    }
}

// X = U 2^k with 2^k |U|_F in [1024, 2048), as a high and a low fp16 part, and
// xs = 2^k (|U|_F + eps): X / xs is the normalised U.
template <typename T>
__global__ void __launch_bounds__(256) split_kernel(const CmuPrepare p)
{
    __shared__ float tile[32][33];
    __shared__ float pw2;
    const int b = blockIdx.z;
    if (threadIdx.x < 32) {
        float s = 0.0f;
        for (int i = threadIdx.x; i < p.partials; i += 32) s += p.partial[b * CMU_MAX_PARTIALS + i];
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (threadIdx.x == 0) {
            const float norm = sqrtf(s);
            const bool finite = norm < INFINITY;
            const int k = norm > 0.0f && finite ? max(-100, min(100, 10 - ilogbf(norm))) : 0;
            const float f = ldexpf(1.0f, k);
            pw2 = finite ? f : NAN;  // an infinity or NaN in U: X is NaN
            if (blockIdx.x == 0 && blockIdx.y == 0) p.xs[b] = f * (norm + p.eps);
        }
    }
    __syncthreads();
    const float f = pw2;
    const int m = p.transposed ? p.cols : p.rows, n = p.transposed ? p.rows : p.cols;
    const long long base = static_cast<long long>(b) * p.rows * p.cols;
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int i0 = blockIdx.y * 32, j0 = blockIdx.x * 32;
    if (p.transposed) {
        for (int r = ty; r < 32; r += 8)
            if (j0 + r < n && i0 + tx < m) tile[tx][r] = update_at<T>(p, base + static_cast<long long>(j0 + r) * p.cols + i0 + tx);
        __syncthreads();
    }
    for (int r = ty; r < 32; r += 8) {
        const int i = i0 + r, j = j0 + tx;
        if (i >= m || j >= n) continue;
        const float u = f * (p.transposed ? tile[r][tx] : update_at<T>(p, base + static_cast<long long>(i) * p.cols + j));
        const long long at = (static_cast<long long>(b) * m + i) * p.pitch_x + j;
        const uint16_t hi = to_half_bits(u);
        p.x_hi[at] = hi;
        if (p.has_lo) p.x_lo[at] = to_half_bits(u - half_bits(hi));
    }
}

// ---------------------------------------------------------------- products
__device__ __forceinline__ void tma_load_3d_to(bool pair, uint32_t dst, const CUtensorMap &map, uint32_t bar, int x, int y,
                                               int z)
{
    if (pair) tma_load_3d_pair(dst, reinterpret_cast<uint64_t>(&map), bar, x, y, z);
    else tma_load_3d(dst, reinterpret_cast<uint64_t>(&map), bar, x, y, z);
}
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t v)
{
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}

// Output tile t: matrix b, tile row tm, tile column tn, blocks [k0, k0 + kn) of
// K.  Symmetric products have only tn <= tm.
struct Tile {
    int b, tm, tn, k0, kn;
    __device__ __forceinline__ Tile(const CmuGemm &p, bool sym, int t)
    {
        b = t / p.tiles;
        const int r = t - b * p.tiles, kblocks = (p.K + CMU_BK - 1) / CMU_BK;
        k0 = 0;
        kn = kblocks;
        if (p.mode == CMU_PARTIAL) {
            tm = tn = 0;
            k0 = static_cast<int>(static_cast<long long>(kblocks) * r / p.tiles);
            kn = static_cast<int>(static_cast<long long>(kblocks) * (r + 1) / p.tiles) - k0;
        } else if (sym) {
            tm = static_cast<int>((sqrtf(8.0f * r + 1.0f) - 1.0f) * 0.5f);
            while ((tm + 1) * (tm + 2) / 2 <= r) ++tm;
            while (tm * (tm + 1) / 2 > r) --tm;
            tn = r - tm * (tm + 1) / 2;
        } else {
            tn = r / p.tiles_m;
            tm = r - tn * p.tiles_m;
        }
    }
};

// Shared memory: the operand ring, the epilogue's staging (a 128 x 64 fp16
// block in 128-byte-swizzled rows, twice, for each group of four warps),
// mbarriers.
template <bool PAIR>
struct Layout {
    static constexpr int kGroups = PAIR ? 2 : 1;             // of epilogue warps, 128 columns each
    static constexpr int kThreads = 128 + 128 * kGroups;
    static constexpr int kTile = PAIR ? 256 : 128;
    static constexpr int kCols = 128 * kGroups;              // TMEM columns an accumulator
    static constexpr int kSmem = 1024 + CMU_STAGES * CMU_STAGE_BYTES + kGroups * CMU_STAGING_BYTES + CMU_BAR_BYTES;
    static_assert(kSmem <= CDG_MAX_DYN_SMEM, "shared memory");
    uint32_t s0, staging, full0, empty0, acc_full0, acc_empty0, drain, epi0;
    __device__ __forceinline__ explicit Layout(uint32_t base)
    {
        s0 = base;
        staging = base + CMU_STAGES * CMU_STAGE_BYTES;
        full0 = staging + kGroups * CMU_STAGING_BYTES;
        empty0 = full0 + 8u * CMU_STAGES;
        acc_full0 = empty0 + 8u * CMU_STAGES;
        acc_empty0 = acc_full0 + 16u;
        drain = acc_empty0 + 16u;
        epi0 = drain + 8u;
    }
    static constexpr int kWords = 8 * (2 * CMU_STAGES + 2 + 2 + 1 + kGroups);  // after the mbarriers
};

// Epilogue of one group of four warps: thread = row of the CTA's 128, 64
// columns at a time.
template <bool PAIR>
struct Epilogue {
    const CmuGemm &p;
    const Layout<PAIR> &L;
    Ctl ctl;
    int group, warp_in_group, lane, row;  // row: of the CTA's 128
    bool elected, sym;
    uint32_t buf0, buf1, bar, phase, sw;

    __device__ __forceinline__ Epilogue(const CmuGemm &p_, const Layout<PAIR> &L_, Ctl c, bool sym_)
        : p(p_), L(L_), ctl(c), sym(sym_)
    {
        const int warp = threadIdx.x / 32 - CDG_EPI_WARP0;
        lane = threadIdx.x % 32;
        group = warp / 4;
        warp_in_group = warp % 4;
        row = warp_in_group * 32 + lane;
        elected = elect_one_sync() && warp_in_group == 0;
        buf0 = L.staging + group * CMU_STAGING_BYTES;
        buf1 = buf0 + CMU_HALF_BYTES;
        bar = L.epi0 + 8u * group;
        phase = 0;
        sw = row & 7;
    }
    __device__ __forceinline__ void sync() const { named_bar_sync(1 + group, 128); }
    // 16-byte piece q (8 columns) of this thread's row in a staging buffer
    __device__ __forceinline__ uint32_t piece(uint32_t buf, int q) const
    {
        return buf + static_cast<uint32_t>(row) * 128u + ((static_cast<uint32_t>(q) ^ sw) << 4);
    }
    // The block of the epilogue's input that a later chunk() needs.
    __device__ __forceinline__ void fetch(int b, int i0, int j0) const
    {
        if (elected) {
            const bool lo = p.mode == CMU_POLY ? p.parts == 3 : p.has_lo != 0;
            bulk_wait_group_read<0>();
            mbar_arrive_expect_tx(bar, lo ? 2 * CMU_HALF_BYTES : CMU_HALF_BYTES);
            tma_load_3d(buf0, reinterpret_cast<uint64_t>(&p.tmE[0]), bar, j0, i0, b);
            if (lo) tma_load_3d(buf1, reinterpret_cast<uint64_t>(&p.tmE[1]), bar, j0, i0, b);
        }
        __syncwarp();
    }
    __device__ __forceinline__ bool fetched()
    {
        const bool ok = wait_bar(bar, phase, ctl);
        phase ^= 1u;
        return !named_bar_red_or(1 + group, 128, !ok);
    }
    // Eight values of the input block: high parts, and low parts where there are any.
    __device__ __forceinline__ void input(int q, bool lo, float (&x)[8]) const
    {
        uint32_t w[4];
        ld_shared_v4(piece(buf0, q), w);
        widen_vec<__half>(make_uint4(w[0], w[1], w[2], w[3]), x);
        if (lo) {
            float y[8];
            ld_shared_v4(piece(buf1, q), w);
            widen_vec<__half>(make_uint4(w[0], w[1], w[2], w[3]), y);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += y[e];
        }
    }
    __device__ __forceinline__ void put(uint32_t buf, int q, const float (&x)[8]) const
    {
        const uint4 w = narrow_vec<__half>(x);
        st_shared_v4(piece(buf, q), w.x, w.y, w.z, w.w);
    }
    __device__ __forceinline__ static void low_part(float (&x)[8])
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] -= __half2float(__float2half_rn(x[e]));
    }

    // v: the sums of columns [j0, j0 + 64) of row i0 + row; j0 < N and i0 < M.
    // False when the launch is giving up.
    __device__ __forceinline__ bool chunk(int b, int i0, int j0, bool mirror, float xs, float (&v)[64])
    {
        const int i = i0 + row;
        if (p.mode == CMU_GRAM) {
            const float f = (CMU_SCALE / xs) / xs;
#pragma unroll
            for (int q = 0; q < 64; ++q) v[q] *= f;
            symmetric(b, i0, j0, mirror, v);
            return true;
        }
        if (!fetched()) return false;
        if (p.mode == CMU_POLY) {
            float d = 0.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                float a[8];
                input(q, p.parts == 3, a);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float &x = v[8 * q + e];
                    x = fmaf(p.b, a[e], p.c * (x * (1.0f / CMU_SCALE)));
                    if (j0 + 8 * q + e == i) {
                        d = x;
                        x = 0.0f;
                    }
                }
            }
            if (i >= j0 && i < j0 + 64 && i < p.M) p.diag[static_cast<long long>(b) * p.M + i] = d * (1.0f / CMU_SCALE);
            symmetric(b, i0, j0, mirror, v);
            return true;
        }
        const float f = 1.0f / xs, g = f / p.poly_scale;
        const float lin = (p.a + (i < p.M ? p.diag[static_cast<long long>(b) * p.M + i] : 0.0f)) * f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float x[8];
            input(q, p.has_lo, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[8 * q + e] = fmaf(lin, x[e], v[8 * q + e] * g);
            if (p.mode == CMU_UPDATE) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = v[8 * q + e] * CMU_SCALE;
                put(buf0, q, x);
                low_part(x);
                put(buf1, q, x);
            }
        }
        if (p.mode == CMU_UPDATE) {
            fence_proxy_async_smem();
            sync();
            if (elected) {
                tma_store_3d(reinterpret_cast<uint64_t>(&p.tmY[0]), buf0, j0, i0, b);
                tma_store_3d(reinterpret_cast<uint64_t>(&p.tmY[1]), buf1, j0, i0, b);
                bulk_commit_group();
            }
        } else {
            result(b, i0, j0, v);
            fence_proxy_async_smem();  // the block has been read: the next fetch may overwrite it
            sync();
        }
        return true;
    }
    // A block of A or B and, off the diagonal, its transpose; high parts, then low parts.
    __device__ __forceinline__ void symmetric(int b, int i0, int j0, bool mirror, float (&v)[64]) const
    {
        for (int part = 0; part < (p.parts == 3 ? 2 : 1); ++part) {
            if (elected) bulk_wait_group_read<0>();
            sync();
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = v[8 * q + e];
                put(buf0, q, x);
                if (mirror) {
                    // column j of this row -> row j, column `row` of two 64-column blocks
                    const uint32_t at = buf1 + static_cast<uint32_t>(row / 64) * 8192u + (row & 7) * 2u;
                    const uint32_t c = (row & 63) >> 3;
#pragma unroll
                    for (int e = 0; e < 8; ++e) st_shared_u16(at + (8 * q + e) * 128u + ((c ^ e) << 4), to_half_bits(x[e]));
                }
                low_part(x);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * q + e] = x[e];
            }
            fence_proxy_async_smem();
            sync();
            if (elected) {
                tma_store_3d(reinterpret_cast<uint64_t>(&p.tmY[part]), buf0, j0, i0, b);
                if (mirror) {
                    tma_store_3d(reinterpret_cast<uint64_t>(&p.tmT[part]), buf1, i0, j0, b);
                    if (i0 + 64 < p.M) tma_store_3d(reinterpret_cast<uint64_t>(&p.tmT[part]), buf1 + 8192u, i0 + 64, j0, b);
                }
                bulk_commit_group();
            }
        }
    }
    __device__ __forceinline__ void write(long long o, float y) const
    {
        if (p.w_in) static_cast<float *>(p.out)[o] = fmaf(p.w_keep, p.w_in[o], -p.w_step * y);
        else if (p.out_type == CDG_T_F32) static_cast<float *>(p.out)[o] = y;
        else if (p.out_type == CDG_T_BF16) static_cast<__nv_bfloat16 *>(p.out)[o] = __float2bfloat16_rn(y);
        else static_cast<__half *>(p.out)[o] = __float2half_rn(y);
    }
    // O or W: lanes along the output's rows either way.
    __device__ __forceinline__ void result(int b, int i0, int j0, const float (&v)[64]) const
    {
        const long long base = static_cast<long long>(b) * p.rows * p.cols;
        const int n = min(64, p.N - j0);
        if (p.transposed) {
            const int i = i0 + row;
            if (i < p.M) {
                const long long at = base + static_cast<long long>(j0) * p.cols + i;
#pragma unroll
                for (int q = 0; q < 64; ++q)
                    if (q < n) write(at + static_cast<long long>(q) * p.cols, v[q]);
            }
            return;
        }
        // through the staging: a warp's 32 rows x 64 columns of fp32, column c of row r at (c + r) % 64
        sync();  // every row's input has been read
        const uint32_t w0 = buf0 + warp_in_group * 8192u;
#pragma unroll
        for (int q = 0; q < 64; ++q) st_shared_f32(w0 + lane * 256u + ((q + lane) & 63) * 4u, v[q]);
        __syncwarp();
        const int r0 = i0 + warp_in_group * 32, rows = min(32, p.M - r0);
        long long at = base + static_cast<long long>(r0) * p.cols + j0 + lane;
        for (int r = 0; r < rows; ++r, at += p.cols) {
            if (lane < n) write(at, ld_shared_f32(w0 + r * 256u + ((lane + r) & 63) * 4u));
            if (lane + 32 < n) write(at + 32, ld_shared_f32(w0 + r * 256u + ((lane + 32 + r) & 63) * 4u));
        }
    }

    // One output tile whose sums are in registers or tensor memory: get(c, v)
    // fills v with 64-column chunk c of this group.
    __device__ __forceinline__ int chunks(int i0, int j0) const { return i0 < p.M ? max(0, min(2, (p.N - j0 + 63) / 64)) : 0; }
};

__device__ __forceinline__ void tmem_ld_64(uint32_t at, float (&v)[64])
{
    uint32_t (&r)[64] = reinterpret_cast<uint32_t(&)[64]>(v);
#pragma unroll
    for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x16(at + 16 * q, *reinterpret_cast<uint32_t(*)[16]>(&r[16 * q]));
    tmem_ld_wait();
}

// Persistent: every CTA (or CTA pair) walks the output tiles.  Warps 0 and 2
// load stages in turn, warp 1 issues the MMAs, warps 4.. run the epilogue,
// which overlaps the next tile's products (two accumulators).  Symmetric
// products compute the tiles on and below the diagonal and store the others as
// their transposes.
//
// One-part products of large matrices run in CTA pairs: 256 x 256 tiles, each
// CTA holding half of the rows of A and of B.  Others take 128 x 128 tiles.
//
// The tensor core rounds every addition to its fp32 sum towards zero, so long
// chains drift (a Gaussian 3000 x 4608 fp32 U: 5e-5 in the result).  Two-part
// products therefore take CMU_CHAIN blocks at a time into one accumulator
// after the other, and the epilogue warps add them up in registers.
template <bool PAIR>
__global__ void __launch_bounds__(Layout<PAIR>::kThreads, 1) gemm_kernel(const __grid_constant__ CmuGemm p)
{
    using Lay = Layout<PAIR>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const Lay L(base);
    uint32_t *slot = reinterpret_cast<uint32_t *>(smem_raw + (L.full0 - raw) + Lay::kWords);
    volatile uint32_t *abort_flag = slot + 1, *used = slot + 2;  // used[stage]: parity of its last load, + 2
    static_assert(Lay::kWords + 8 + 4 * CMU_STAGES <= CMU_BAR_BYTES, "barrier area");
    const bool sym = p.mode <= CMU_POLY || p.mode == CMU_PARTIAL;  // B is K-major, as A
    const int warp = threadIdx.x / 32;
    const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
    const int first = PAIR ? blockIdx.x / 2 : blockIdx.x, step = PAIR ? gridDim.x / 2 : gridDim.x;
    const int total = p.tiles * p.batch;
    const int chain = p.parts > 1 || p.mode == CMU_PARTIAL ? CMU_CHAIN : INT_MAX;
    grid_dep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < CMU_STAGES; ++s) {
            mbar_init(L.full0 + 8u * s, 1);
            mbar_init(L.empty0 + 8u * s, 1);
            used[s] = 0u;
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(L.acc_full0 + 8u * a, 1);
            mbar_init(L.acc_empty0 + 8u * a, PAIR ? 16 : 4);  // one arrival per epilogue warp (of both CTAs)
        }
        mbar_init(L.drain, 1);
        for (int g = 0; g < Lay::kGroups; ++g) mbar_init(L.epi0 + 8u * g, 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    grid_dep_wait();
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(smem_u32(slot), 2 * Lay::kCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(slot), 2 * Lay::kCols);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // both CTAs' barriers exist before anything crosses over
    tc_fence_after();
    const uint32_t tmem = *slot;
    const Ctl ctl{abort_flag, p.status};

    if (warp == 0 || warp == 2) {
        const bool leader = elect_one_sync();
        const uint32_t lead_full0 = PAIR ? mapa_shared(L.full0, 0) : L.full0;
        int s = 0, turn = 0;
        uint32_t parity = 0;
        bool ok = true;
        for (int t = first; ok && t < total; t += step) {
            const Tile tile(p, sym, t);
            const int row0 = tile.tm * Lay::kTile + rank * 128, col0 = tile.tn * Lay::kTile + rank * 128;
            const int blocks = p.parts * tile.kn;
            for (int k = 0; k < blocks; ++k) {
                if (turn == warp) {
                    if (!wait_bar(L.empty0 + 8u * s, parity ^ 1u, ctl)) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        used[s] = parity | 2u;
                        const uint32_t sa = L.s0 + s * CMU_STAGE_BYTES, sb = sa + CMU_HALF_BYTES;
                        const uint32_t bar = lead_full0 + 8u * s;
                        // low x high, high x low, then high x high: the tensor core rounds every
                        // addition towards zero, and the small parts go in while the sum is small
                        const int part = k / tile.kn, k0 = (tile.k0 + k - part * tile.kn) * CMU_BK;
                        const CUtensorMap &ma = p.tmA[p.parts > 1 && part == 0], &mb = p.tmB[p.parts == 3 && part == 1];
                        if (rank == 0) mbar_arrive_expect_tx(L.full0 + 8u * s, (PAIR ? 2 : 1) * CMU_STAGE_BYTES);
                        tma_load_3d_to(PAIR, sa, ma, bar, k0, row0, tile.b);
                        if (sym) {
                            tma_load_3d_to(PAIR, sb, mb, bar, k0, col0, tile.b);
                        } else {
                            tma_load_3d_to(PAIR, sb, mb, bar, col0, k0, tile.b);
                            tma_load_3d_to(PAIR, sb + 8192u, mb, bar, col0 + 64, k0, tile.b);
                        }
                    }
                    __syncwarp();
                }
                turn ^= 2;
                if (++s == CMU_STAGES) {
                    s = 0;
                    parity ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        volatile uint32_t no_abort = 0;
        if (rank == 0) {
            const bool leader = elect_one_sync();
            const uint32_t idesc = (1u << 4) | (sym ? 0u : 1u << 16) | (static_cast<uint32_t>(Lay::kCols >> 3) << 17) |
                                   (static_cast<uint32_t>(Lay::kTile >> 4) << 24);
            int s = 0;
            uint32_t parity = 0, link = 0;
            bool ok = true;
            for (int t = first; ok && t < total; t += step) {
                const int blocks = p.parts * Tile(p, sym, t).kn;
                for (int k = 0, in_chain = 0; k < blocks; ++k) {
                    const uint32_t acc = link & 1u;
                    if ((in_chain == 0 && !wait_bar(L.acc_empty0 + 8u * acc, ((link >> 1) & 1u) ^ 1u, ctl)) ||
                        !wait_bar(L.full0 + 8u * s, parity, ctl)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const bool last = in_chain == chain - 1 || k == blocks - 1;
                    if (leader) {
                        const uint32_t sa = L.s0 + s * CMU_STAGE_BYTES, sb = sa + CMU_HALF_BYTES;
                        const uint64_t ad = sdesc_k128_sw128(sa);
                        const uint64_t bd = sym ? sdesc_k128_sw128(sb) : desc_mn_sw128(sb, 8192);
                        const uint32_t bstep = sym ? 2u : 128u, d = tmem + acc * Lay::kCols;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (PAIR) umma_f16_pair(d, ad + 2u * q, bd + bstep * q, idesc, (in_chain | q) != 0);
                            else umma_f16(d, ad + 2u * q, bd + bstep * q, idesc, (in_chain | q) != 0);
                        }
                        if (PAIR) {
                            umma_commit_pair(L.empty0 + 8u * s);
                            if (last) umma_commit_pair(L.acc_full0 + 8u * acc);
                        } else {
                            umma_commit(L.empty0 + 8u * s);
                            if (last) umma_commit(L.acc_full0 + 8u * acc);
                        }
                    }
                    __syncwarp();
                    ++in_chain;
                    if (last) {
                        in_chain = 0;
                        ++link;
                    }
                    if (++s == CMU_STAGES) {
                        s = 0;
                        parity ^= 1u;
                    }
                }
            }
            if (leader) {
                if (PAIR) umma_commit_pair(L.drain);
                else umma_commit(L.drain);
            }
            __syncwarp();
        }
        // tensor memory is freed only after the MMAs in flight
        wait_bar(L.drain, 0, Ctl{&no_abort, p.status});
    } else if (warp >= CDG_EPI_WARP0) {
        Epilogue<PAIR> e(p, L, ctl, sym);
        const uint32_t lane_base = static_cast<uint32_t>(e.warp_in_group * 32) << 16;
        uint32_t link = 0;
        bool ok = true;
        auto hand_back = [&](uint32_t acc) {
            tc_fence_before();
            __syncwarp();
            if (e.lane == 0) {
                if (PAIR && rank != 0) mbar_arrive_cluster(mapa_shared(L.acc_empty0 + 8u * acc, 0));
                else mbar_arrive(L.acc_empty0 + 8u * acc);
            }
        };
        for (int t = first; ok && t < total; t += step) {
            const Tile tile(p, sym, t);
            const int i0 = tile.tm * Lay::kTile + rank * 128, j0 = tile.tn * Lay::kTile + e.group * 128;
            const int n = e.chunks(i0, j0);
            const bool mirror = sym && tile.tn < tile.tm;
            const float xs = p.first ? p.xs[tile.b] : CMU_SCALE;
            const bool fetches = p.mode != CMU_GRAM && p.mode != CMU_PARTIAL;
            if (n > 0 && fetches) e.fetch(tile.b, i0, j0);
            if constexpr (PAIR) {
                const uint32_t acc = link & 1u;
                ok = wait_bar(L.acc_full0 + 8u * acc, (link >> 1) & 1u, ctl);
                if (named_bar_red_or(1 + e.group, 128, !ok)) break;
                ++link;
                tc_fence_after();
                for (int c = 0; c < n; ++c) {
                    float v[64];
                    tmem_ld_64(tmem + acc * Lay::kCols + e.group * 128 + c * 64 + lane_base, v);
                    if (c == n - 1) hand_back(acc);
                    if (!(ok = e.chunk(tile.b, i0, j0 + 64 * c, mirror, xs, v))) break;
                    if (c + 1 < n && fetches) e.fetch(tile.b, i0, j0 + 64 * (c + 1));
                }
                if (n == 0) hand_back(acc);
            } else {
                float sum[2][64];
                const int links = (p.parts * tile.kn - 1) / chain + 1;
                for (int k = 0; ok && k < links; ++k, ++link) {
                    const uint32_t acc = link & 1u;
                    ok = __all_sync(0xFFFFFFFFu, wait_bar(L.acc_full0 + 8u * acc, (link >> 1) & 1u, ctl));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint32_t r[16];
                        tmem_ld_32x32b_x16(tmem + acc * Lay::kCols + c * 16 + lane_base, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            float &x = sum[c / 4][c % 4 * 16 + q];
                            x = k ? x + __uint_as_float(r[q]) : __uint_as_float(r[q]);
                        }
                    }
                    hand_back(acc);
                }
                if (named_bar_red_or(1, 128, !ok)) break;
                if (p.mode == CMU_PARTIAL) {
                    // rows and columns below M, 16 bytes at a time (pads up to a multiple of 4 are sums of zeros)
                    float *out = p.partial + static_cast<long long>(t) * (CMU_SIDE * CMU_SIDE) + e.row * CMU_SIDE;
                    if (e.row < p.M)
#pragma unroll
                        for (int q = 0; q < 128; q += 4)
                            if (q < p.N)
                                *reinterpret_cast<float4 *>(out + q) =
                                    make_float4(sum[q / 64][q % 64], sum[q / 64][q % 64 + 1], sum[q / 64][q % 64 + 2],
                                                sum[q / 64][q % 64 + 3]);
                    __syncwarp();
                    continue;
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (c >= n) break;
                    if (!(ok = e.chunk(tile.b, i0, j0 + 64 * c, mirror, xs, sum[c]))) break;
                    if (c + 1 < n && fetches) e.fetch(tile.b, i0, j0 + 64 * (c + 1));
                }
            }
        }
        if (e.elected) bulk_wait_group_all();
    }

    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) {
        // copies in flight land before the CTA exits
        volatile uint32_t no_abort = 0;
        const Ctl drain{&no_abort, p.status};
        if (rank == 0) {
            for (int s = 0; s < CMU_STAGES; ++s)
                if (used[s] & 2u) wait_bar(L.full0 + 8u * s, used[s] & 1u, drain);
        }
        const uint64_t t0 = global_timer_ns();  // the peer's barrier, and the epilogue's blocks
        while (global_timer_ns() - t0 < 200000ull) {
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // neither CTA leaves while the other may still signal it
    if (warp == 1) {
        tc_fence_after();
        if (PAIR) tmem_dealloc_pair(tmem, 2 * Lay::kCols);
        else tmem_dealloc(tmem, 2 * Lay::kCols);
    }
}

template <bool PAIR>
cudaError_t launch_gemm(CmuGemm p, int sms, cudaStream_t s)
{
    using Lay = Layout<PAIR>;
    p.tiles_m = (p.M + Lay::kTile - 1) / Lay::kTile;
    const int tiles_n = (p.N + Lay::kTile - 1) / Lay::kTile;
    if (p.mode != CMU_PARTIAL)
        p.tiles = p.mode <= CMU_POLY ? p.tiles_m * (p.tiles_m + 1) / 2 : p.tiles_m * tiles_n;
    const long long total = static_cast<long long>(p.tiles) * p.batch;
    if (total > INT_MAX / 2) return cudaErrorInvalidConfiguration;
    const int width = PAIR ? 2 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(width * std::min<long long>(total, std::max(1, sms / width))));
    cfg.blockDim = dim3(Lay::kThreads);
    cfg.dynamicSmemBytes = Lay::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = width;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, gemm_kernel<PAIR>, p);
}

// ---------------------------------------------------------------- small matrices
// Up to 128 rows, the iteration runs on the m x m Gram matrix alone, one CTA a
// matrix, every operand in shared memory:
//
//   A = X X^T;  steps times:  Q = a I + b A + c A^2,  P <- Q P,  A <- Q A Q
//
// (all polynomials of A: symmetric, and they commute), and the result is P X,
// one more product.  Against the three products a step over all of X this is
// 14 dependent products of 128 x 128 instead of 15 launches.  Operands are two
// fp16 parts (22 bits): a small singular value s enters A as s^2, and the
// factor P on it, up to a^steps = 485, comes out within 1e-4 to 1e-3 of the
// iteration on X (64-bit simulation; spectra over four decades).
//
// 256 threads: thread t holds row t % 128, columns 64 (t / 128) .. + 63 of the
// accumulators.
constexpr int kItThreads = 256;
constexpr uint32_t kMatBytes = 4 * CMU_HALF_BYTES;  // high parts of columns 0-63, 64-127; then low parts
constexpr int kItSmem = 1024 + 3 * static_cast<int>(kMatBytes) + 256;

__global__ void __launch_bounds__(kItThreads, 1) iterate_kernel(const CmuIterate p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t mA = base, mQ = base + kMatBytes, mP = base + 2 * kMatBytes, bar0 = base + 3 * kMatBytes;
    uint32_t *slot = reinterpret_cast<uint32_t *>(smem_raw + (bar0 - raw) + 16);
    volatile uint32_t *abort_flag = slot + 1;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int row = tid % 128, half = tid / 128, b = blockIdx.x;
    grid_dep_launch_dependents();
    if (tid == 0) {
        mbar_init(bar0, 1);
        mbar_init(bar0 + 8, 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    grid_dep_wait();
    if (warp == 0) {
        tmem_alloc(smem_u32(slot), 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    const Ctl ctl{abort_flag, p.status};
    const bool leader = warp == 0 && elect_one_sync();
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;

    // the ranges' partial sums, in order, to A = sum / xs^2 (fp32, in Q's and P's place)
    {
        const float f = (1.0f / p.xs[b]) / p.xs[b];
        const float *src = p.partial + static_cast<long long>(b) * p.splits * (CMU_SIDE * CMU_SIDE);
        const int n4 = (p.m + 3) / 4;
        for (int x = tid; x < p.m * n4; x += kItThreads) {
            const int r = x / n4, c = x - r * n4;
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int k = 0; k < p.splits; ++k) {
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + static_cast<long long>(k) * (CMU_SIDE * CMU_SIDE) +
                                                                         r * CMU_SIDE) + c);
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            }
            st_shared_v4(mQ + r * 512u + ((static_cast<uint32_t>(c) ^ (r & 31)) << 4), __float_as_uint(s.x * f),
                         __float_as_uint(s.y * f), __float_as_uint(s.z * f), __float_as_uint(s.w * f));
        }
        __syncthreads();
    }

    // piece q (8 columns) of this thread's row half in matrix `mat`, part 0 or 1
    auto piece = [&](uint32_t mat, int part, int q) {
        return mat + static_cast<uint32_t>(2 * part + half) * CMU_HALF_BYTES + static_cast<uint32_t>(row) * 128u +
               ((static_cast<uint32_t>(q) ^ (row & 7)) << 4);
    };
    auto put = [&](uint32_t mat, int q, const float (&x)[8]) {
        uint4 w = narrow_vec<__half>(x);
        st_shared_v4(piece(mat, 0, q), w.x, w.y, w.z, w.w);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e] - __half2float(__float2half_rn(x[e]));
        w = narrow_vec<__half>(y);
        st_shared_v4(piece(mat, 1, q), w.x, w.y, w.z, w.w);
    };
    auto get = [&](uint32_t mat, int q, float (&x)[8]) {
        uint32_t w[4];
        float y[8];
        ld_shared_v4(piece(mat, 0, q), w);
        widen_vec<__half>(make_uint4(w[0], w[1], w[2], w[3]), x);
        ld_shared_v4(piece(mat, 1, q), w);
        widen_vec<__half>(make_uint4(w[0], w[1], w[2], w[3]), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += y[e];
    };
    // accumulator d <- X Y: low x high, high x low, high x high
    const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(128 >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
    auto multiply = [&](uint32_t d, uint32_t x, uint32_t y) {
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint64_t ad = sdesc_k128_sw128(x + (2u * (part == 0) + s) * CMU_HALF_BYTES);
                const uint64_t bd = sdesc_k128_sw128(y + (2u * (part == 1) + s) * CMU_HALF_BYTES);
#pragma unroll
                for (int q = 0; q < 4; ++q) umma_f16(tmem + 128 * d, ad + 2u * q, bd + 2u * q, idesc, (part | s | q) != 0);
            }
        umma_commit(bar0 + 8 * d);
    };
    // everything written to shared memory is seen by the products issued next
    auto ready = [&]() {
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };
    uint32_t phase[2] = {0u, 0u};
    auto wait = [&](int d) {
        const bool ok = wait_bar(bar0 + 8u * d, phase[d], ctl);
        phase[d] ^= 1u;
        tc_fence_after();
        return __syncthreads_and(ok) != 0;
    };
    auto load = [&](int d, int q, float (&v)[16]) {  // 16 columns of accumulator d
        uint32_t(&r)[16] = reinterpret_cast<uint32_t(&)[16]>(v);
        tmem_ld_32x32b_x16(tmem + 128 * d + half * 64 + 16 * q + lane_base, r);
        tmem_ld_wait();
    };

    // A to its two parts
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        float x[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t c = half * 16u + 2u * q + h;
            uint32_t w[4] = {0u, 0u, 0u, 0u};
            if (row < p.m && static_cast<int>(4 * c) < p.m) ld_shared_v4(mQ + row * 512u + ((c ^ (row & 31)) << 4), w);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * h + e] = CMU_SCALE * __uint_as_float(w[e]);
        }
        put(mA, q, x);
    }
    ready();
    constexpr float kInv = 1.0f / CMU_SCALE;
    bool ok = true;
    for (int k = 0; k < p.steps; ++k) {
        // Q = a I + b A + c A A
        if (leader) multiply(0, mA, mA);
        __syncwarp();
        if (!(ok = wait(0))) break;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v[16];
            load(0, q, v);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x[8];
                get(mA, 2 * q + h, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = fmaf(p.b, x[e], p.c * (v[8 * h + e] * kInv));
                    if (half * 64 + 16 * q + 8 * h + e == row) x[e] += p.a * CMU_SCALE;
                }
                put(mQ, 2 * q + h, x);
                if (k == 0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] *= CMU_POLY_SCALE * kInv;
                    put(mP, 2 * q + h, x);
                }
            }
        }
        ready();
        const bool last = k == p.steps - 1;
        if (leader) {
            if (!last) multiply(0, mQ, mA);
            if (k > 0) multiply(1, mQ, mP);
        }
        __syncwarp();
        if (!last) {  // T = Q A, in A's place
            if (!(ok = wait(0))) break;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[16];
                load(0, q, v);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = v[8 * h + e] * kInv;
                    put(mA, 2 * q + h, x);
                }
            }
            ready();
            if (leader) multiply(0, mA, mQ);  // A <- T Q
            __syncwarp();
        }
        if (k > 0) {  // P <- Q P
            if (!(ok = wait(1))) break;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[16];
                load(1, q, v);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = v[8 * h + e] * kInv;
                    put(mP, 2 * q + h, x);
                }
            }
        }
        if (!last) {
            if (!(ok = wait(0))) break;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[16];
                load(0, q, v);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = v[8 * h + e] * kInv;
                    put(mA, 2 * q + h, x);
                }
            }
            ready();
        }
    }
    // P without its diagonal, and the diagonal
    if (ok && row < p.m) {
        const long long at = (static_cast<long long>(b) * p.m + row) * p.pitch_a + half * 64;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int j = half * 64 + 8 * q;
            if (j >= p.m) break;
            float x[8], y[8];
            get(mP, q, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (j + e == row) {
                    p.diag[static_cast<long long>(b) * p.m + row] = x[e] * (1.0f / CMU_POLY_SCALE);
                    x[e] = 0.0f;
                }
                y[e] = x[e] - __half2float(__float2half_rn(x[e]));
            }
            *reinterpret_cast<uint4 *>(p.poly + at + 8 * q) = narrow_vec<__half>(x);
            *reinterpret_cast<uint4 *>(p.poly_lo + at + 8 * q) = narrow_vec<__half>(y);
        }
    }
    if (!ok) {  // giving up: what is in flight ends before tensor memory is freed
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 200000ull) {
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

template <typename T>
void launch_norm(const CmuPrepare &p, cudaStream_t s)
{
    norm_kernel<T><<<dim3(p.partials, p.batch), 256, 0, s>>>(p);
}
template <typename T>
void launch_split(const CmuPrepare &p, cudaStream_t s)
{
    const int m = p.transposed ? p.cols : p.rows, n = p.transposed ? p.rows : p.cols;
    split_kernel<T><<<dim3((n + 31) / 32, (m + 31) / 32, p.batch), 256, 0, s>>>(p);
}

}  // namespace
}  // namespace cdg

cudaError_t cmu_prepare_kernels()
{
    const cudaError_t e = cudaFuncSetAttribute(cdg::gemm_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               cdg::Layout<false>::kSmem);
    if (e != cudaSuccess) return e;
    const cudaError_t i = cudaFuncSetAttribute(cdg::iterate_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, cdg::kItSmem);
    return i != cudaSuccess ? i
                            : cudaFuncSetAttribute(cdg::gemm_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   cdg::Layout<true>::kSmem);
}

cudaError_t cmu_launch_norm(const CmuPrepare &p, cudaStream_t s)
{
    if (p.dtype == CDG_F32) cdg::launch_norm<float>(p, s);
    else if (p.dtype == CDG_F16) cdg::launch_norm<__half>(p, s);
    else cdg::launch_norm<__nv_bfloat16>(p, s);
    return cudaGetLastError();
}

cudaError_t cmu_launch_split(const CmuPrepare &p, cudaStream_t s)
{
    if (p.dtype == CDG_F32) cdg::launch_split<float>(p, s);
    else if (p.dtype == CDG_F16) cdg::launch_split<__half>(p, s);
    else cdg::launch_split<__nv_bfloat16>(p, s);
    return cudaGetLastError();
}

cudaError_t cmu_launch_iterate(const CmuIterate &p, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.batch));
    cfg.blockDim = dim3(cdg::kItThreads);
    cfg.dynamicSmemBytes = cdg::kItSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cdg::iterate_kernel, p);
}

cudaError_t cmu_launch_gemm(const CmuGemm &p, int sms, cudaStream_t s)
{
    return p.pair ? cdg::launch_gemm<true>(p, sms, s) : cdg::launch_gemm<false>(p, sms, s);
}
