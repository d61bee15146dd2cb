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
// That is 1e-4 to 1e-3 off, and up to 1.8e-3 where all singular values are equal
// (512 x 512).  Where it is not enough -- fp32 gradients, and small matrices,
// whose few directions do not average the rounding -- every operand is two fp16
// parts (22 bits) and a product three: high x high, high x low, low x high.  The
// result then has fp32 accuracy (2e-7 to 8e-6), at 1.6 to 4.5 times the time of
// 16-bit updates (512 x 4608: 280 us against 171; 4096 x 4096: 4.7 ms against
// 1.06).
// X starts as U times a power of two, exact for fp16 and bf16 gradients; the
// rest of the division by |U|_F goes into the first step's factors.
//
// What bounds it.  Large matrices: the tensor cores; 4096 x 4096 takes 1.06 ms of
// which the products without their mirrored halves need 0.71 at cuBLAS's rate
// (136 of 152 tiles' worth of pairs busy in a symmetric product's two waves, 630
// cycles a block of K against 512 of tensor work).  Middle ones: what a launch
// costs beyond its products, about 4 us (start, first load, epilogue, end), and
// the 64 bytes a cycle an SM loads (512 cycles a block of a 128 x 128 tile):
// 512 x 4608 171 us.  Small ones: five launches, each of which reads from L2 what
// the one before it wrote (three 64 x 576: 37.5 us; the chain of 14 dependent
// products in one of them is about 13, and that launch 23.5 of the five's 55
// when each starts cold).
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

__device__ __forceinline__ uint16_t to_half_bits(float v) { return __half_as_ushort(__float2half_rn(v)); }

// ---------------------------------------------------------------- norm and first X
// Eight consecutive values of U, from element e (a multiple of 8): U itself,
// or from G and the momentum.  FIRST: the momentum is updated on the way.
template <typename T, bool FIRST>
__device__ __forceinline__ void update_8(const CmuPrepare &p, long long e, float (&u)[8])
{
    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.u) + e);
    if constexpr (sizeof(T) == 4) {
        float lo[4], hi[4];
        widen_vec<T>(src[0], lo);
        widen_vec<T>(src[1], hi);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            u[q] = lo[q];
            u[4 + q] = hi[q];
        }
    } else {
        widen_vec<T>(src[0], u);
    }
    if (p.nesterov < 0) return;
    float m[8];
    const float4 *mi = reinterpret_cast<const float4 *>((FIRST ? p.m_in : p.m_out) + e);
    float4 *mo = reinterpret_cast<float4 *>(p.m_out + e);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float4 v = mi[h];
        if (FIRST) {
            v = make_float4(fmaf(p.momentum, v.x, u[4 * h]), fmaf(p.momentum, v.y, u[4 * h + 1]),
                            fmaf(p.momentum, v.z, u[4 * h + 2]), fmaf(p.momentum, v.w, u[4 * h + 3]));
            mo[h] = v;
        }
        m[4 * h] = v.x;
        m[4 * h + 1] = v.y;
        m[4 * h + 2] = v.z;
        m[4 * h + 3] = v.w;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) u[q] = p.nesterov ? fmaf(p.momentum, m[q], u[q]) : m[q];
}
template <typename T, bool FIRST>
__device__ __forceinline__ float update_1(const CmuPrepare &p, long long e)
{
    const float g = Elem<T>::get(static_cast<const T *>(p.u)[e]);
    if (p.nesterov < 0) return g;
    float m = (FIRST ? p.m_in : p.m_out)[e];
    if (FIRST) p.m_out[e] = m = fmaf(p.momentum, m, g);
    return p.nesterov ? fmaf(p.momentum, m, g) : m;
}

constexpr int kPrepareThreads = 256;

// The momentum, and partial sums of squares of U.  A matrix's elements in
// groups of eight from a multiple of eight, single ones at its ends.
template <typename T>
__global__ void __launch_bounds__(kPrepareThreads) norm_kernel(const CmuPrepare p)
{
    __shared__ float part[kPrepareThreads / 32];
    const long long per = static_cast<long long>(p.rows) * p.cols, a = blockIdx.y * per, b = a + per;
    const long long a8 = min((a + 7) / 8 * 8, b), b8 = max(a8, b / 8 * 8);
    grid_dep_launch_dependents();
    grid_dep_wait();
    float s = 0.0f;
    const long long first = blockIdx.x * static_cast<long long>(kPrepareThreads) + threadIdx.x;
#pragma unroll 2
    for (long long g = a8 / 8 + first; g < b8 / 8; g += static_cast<long long>(gridDim.x) * kPrepareThreads) {
        float u[8];
        update_8<T, true>(p, 8 * g, u);
#pragma unroll
        for (int q = 0; q < 8; ++q) s = fmaf(u[q], u[q], s);
    }
    if (first < a8 - a) {
        const float u = update_1<T, true>(p, a + first);
        s = fmaf(u, u, s);
    } else if (first >= 8 && first - 8 < b - b8) {
        const float u = update_1<T, true>(p, b8 + first - 8);
        s = fmaf(u, u, s);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        float t = 0.0f;
        for (int w = 0; w < kPrepareThreads / 32; ++w) t += part[w];
        p.partial[blockIdx.y * CMU_MAX_PARTIALS + blockIdx.x] = t;
    }
}

// X = U 2^k with 2^k |U|_F in [1024, 2048), as a high and a low fp16 part, and
// xs = 2^k (|U|_F + eps): X / xs is the normalised U.  The factor 2^k of matrix
// b, by every CTA.
__device__ __forceinline__ float first_scale(const CmuPrepare &p, int b, bool write)
{
    __shared__ float pw2;
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
            // (a zero X: any divisor that has a finite square, which a small eps has not)
            if (write) p.xs[b] = norm == 0.0f ? 1.0f : f * (norm + p.eps);
        }
    }
    __syncthreads();
    return pw2;
}

__device__ __forceinline__ void put_parts(const CmuPrepare &p, long long at, const float (&x)[8])
{
    *reinterpret_cast<uint4 *>(p.x_hi + at) = narrow_vec<__half>(x);
    if (p.has_lo) {
        float y[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) y[q] = x[q] - __half2float(__float2half_rn(x[q]));
        *reinterpret_cast<uint4 *>(p.x_lo + at) = narrow_vec<__half>(y);
    }
}

// Rows of a multiple of eight columns, not transposed: X has U's layout.
template <typename T>
__global__ void __launch_bounds__(kPrepareThreads) split_flat_kernel(const CmuPrepare p)
{
    grid_dep_launch_dependents();
    grid_dep_wait();
    const long long groups = static_cast<long long>(p.rows) * p.cols / 8;
    const float f = first_scale(p, blockIdx.y, blockIdx.x == 0);
#pragma unroll 2
    for (long long g = blockIdx.x * static_cast<long long>(kPrepareThreads) + threadIdx.x; g < groups;
         g += static_cast<long long>(gridDim.x) * kPrepareThreads) {
        const long long e = 8 * (blockIdx.y * groups + g);
        float u[8];
        update_8<T, false>(p, e, u);
#pragma unroll
        for (int q = 0; q < 8; ++q) u[q] *= f;
        put_parts(p, e, u);
    }
}

// Any other shape: 64 x 64 blocks of X through shared memory, read along U's
// rows and written eight columns at a time (the pitch is a multiple of eight).
template <typename T>
__global__ void __launch_bounds__(kPrepareThreads) split_kernel(const CmuPrepare p)
{
    __shared__ float tile[64][65];
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int b = blockIdx.z, tid = threadIdx.x;
    const float f = first_scale(p, b, blockIdx.x == 0 && blockIdx.y == 0);
    const int m = p.transposed ? p.cols : p.rows, n = p.transposed ? p.rows : p.cols;
    const long long base = static_cast<long long>(b) * p.rows * p.cols;
    const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
    const int x = tid % 64, y = tid / 64;  // x along U's rows
    const int u_row0 = p.transposed ? j0 : i0, u_col = (p.transposed ? i0 : j0) + x;
#pragma unroll 8
    for (int r = y; r < 64; r += kPrepareThreads / 64) {
        const float v = u_row0 + r < p.rows && u_col < p.cols
                            ? f * update_1<T, false>(p, base + static_cast<long long>(u_row0 + r) * p.cols + u_col)
                            : 0.0f;
        if (p.transposed) tile[x][r] = v;
        else tile[r][x] = v;
    }
    __syncthreads();
#pragma unroll
    for (int g = tid; g < 64 * 8; g += kPrepareThreads) {
        const int i = i0 + g / 8, j = j0 + g % 8 * 8;
        if (i >= m || j >= n) continue;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = tile[g / 8][g % 8 * 8 + q];
        put_parts(p, (static_cast<long long>(b) * m + i) * p.pitch_x + j, v);
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
// All threads of the cluster; shared memory written before arriving is seen after waiting.
__device__ __forceinline__ void cluster_barrier_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_barrier_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t v)
{
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}

// Output tile t: matrix b, tile row tm, tile column tn, blocks [k0, k0 + kn) of
// K.  Symmetric products have only the tiles that reach the diagonal or lie
// below it; `mirror`: wholly below it.
template <int FORM>
struct Tile {
    int b, tm, tn, k0, kn;
    bool mirror;
    __device__ __forceinline__ Tile(const CmuGemm &p, bool sym, int t, int rank)
    {
        b = t / p.tiles;
        const int r = t - b * p.tiles, kblocks = (p.K + CMU_BK - 1) / CMU_BK;
        int part = 0, parts = 1;
        mirror = false;
        if (p.mode == CMU_PARTIAL) {
            tm = tn = 0;
            part = r;
            parts = p.tiles;
        } else if (sym) {
            // tile rows before tm hold tm (tm + 1) / 2 square tiles, or twice as many narrow ones
            const int h = FORM == CMU_NARROW ? r / 2 : r;
            tm = static_cast<int>((sqrtf(8.0f * h + 1.0f) - 1.0f) * 0.5f);
            while ((tm + 1) * (tm + 2) / 2 <= h) ++tm;
            while (tm * (tm + 1) / 2 > h) --tm;
            tn = r - (FORM == CMU_NARROW ? 2 : 1) * (tm * (tm + 1) / 2);
            mirror = (FORM == CMU_NARROW ? tn / 2 : tn) < tm;
        } else {
            tn = r / p.tiles_m;
            tm = r - tn * p.tiles_m;
        }
        if (FORM == CMU_NARROW) {
            part = rank;
            parts = p.split;
        }
        k0 = static_cast<int>(static_cast<long long>(kblocks) * part / parts);
        kn = static_cast<int>(static_cast<long long>(kblocks) * (part + 1) / parts) - k0;
    }
};

// Shared memory: the operand ring, the epilogue's staging (a 128 x 64 fp16
// block in 128-byte-swizzled rows, twice, for each group of eight warps),
// mbarriers.
template <int FORM>
struct Layout {
    static constexpr bool kPair = FORM == CMU_PAIR;
    // Groups of eight epilogue warps, a 64-column chunk at a time, for every 128 columns of the tile.
    static constexpr int kGroups = kPair ? 2 : 1;
    static constexpr int kGroupThreads = 256, kThreads = 128 + kGroups * kGroupThreads;
    static constexpr int kOwn = 64 * 128 / kGroupThreads;    // columns of a chunk a thread holds
    static constexpr int kTileM = kPair ? 256 : 128, kTileN = kPair ? 256 : FORM == CMU_SQUARE ? 128 : 64;
    static constexpr int kCols = kTileN;                     // TMEM columns an accumulator
    static constexpr uint32_t kBBytes = FORM == CMU_NARROW ? CMU_HALF_BYTES / 2 : CMU_HALF_BYTES;
    static constexpr uint32_t kStage = CMU_HALF_BYTES + kBBytes;
    static constexpr int kSmem = 1024 + CMU_STAGES * static_cast<int>(kStage) + kGroups * CMU_STAGING_BYTES + CMU_BAR_BYTES;
    static_assert(kSmem <= CDG_MAX_DYN_SMEM, "shared memory");
    uint32_t s0, staging, full0, empty0, acc_full0, acc_empty0, drain, epi0;
    __device__ __forceinline__ explicit Layout(uint32_t base)
    {
        s0 = base;
        staging = base + CMU_STAGES * kStage;
        full0 = staging + kGroups * CMU_STAGING_BYTES;
        empty0 = full0 + 8u * CMU_STAGES;
        acc_full0 = empty0 + 8u * CMU_STAGES;
        acc_empty0 = acc_full0 + 16u;
        drain = acc_empty0 + 16u;
        epi0 = drain + 8u;
    }
    static constexpr int kWords = 8 * (2 * CMU_STAGES + 2 + 2 + 1 + kGroups);  // after the mbarriers
};

// Epilogue of one group of warps: a thread holds kOwn columns of one of the
// CTA's 128 rows, of 64 columns at a time.
template <int FORM>
struct Epilogue {
    using Lay = Layout<FORM>;
    static constexpr int OWN = Lay::kOwn, PIECES = OWN / 8;
    const CmuGemm &p;
    const Lay &L;
    Ctl ctl;
    int group, quad, part, lane, row;  // row: of the CTA's 128; part: which of its columns in a chunk
    bool elected, sym;
    uint32_t buf0, buf1, bar, phase, sw;

    __device__ __forceinline__ Epilogue(const CmuGemm &p_, const Lay &L_, Ctl c, bool sym_) : p(p_), L(L_), ctl(c), sym(sym_)
    {
        const int warp = threadIdx.x / 32 - CDG_EPI_WARP0;
        lane = threadIdx.x % 32;
        group = warp / 8;
        part = warp % 8 / 4;
        quad = warp % 4;
        row = quad * 32 + lane;
        elected = elect_one_sync() && quad == 0 && part == 0;
        buf0 = L.staging + group * CMU_STAGING_BYTES;
        buf1 = buf0 + CMU_HALF_BYTES;
        bar = L.epi0 + 8u * group;
        phase = 0;
        sw = row & 7;
    }
    __device__ __forceinline__ void sync() const { named_bar_sync(1 + group, Lay::kGroupThreads); }
    __device__ __forceinline__ bool any(bool x) const { return named_bar_red_or(1 + group, Lay::kGroupThreads, x); }
    // this thread's q-th 16-byte piece (8 columns) of its row in a staging buffer
    __device__ __forceinline__ uint32_t piece(uint32_t buf, int q) const
    {
        return buf + static_cast<uint32_t>(row) * 128u + ((static_cast<uint32_t>(part * PIECES + q) ^ sw) << 4);
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
        return !any(!ok);
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
    // Eight values rounded to fp16 into a staging buffer; x becomes what the rounding left.
    __device__ __forceinline__ void put(uint32_t buf, int q, float (&x)[8]) const
    {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __half2 h = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
            const float2 f = __half22float2(h);
            w[e] = *reinterpret_cast<const uint32_t *>(&h);
            x[2 * e] -= f.x;
            x[2 * e + 1] -= f.y;
        }
        st_shared_v4(piece(buf, q), w[0], w[1], w[2], w[3]);
    }

    // v: this thread's sums of the chunk of columns [j0, j0 + 64), row i0 + row;
    // j0 < N and i0 < M.  False when the launch is giving up.
    __device__ __forceinline__ bool chunk(int b, int i0, int j0, bool mirror, float xs, float (&v)[OWN])
    {
        const int i = i0 + row, mine = j0 + part * OWN;  // this thread's first column
        if (p.mode == CMU_GRAM) {
            const float f = (CMU_SCALE / xs) / xs;
#pragma unroll
            for (int q = 0; q < OWN; ++q) v[q] *= f;
            symmetric(b, i0, j0, mirror, v);
            return true;
        }
        if (!fetched()) return false;
        if (p.mode == CMU_POLY) {
            const float g = p.c * (1.0f / CMU_SCALE);
#pragma unroll
            for (int q = 0; q < PIECES; ++q) {
                float a[8];
                input(q, p.parts == 3, a);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * q + e] = fmaf(p.b, a[e], g * v[8 * q + e]);
            }
            if (i >= mine && i < mine + OWN && i < p.M) {  // the diagonal, apart
                float d = 0.0f;
#pragma unroll
                for (int q = 0; q < OWN; ++q)
                    if (mine + q == i) {
                        d = v[q];
                        v[q] = 0.0f;
                    }
                p.diag[static_cast<long long>(b) * p.M + i] = d * (1.0f / CMU_SCALE);
            }
            symmetric(b, i0, j0, mirror, v);
            return true;
        }
        const float f = 1.0f / xs, g = f / p.poly_scale;
        const float lin = (p.a + (i < p.M ? p.diag[static_cast<long long>(b) * p.M + i] : 0.0f)) * f;
#pragma unroll
        for (int q = 0; q < PIECES; ++q) {
            float x[8];
            input(q, p.has_lo, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[8 * q + e] = fmaf(lin, x[e], v[8 * q + e] * g);
            if (p.mode == CMU_UPDATE) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = v[8 * q + e] * CMU_SCALE;
                put(buf0, q, x);
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
            __syncwarp();
        } else {
            if (p.w_in) result<float, true>(b, i0, j0, v);
            else if (p.out_type == CDG_T_F32) result<float, false>(b, i0, j0, v);
            else if (p.out_type == CDG_T_BF16) result<__nv_bfloat16, false>(b, i0, j0, v);
            else result<__half, false>(b, i0, j0, v);
            __syncwarp();
            fence_proxy_async_smem();  // the block has been read: the next fetch may overwrite it
            sync();
        }
        return true;
    }
    // A block of A or B and, off the diagonal, its transpose; high parts, then low parts.
    __device__ __forceinline__ void symmetric(int b, int i0, int j0, bool mirror, float (&v)[OWN]) const
    {
        for (int half = 0; half < (p.parts == 3 ? 2 : 1); ++half) {
            if (elected) bulk_wait_group_read<0>();
            sync();
#pragma unroll
            for (int q = 0; q < PIECES; ++q) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = v[8 * q + e];
                if (mirror) {
                    // column j of this row -> row j, column `row` of two 64-column blocks
                    const uint32_t at = buf1 + static_cast<uint32_t>(row / 64) * 8192u + (row & 7) * 2u;
                    const uint32_t c = (row & 63) >> 3;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        st_shared_u16(at + (part * OWN + 8 * q + e) * 128u + ((c ^ e) << 4), to_half_bits(x[e]));
                }
                put(buf0, q, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * q + e] = x[e];
            }
            fence_proxy_async_smem();
            sync();
            if (elected) {
                tma_store_3d(reinterpret_cast<uint64_t>(&p.tmY[half]), buf0, j0, i0, b);
                if (mirror) {
                    tma_store_3d(reinterpret_cast<uint64_t>(&p.tmT[half]), buf1, i0, j0, b);
                    if (i0 + 64 < p.M) tma_store_3d(reinterpret_cast<uint64_t>(&p.tmT[half]), buf1 + 8192u, i0 + 64, j0, b);
                }
                bulk_commit_group();
            }
            __syncwarp();
        }
    }
    // O or (STEP) W, lanes along the output's rows either way: eight elements'
    // loads and stores at a time.
    template <typename O, bool STEP>
    __device__ __forceinline__ void result(int b, int i0, int j0, const float (&v)[OWN]) const
    {
        const long long base = static_cast<long long>(b) * p.rows * p.cols;
        O *const out = static_cast<O *>(p.out) + base;
        const float *const w_in = STEP ? p.w_in + base : nullptr;
        const int mine = j0 + part * OWN, n = min(OWN, p.N - mine);
        if (p.transposed) {
            const int i = i0 + row;
            if (i >= p.M) return;
#pragma unroll
            for (int q0 = 0; q0 < OWN; q0 += 8) {
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (STEP && q0 + e < n) w[e] = w_in[static_cast<long long>(mine + q0 + e) * p.cols + i];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (q0 + e < n)
                        out[static_cast<long long>(mine + q0 + e) * p.cols + i] =
                            Elem<O>::put(STEP ? fmaf(p.w_keep, w[e], -p.w_step * v[q0 + e]) : v[q0 + e]);
            }
            return;
        }
        // through the staging: this warp's 32 rows x OWN columns of fp32, column c of row r at (c + r) % OWN
        sync();  // every row's input has been read
        const uint32_t w0 = buf0 + static_cast<uint32_t>(part * 4 + quad) * (32u * OWN * 4u);
#pragma unroll
        for (int q = 0; q < OWN; ++q) st_shared_f32(w0 + lane * (OWN * 4u) + ((q + lane) & (OWN - 1)) * 4u, v[q]);
        __syncwarp();
        const int r0 = i0 + quad * 32, rows = min(32, p.M - r0);
        for (int c0 = 0; c0 < OWN; c0 += 32) {
            const int c = c0 + lane;
            const long long at = static_cast<long long>(r0) * p.cols + mine + c;
            for (int r = 0; r < rows; r += 8) {
                float y[8], w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[e] = ld_shared_f32(w0 + (r + e) * (OWN * 4u) + ((c + r + e) & (OWN - 1)) * 4u);
                    if (STEP && r + e < rows && c < n) w[e] = w_in[at + static_cast<long long>(r + e) * p.cols];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (r + e < rows && c < n)
                        out[at + static_cast<long long>(r + e) * p.cols] =
                            Elem<O>::put(STEP ? fmaf(p.w_keep, w[e], -p.w_step * y[e]) : y[e]);
            }
        }
    }

    // 64-column chunks of this group in the tile at (i0, j0)
    __device__ __forceinline__ int chunks(int i0, int j0) const
    {
        return i0 < p.M ? max(0, min(FORM == CMU_NARROW ? 1 : 2, (p.N - j0 + 63) / 64)) : 0;
    }
};

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t at, float (&v)[N])
{
    uint32_t (&r)[N] = reinterpret_cast<uint32_t(&)[N]>(v);
#pragma unroll
    for (int q = 0; q < N / 16; ++q) tmem_ld_32x32b_x16(at + 16 * q, *reinterpret_cast<uint32_t(*)[16]>(&r[16 * q]));
    tmem_ld_wait();
}

// Persistent: every CTA (or CTA pair) walks the output tiles.  Warps 0 and 2
// load stages in turn, warp 1 issues the MMAs, warps 4.. run the epilogue,
// which overlaps the next tile's products (two accumulators).  Symmetric
// products compute the tiles on and below the diagonal and store the others as
// their transposes.
//
// One-part products of large matrices run in CTA pairs: 256 x 256 tiles, each
// CTA holding half of the rows of A and of B.  Others take 128 x 128 tiles, or,
// where those would leave most SMs idle, 128 x 64 tiles by clusters that split K:
// each CTA sums its range, the others leave their sums in shared memory, and
// the first adds them in order and runs the epilogue.
//
// The tensor core rounds every addition to its fp32 sum towards zero, so long
// chains drift (a Gaussian 3000 x 4608 fp32 U: 5e-5 in the result).  Two-part
// products therefore take CMU_CHAIN blocks at a time into one accumulator
// after the other, and the epilogue warps add them up in registers.
template <int FORM>
__global__ void __launch_bounds__(Layout<FORM>::kThreads, 1) gemm_kernel(const __grid_constant__ CmuGemm p)
{
    using Lay = Layout<FORM>;
    constexpr bool PAIR = Lay::kPair, NARROW = FORM == CMU_NARROW;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const Lay L(base);
    uint32_t *slot = reinterpret_cast<uint32_t *>(smem_raw + (L.full0 - raw) + Lay::kWords);
    volatile uint32_t *abort_flag = slot + 1, *used = slot + 2;  // used[stage]: parity of its last load, + 2
    static_assert(Lay::kWords + 8 + 4 * CMU_STAGES <= CMU_BAR_BYTES, "barrier area");
    const bool sym = p.mode <= CMU_POLY || p.mode == CMU_PARTIAL;  // B is K-major, as A
    const int warp = threadIdx.x / 32;
    const int width = PAIR ? 2 : NARROW ? p.split : 1;  // CTAs a tile
    const int rank = width > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int half = PAIR ? rank : 0;                   // of the pair's rows
    const int first = blockIdx.x / width, step = gridDim.x / width;
    const int total = p.tiles * p.batch;
    const int chain = p.parts > 1 || p.mode == CMU_PARTIAL ? CMU_CHAIN : INT_MAX;
    grid_dep_launch_dependents();
    if (threadIdx.x < 10)  // the tensor maps (five pairs, one after the other), fetched while the launch waits
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(p.tmA + threadIdx.x)) : "memory");
    if (threadIdx.x == 0) {
        for (int s = 0; s < CMU_STAGES; ++s) {
            mbar_init(L.full0 + 8u * s, 1);
            mbar_init(L.empty0 + 8u * s, 1);
            used[s] = 0u;
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(L.acc_full0 + 8u * a, 1);
            mbar_init(L.acc_empty0 + 8u * a, PAIR ? 32 : 8);  // one arrival per epilogue warp (of both CTAs)
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

    bool at_barrier = false;  // this thread has been at the barrier of a split K
    if (warp == 0 || warp == 2) {
        const bool leader = elect_one_sync();
        const uint32_t lead_full0 = PAIR ? mapa_shared(L.full0, 0) : L.full0;
        int s = 0, turn = 0;
        uint32_t parity = 0;
        bool ok = true;
        for (int t = first; ok && t < total; t += step) {
            const Tile<FORM> tile(p, sym, t, rank);
            const int row0 = tile.tm * Lay::kTileM + half * 128, col0 = tile.tn * Lay::kTileN + half * 128;
            const int blocks = p.parts * tile.kn;
            for (int k = 0; k < blocks; ++k) {
                if (turn == warp) {
                    if (!wait_bar(L.empty0 + 8u * s, parity ^ 1u, ctl)) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        used[s] = parity | 2u;
                        const uint32_t sa = L.s0 + s * Lay::kStage, sb = sa + CMU_HALF_BYTES;
                        const uint32_t bar = lead_full0 + 8u * s;
                        // low x high, high x low, then high x high: the tensor core rounds every
                        // addition towards zero, and the small parts go in while the sum is small
                        const int part = k / tile.kn, k0 = (tile.k0 + k - part * tile.kn) * CMU_BK;
                        const CUtensorMap &ma = p.tmA[p.parts > 1 && part == 0], &mb = p.tmB[p.parts == 3 && part == 1];
                        if (half == 0) mbar_arrive_expect_tx(L.full0 + 8u * s, (PAIR ? 2 : 1) * Lay::kStage);
                        tma_load_3d_to(PAIR, sa, ma, bar, k0, row0, tile.b);
                        if (sym) {
                            tma_load_3d_to(PAIR, sb, mb, bar, k0, col0, tile.b);
                        } else {
                            tma_load_3d_to(PAIR, sb, mb, bar, col0, k0, tile.b);
                            if (!NARROW) tma_load_3d_to(PAIR, sb + 8192u, mb, bar, col0 + 64, k0, tile.b);
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
        if (half == 0) {
            const bool leader = elect_one_sync();
            const uint32_t idesc = (1u << 4) | (sym ? 0u : 1u << 16) | (static_cast<uint32_t>(Lay::kCols >> 3) << 17) |
                                   (static_cast<uint32_t>(Lay::kTileM >> 4) << 24);
            int s = 0;
            uint32_t parity = 0, link = 0;
            bool ok = true;
            for (int t = first; ok && t < total; t += step) {
                const int blocks = p.parts * Tile<FORM>(p, sym, t, rank).kn;
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
                        const uint32_t sa = L.s0 + s * Lay::kStage, sb = sa + CMU_HALF_BYTES;
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
        Epilogue<FORM> e(p, L, ctl, sym);
        constexpr int OWN = Lay::kOwn;
        const uint32_t lane_base = (static_cast<uint32_t>(e.quad * 32) << 16) + e.part * OWN;
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
            const Tile<FORM> tile(p, sym, t, rank);
            const int i0 = tile.tm * Lay::kTileM + half * 128, j0 = tile.tn * Lay::kTileN + e.group * 128;
            const int n = NARROW && rank ? 0 : e.chunks(i0, j0);
            const bool mirror = tile.mirror;
            const float xs = p.first ? p.xs[tile.b] : CMU_SCALE;
            const bool fetches = p.mode != CMU_GRAM && p.mode != CMU_PARTIAL;
            if (n > 0 && fetches) e.fetch(tile.b, i0, j0);
            if constexpr (PAIR) {
                const uint32_t acc = link & 1u;
                ok = wait_bar(L.acc_full0 + 8u * acc, (link >> 1) & 1u, ctl);
                if (e.any(!ok)) break;
                ++link;
                tc_fence_after();
                for (int c = 0; c < n; ++c) {
                    float v[OWN];
                    tmem_ld(tmem + acc * Lay::kCols + e.group * 128 + c * 64 + lane_base, v);
                    if (c == n - 1) hand_back(acc);
                    if (!(ok = e.chunk(tile.b, i0, j0 + 64 * c, mirror, xs, v))) break;
                    if (c + 1 < n && fetches) e.fetch(tile.b, i0, j0 + 64 * (c + 1));
                }
                if (n == 0) hand_back(acc);
            } else {
                constexpr int CHUNKS = Lay::kTileN / 64;
                float sum[CHUNKS][OWN];
                const int links = (p.parts * tile.kn - 1) / chain + 1;
                for (int k = 0; ok && k < links; ++k, ++link) {
                    const uint32_t acc = link & 1u;
                    ok = __all_sync(0xFFFFFFFFu, wait_bar(L.acc_full0 + 8u * acc, (link >> 1) & 1u, ctl));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < CHUNKS; ++c) {
                        float v[OWN];
                        tmem_ld(tmem + acc * Lay::kCols + c * 64 + lane_base, v);
#pragma unroll
                        for (int q = 0; q < OWN; ++q) sum[c][q] = k ? sum[c][q] + v[q] : v[q];
                    }
                    hand_back(acc);
                }
                if (e.any(!ok)) {
                    ok = false;
                    break;
                }
                if (NARROW && p.split > 1) {
                    // the other CTAs' sums in their ring (all of it read: the range is done), four columns in a 16-byte
                    // piece, piece c of row r at (c + r) % 8 of the thread's eight; the first CTA adds them in rank order
                    const uint32_t own = (e.part * 128 + e.row) * (OWN * 4u);
                    if (rank) {
#pragma unroll
                        for (int c = 0; c < OWN / 4; ++c)
                            st_shared_v4(L.s0 + own + ((c + e.lane) % (OWN / 4)) * 16u, __float_as_uint(sum[0][4 * c]),
                                         __float_as_uint(sum[0][4 * c + 1]), __float_as_uint(sum[0][4 * c + 2]),
                                         __float_as_uint(sum[0][4 * c + 3]));
                    }
                    __syncwarp();
                    cluster_barrier_arrive();
                    cluster_barrier_wait();
                    at_barrier = true;
                    if (rank == 0 && n > 0) {
                        for (int r = 1; r < p.split; ++r) {
                            const uint32_t at = mapa_shared(L.s0, r) + own;
                            float4 x[OWN / 4];  // all loads before the additions: a load takes hundreds of cycles
#pragma unroll
                            for (int c = 0; c < OWN / 4; ++c) x[c] = ld_cluster_f32x4(at + ((c + e.lane) % (OWN / 4)) * 16u);
#pragma unroll
                            for (int c = 0; c < OWN / 4; ++c) {
                                sum[0][4 * c] += x[c].x;
                                sum[0][4 * c + 1] += x[c].y;
                                sum[0][4 * c + 2] += x[c].z;
                                sum[0][4 * c + 3] += x[c].w;
                            }
                        }
                    }
                }
                if (FORM == CMU_SQUARE && p.mode == CMU_PARTIAL) {
                    // rows and columns below M, 16 bytes at a time (pads up to a multiple of 4 are sums of zeros)
                    float *out = p.partial + static_cast<long long>(t) * (CMU_SIDE * CMU_SIDE) + e.row * CMU_SIDE;
                    if (e.row < p.M)
#pragma unroll
                        for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
                            for (int q = 0; q < OWN; q += 4) {
                                const int col = 64 * c + e.part * OWN + q;
                                if (col < p.N)
                                    *reinterpret_cast<float4 *>(out + col) =
                                        make_float4(sum[c][q], sum[c][q + 1], sum[c][q + 2], sum[c][q + 3]);
                            }
                    __syncwarp();
                    continue;
                }
#pragma unroll
                for (int c = 0; c < CHUNKS; ++c) {
                    if (c >= n) break;
                    if (!(ok = e.chunk(tile.b, i0, j0 + 64 * c, mirror, xs, sum[c]))) break;
                    if (c + 1 < n && fetches) e.fetch(tile.b, i0, j0 + 64 * (c + 1));
                }
            }
        }
        if (e.elected) bulk_wait_group_all();
    }
    if (NARROW && p.split > 1) {
        // the loaders and the MMA warp stand at the cluster's barrier too (the epilogue warps have passed it, unless
        // the launch is giving up before they came there)
        if (warp < CDG_EPI_WARP0 || !at_barrier) {
            cluster_barrier_arrive();
            cluster_barrier_wait();
        }
    }

    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) {
        // copies in flight land before the CTA exits
        volatile uint32_t no_abort = 0;
        const Ctl drain{&no_abort, p.status};
        if (half == 0) {
            for (int s = 0; s < CMU_STAGES; ++s)
                if (used[s] & 2u) wait_bar(L.full0 + 8u * s, used[s] & 1u, drain);
        }
        const uint64_t t0 = global_timer_ns();  // the peer's barrier, and the epilogue's blocks
        while (global_timer_ns() - t0 < 200000ull) {
        }
    }
    tc_fence_before();
    __syncthreads();
    if (width > 1) cluster_sync();  // no CTA leaves while another may still signal it or read its shared memory
    if (warp == 1) {
        tc_fence_after();
        if (PAIR) tmem_dealloc_pair(tmem, 2 * Lay::kCols);
        else tmem_dealloc(tmem, 2 * Lay::kCols);
    }
}

// Tiles of a matrix in one form.
template <int FORM>
void count_tiles(CmuGemm &p)
{
    using Lay = Layout<FORM>;
    p.tiles_m = (p.M + Lay::kTileM - 1) / Lay::kTileM;
    const int tiles_n = (p.N + Lay::kTileN - 1) / Lay::kTileN;
    if (p.mode == CMU_PARTIAL) return;  // the caller's ranges of K
    if (p.mode > CMU_POLY) p.tiles = p.tiles_m * tiles_n;
    else if (FORM == CMU_NARROW) p.tiles = p.tiles_m * (p.tiles_m + 1) - (tiles_n < 2 * p.tiles_m);  // its last row may lack a tile
    else p.tiles = p.tiles_m * (p.tiles_m + 1) / 2;
}

template <int FORM>
cudaError_t launch_gemm(CmuGemm p, int sms, cudaStream_t s)
{
    using Lay = Layout<FORM>;
    count_tiles<FORM>(p);
    const long long total = static_cast<long long>(p.tiles) * p.batch;
    if (total > INT_MAX / 16) return cudaErrorInvalidConfiguration;
    const int width = Lay::kPair ? 2 : FORM == CMU_NARROW ? p.split : 1;
    cudaLaunchConfig_t cfg = {};
    // persistent, but for tiles whose K is split (their ring holds the sums at the end)
    const long long at_once = FORM == CMU_NARROW ? total : std::min<long long>(total, std::max(1, sms / width));
    cfg.gridDim = dim3(static_cast<unsigned>(width * at_once));
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
    cfg.numAttrs = width > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, gemm_kernel<FORM>, p);
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
// 512 threads: thread t holds row t % 128 and, of the accumulators' columns,
// the 16 from 16 (t / 128) and the 16 from 64 + 16 (t / 128).  Only the first
// m rows and columns, rounded up to 16, are multiplied and read.
constexpr int kItThreads = 512;
constexpr uint32_t kMatBytes = 4 * CMU_HALF_BYTES;  // high parts of columns 0-63, 64-127; then low parts
constexpr int kItSmem = 1024 + 3 * static_cast<int>(kMatBytes) + 256;

__global__ void __launch_bounds__(kItThreads, 1) iterate_kernel(const CmuIterate p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t mA = base, mQ = base + kMatBytes, mP = base + 2 * kMatBytes, bar0 = base + 3 * kMatBytes;
    uint32_t *slot = reinterpret_cast<uint32_t *>(smem_raw + (bar0 - raw) + 16);
    volatile uint32_t *abort_flag = slot + 1;
    const int tid = threadIdx.x, warp = tid / 32;
    const int row = tid % 128, group = tid / 128, b = blockIdx.x;
    const int used = (p.m + 15) / 16 * 16;
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
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    // this thread's chunks of 16 columns: from 16 group, and 64 + 16 group
    const bool rows = (warp & 3) * 32 < used;  // warp-uniform
    const int chunks = !rows ? 0 : 64 + 16 * group < used ? 2 : 16 * group < used ? 1 : 0;

    // the ranges' partial sums, in order, to A = sum / xs^2 (fp32, in Q's place)
    {
        const float f = (1.0f / p.xs[b]) / p.xs[b];
        const float *src = p.partial + static_cast<long long>(b) * p.splits * (CMU_SIDE * CMU_SIDE);
        const int n4 = (p.m + 3) / 4;
        for (int x = tid; x < p.m * n4; x += kItThreads) {
            const int r = x / n4, c = x - r * n4;
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
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

    // columns 64 s + 8 q .. + 7 of this thread's row in matrix `mat`, part 0 or 1
    auto piece = [&](uint32_t mat, int part, int s, int q) {
        return mat + static_cast<uint32_t>(2 * part + s) * CMU_HALF_BYTES + static_cast<uint32_t>(row) * 128u +
               ((static_cast<uint32_t>(q) ^ (row & 7)) << 4);
    };
    auto put = [&](uint32_t mat, int s, int q, const float *x) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __half2 h = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
            const float2 w = __half22float2(h);
            const __half2 l = __floats2half2_rn(x[2 * e] - w.x, x[2 * e + 1] - w.y);
            hi[e] = *reinterpret_cast<const uint32_t *>(&h);
            lo[e] = *reinterpret_cast<const uint32_t *>(&l);
        }
        st_shared_v4(piece(mat, 0, s, q), hi[0], hi[1], hi[2], hi[3]);
        st_shared_v4(piece(mat, 1, s, q), lo[0], lo[1], lo[2], lo[3]);
    };
    auto get = [&](uint32_t mat, int s, int q, float (&x)[8]) {
        uint32_t w[4];
        float y[8];
        ld_shared_v4(piece(mat, 0, s, q), w);
        widen_vec<__half>(make_uint4(w[0], w[1], w[2], w[3]), x);
        ld_shared_v4(piece(mat, 1, s, q), w);
        widen_vec<__half>(make_uint4(w[0], w[1], w[2], w[3]), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += y[e];
    };
    // accumulator d <- X Y: low x high, high x low, high x high; by one lane of the first warp
    const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(used >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
    const int ksteps = used / 16;
    auto multiply = [&](uint32_t d, uint32_t x, uint32_t y) {
        const uint32_t acc = tmem + 128 * d;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
            const uint64_t ad = sdesc_k128_sw128(x + (part == 0 ? 2u * CMU_HALF_BYTES : 0u));
            const uint64_t bd = sdesc_k128_sw128(y + (part == 1 ? 2u * CMU_HALF_BYTES : 0u));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t step = (k / 4) * (CMU_HALF_BYTES >> 4) + (k % 4) * 2u;  // descriptor units
                if (k < ksteps) umma_f16(acc, ad + step, bd + step, idesc, (part | k) != 0);
            }
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
    // accumulator d times f into matrix `mat`, after `also` has seen or changed each
    // piece: also(values, slice, piece)
    auto store = [&](int d, float f, uint32_t mat, auto also) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (c >= chunks) break;
            float v[16];
            tmem_ld_32x32b_x16(tmem + 128 * d + 64 * c + 16 * group + lane_base, reinterpret_cast<uint32_t(&)[16]>(v));
            tmem_ld_wait();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * h + e] *= f;
                also(v + 8 * h, c, 2 * group + h);
                put(mat, c, 2 * group + h, v + 8 * h);
            }
            __syncwarp();
        }
    };
    auto nothing = [](float *, int, int) {};

    // A to its two parts
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (c >= chunks) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x[8];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const uint32_t at = 16u * c + 4u * group + 2u * h + g;  // of the row's 16-byte pieces of fp32
                uint32_t w[4] = {0u, 0u, 0u, 0u};
                if (row < p.m && static_cast<int>(4 * at) < p.m) ld_shared_v4(mQ + row * 512u + ((at ^ (row & 31)) << 4), w);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * g + e] = CMU_SCALE * __uint_as_float(w[e]);
            }
            put(mA, c, 2 * group + h, x);
        }
    }
    ready();
    constexpr float kInv = 1.0f / CMU_SCALE;
    bool ok = true;
    for (int k = 0; k < p.steps; ++k) {
        // Q = a I + b A + c A A
        if (warp == 0) {
            if (elect_one_sync()) multiply(0, mA, mA);
            __syncwarp();
        }
        if (!(ok = wait(0))) break;
        store(0, p.c * kInv, mQ, [&](float *v, int s, int q) {
            float x[8];
            get(mA, s, q, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = fmaf(p.b, x[e], v[e]);
                if (64 * s + 8 * q + e == row) v[e] += p.a * CMU_SCALE;
            }
            if (k == 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = v[e] * (CMU_POLY_SCALE * kInv);
                put(mP, s, q, x);
            }
        });
        ready();
        const bool last = k == p.steps - 1;
        if (warp == 0) {
            if (elect_one_sync()) {
                if (!last) multiply(0, mQ, mA);
                if (k > 0) multiply(1, mQ, mP);
            }
            __syncwarp();
        }
        if (!last) {  // T = Q A, in A's place
            if (!(ok = wait(0))) break;
            store(0, kInv, mA, nothing);
            ready();
            if (warp == 0) {
                if (elect_one_sync()) multiply(0, mA, mQ);  // A <- T Q
                __syncwarp();
            }
        }
        if (k > 0) {  // P <- Q P
            if (!(ok = wait(1))) break;
            store(1, kInv, mP, nothing);
        }
        if (!last) {
            if (!(ok = wait(0))) break;
            store(0, kInv, mA, nothing);
            ready();
        }
    }
    // P without its diagonal, and the diagonal
    if (ok && row < p.m) {
        const long long at = (static_cast<long long>(b) * p.m + row) * p.pitch_a;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = 64 * c + 16 * group + 8 * h;
                if (c >= chunks || j >= p.m) continue;
                float x[8], y[8];
                get(mP, c, 2 * group + h, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (j + e == row) {
                        p.diag[static_cast<long long>(b) * p.m + row] = x[e] * (1.0f / CMU_POLY_SCALE);
                        x[e] = 0.0f;
                    }
                    y[e] = x[e] - __half2float(__float2half_rn(x[e]));
                }
                *reinterpret_cast<uint4 *>(p.poly + at + j) = narrow_vec<__half>(x);
                *reinterpret_cast<uint4 *>(p.poly_lo + at + j) = narrow_vec<__half>(y);
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
cudaError_t launch_norm(const CmuPrepare &p, cudaStream_t s)
{
    return launch_early(norm_kernel<T>, dim3(p.partials, p.batch), kPrepareThreads, 0, s, p);
}
template <typename T>
cudaError_t launch_split(const CmuPrepare &p, cudaStream_t s)
{
    if (!p.transposed && p.cols % 8 == 0)
        return launch_early(split_flat_kernel<T>, dim3(p.partials, p.batch), kPrepareThreads, 0, s, p);
    const int m = p.transposed ? p.cols : p.rows, n = p.transposed ? p.rows : p.cols;
    return launch_early(split_kernel<T>, dim3((n + 63) / 64, (m + 63) / 64, p.batch), kPrepareThreads, 0, s, p);
}

}  // namespace
}  // namespace cdg

cudaError_t cmu_prepare_kernels()
{
    using namespace cdg;
    const auto raise = [](const void *f, int bytes) {
        return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    };
    cudaError_t e = raise(reinterpret_cast<const void *>(gemm_kernel<CMU_PAIR>), Layout<CMU_PAIR>::kSmem);
    if (e == cudaSuccess) e = raise(reinterpret_cast<const void *>(gemm_kernel<CMU_SQUARE>), Layout<CMU_SQUARE>::kSmem);
    if (e == cudaSuccess) e = raise(reinterpret_cast<const void *>(gemm_kernel<CMU_NARROW>), Layout<CMU_NARROW>::kSmem);
    if (e == cudaSuccess) e = raise(reinterpret_cast<const void *>(iterate_kernel), kItSmem);
    return e;
}

cudaError_t cmu_launch_norm(const CmuPrepare &p, cudaStream_t s)
{
    return p.dtype == CDG_F32 ? cdg::launch_norm<float>(p, s)
                              : p.dtype == CDG_F16 ? cdg::launch_norm<__half>(p, s) : cdg::launch_norm<__nv_bfloat16>(p, s);
}

cudaError_t cmu_launch_split(const CmuPrepare &p, cudaStream_t s)
{
    return p.dtype == CDG_F32 ? cdg::launch_split<float>(p, s)
                              : p.dtype == CDG_F16 ? cdg::launch_split<__half>(p, s) : cdg::launch_split<__nv_bfloat16>(p, s);
}

cudaError_t cmu_launch_iterate(const CmuIterate &p, cudaStream_t s)
{
    return cdg::launch_early(cdg::iterate_kernel, dim3(p.batch), cdg::kItThreads, cdg::kItSmem, s, p);
}

cudaError_t cmu_launch_gemm(const CmuGemm &p, int sms, cudaStream_t s)
{
    if (p.form == CMU_PAIR) return cdg::launch_gemm<CMU_PAIR>(p, sms, s);
    if (p.form == CMU_NARROW) return cdg::launch_gemm<CMU_NARROW>(p, sms, s);
    return cdg::launch_gemm<CMU_SQUARE>(p, sms, s);
}
