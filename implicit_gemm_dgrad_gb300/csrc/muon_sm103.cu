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
struct Epilogue {
    const CmuGemm &p;
    int b, i;         // matrix, row of the output
    float xs;         // scale of X
    bool mirror;      // symmetric, off the diagonal: write the transpose too

    // Columns [j, j + 32) of row i: acc holds the sums.
    __device__ __forceinline__ void chunk(int j0, const float *acc) const
    {
        if (p.mode == CMU_GRAM) {
            const float f = (CMU_SCALE / xs) / xs;
            float v[32];
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] = acc[q] * f;
            symmetric(p.mat, p.mat_lo, j0, v);
        } else if (p.mode == CMU_POLY) {
            const long long row = (static_cast<long long>(b) * p.M + i) * p.pitch_a + j0;
            float v[32];
#pragma unroll
            for (int q = 0; q < 32; ++q) {
                float a = 0.0f;
                if (i < p.M && j0 + q < p.N) {
                    a = half_bits(p.mat[row + q]);
                    if (p.parts == 3) a += half_bits(p.mat_lo[row + q]);
                }
                v[q] = fmaf(p.b, a, p.c * (acc[q] * (1.0f / CMU_SCALE)));
                if (j0 + q == i && i < p.M) {
                    p.diag[static_cast<long long>(b) * p.M + i] = v[q] * (1.0f / CMU_SCALE);
                    v[q] = 0.0f;
                }
            }
            symmetric(p.poly, p.poly_lo, j0, v);
        } else {
            if (i >= p.M) return;
            const long long at = (static_cast<long long>(b) * p.M + i) * p.pitch_x + j0;
            const float f = 1.0f / xs, lin = (p.a + p.diag[static_cast<long long>(b) * p.M + i]) * f;
#pragma unroll
            for (int q = 0; q < 32; ++q) {
                const int j = j0 + q;
                if (j >= p.N) break;
                float x = half_bits(p.x_hi[at + q]);
                if (p.has_lo) x += half_bits(p.x_lo[at + q]);
                const float y = fmaf(lin, x, acc[q] * (f / CMU_SCALE));
                if (p.mode == CMU_UPDATE) {
                    const float s = y * CMU_SCALE;
                    const uint16_t hi = to_half_bits(s);
                    p.y_hi[at + q] = hi;
                    p.y_lo[at + q] = to_half_bits(s - half_bits(hi));
                } else {
                    const long long o = static_cast<long long>(b) * p.rows * p.cols +
                                        (p.transposed ? static_cast<long long>(j) * p.cols + i
                                                      : static_cast<long long>(i) * p.cols + j);
                    if (p.w_in) static_cast<float *>(p.out)[o] = fmaf(p.w_keep, p.w_in[o], -p.w_step * y);
                    else if (p.out_type == CDG_T_F32) static_cast<float *>(p.out)[o] = y;
                    else if (p.out_type == CDG_T_BF16) static_cast<__nv_bfloat16 *>(p.out)[o] = __float2bfloat16_rn(y);
                    else static_cast<__half *>(p.out)[o] = __float2half_rn(y);
                }
            }
        }
    }
    __device__ __forceinline__ void symmetric(uint16_t *out, uint16_t *out_lo, int j0, const float (&v)[32]) const
    {
        if (i >= p.M) return;
        const long long base = static_cast<long long>(b) * p.M * p.pitch_a;
#pragma unroll
        for (int q = 0; q < 32; ++q) {
            if (j0 + q >= p.N) break;
            const long long at = base + static_cast<long long>(i) * p.pitch_a + j0 + q;
            const long long to = base + static_cast<long long>(j0 + q) * p.pitch_a + i;
            const uint16_t hi = to_half_bits(v[q]);
            out[at] = hi;
            if (mirror) out[to] = hi;
            if (p.parts == 3) {
                const uint16_t lo = to_half_bits(v[q] - half_bits(hi));
                out_lo[at] = lo;
                if (mirror) out_lo[to] = lo;
            }
        }
    }
};

// One 128 x 128 output tile a CTA: warp 0 loads, warp 1 issues the MMAs, warps
// 4-7 read the accumulator.  Symmetric products compute the tiles on and below
// the diagonal and write the others as their transposes.
//
// The tensor core rounds every addition to its fp32 sum towards zero, so long
// chains drift (a Gaussian 3000 x 4608 fp32 U: 5e-5 in the result).  Two-part
// products therefore take CMU_CHAIN blocks at a time into one of two
// accumulators, and the epilogue warps add them up in registers.
__global__ void __launch_bounds__(CDG_THREADS, 1) gemm_kernel(const __grid_constant__ CmuGemm p)
{
    extern __shared__ uint8_t smem_raw[];
    const bool sym = p.mode <= CMU_POLY;
    const int tm = blockIdx.y, tn = blockIdx.x, b = blockIdx.z;
    if (sym && tn > tm) return;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t bars = base + CMU_STAGES * CMU_STAGE_BYTES;
    const uint32_t full0 = bars, empty0 = bars + 8u * CMU_STAGES, acc_full0 = bars + 16u * CMU_STAGES,
                   acc_empty0 = acc_full0 + 16u, drain_bar = acc_full0 + 32u;
    uint32_t *slot = reinterpret_cast<uint32_t *>(smem_raw + (bars - raw) + 16 * CMU_STAGES + 40);
    volatile uint32_t *abort_flag = slot + 1;
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < CMU_STAGES; ++s) {
            mbar_init(full0 + 8u * s, 1);
            mbar_init(empty0 + 8u * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(acc_full0 + 8u * a, 1);
            mbar_init(acc_empty0 + 8u * a, 4);  // one arrival per epilogue warp
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(slot), 2 * CMU_BN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    const Ctl ctl{abort_flag, p.status};
    const int kblocks = (p.K + CMU_BK - 1) / CMU_BK, blocks = p.parts * kblocks;
    const int chain = p.parts == 3 ? CMU_CHAIN : blocks;

    if (warp == 0) {
        const bool leader = elect_one_sync();
        uint32_t loaded = 0;
        for (int k = 0; k < blocks; ++k) {
            const int s = k % CMU_STAGES;
            if (!wait_bar(empty0 + 8u * s, ((k / CMU_STAGES) & 1u) ^ 1u, ctl)) break;
            if (leader) {
                const uint32_t sa = base + s * CMU_STAGE_BYTES, sb = sa + CMU_BM * CMU_BK * 2, bar = full0 + 8u * s;
                // low x high, high x low, then high x high: the tensor core rounds every
                // addition towards zero, and the small parts go in while the sum is small
                const int part = k / kblocks, k0 = (k - part * kblocks) * CMU_BK;
                const uint64_t mapA = reinterpret_cast<uint64_t>(&p.tmA[p.parts == 3 && part == 0]);
                const uint64_t mapB = reinterpret_cast<uint64_t>(&p.tmB[p.parts == 3 && part == 1]);
                mbar_arrive_expect_tx(bar, CMU_STAGE_BYTES);
                tma_load_3d(sa, mapA, bar, k0, tm * CMU_BM, b);
                if (sym) {
                    tma_load_3d(sb, mapB, bar, k0, tn * CMU_BN, b);
                } else {
                    for (int q = 0; q < CMU_BN / 64; ++q)
                        tma_load_3d(sb + q * 8192, mapB, bar, tn * CMU_BN + q * 64, k0, b);
                }
            }
            __syncwarp();
            loaded = k + 1;
        }
        // on an abort, let the loads in flight land before the CTA exits
        if (*abort_flag) {
            volatile uint32_t no_abort = 0;
            const Ctl drain{&no_abort, p.status};
            for (uint32_t k = loaded > CMU_STAGES ? loaded - CMU_STAGES : 0; k < loaded; ++k)
                wait_bar(full0 + 8u * (k % CMU_STAGES), (k / CMU_STAGES) & 1u, drain);
        }
    } else if (warp == 1) {
        const bool leader = elect_one_sync();
        const uint32_t idesc = (1u << 4) | (sym ? 0u : 1u << 16) | (static_cast<uint32_t>(CMU_BN >> 3) << 17) |
                               (static_cast<uint32_t>(CMU_BM >> 4) << 24);
        for (int k = 0; k < blocks; ++k) {
            const int s = k % CMU_STAGES, link = k / chain, in_chain = k - link * chain;
            const uint32_t acc = link & 1;
            if (in_chain == 0 && !wait_bar(acc_empty0 + 8u * acc, ((link >> 1) & 1u) ^ 1u, ctl)) break;
            if (!wait_bar(full0 + 8u * s, (k / CMU_STAGES) & 1u, ctl)) break;
            tc_fence_after();
            if (leader) {
                const uint32_t sa = base + s * CMU_STAGE_BYTES, sb = sa + CMU_BM * CMU_BK * 2;
                const uint64_t ad = sdesc_k128_sw128(sa);
                const uint64_t bd = sym ? sdesc_k128_sw128(sb) : desc_mn_sw128(sb, 8192);
                const uint32_t bstep = sym ? 2u : 128u;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    umma_f16(tmem + acc * CMU_BN, ad + 2u * q, bd + bstep * q, idesc, (in_chain | q) != 0);
                umma_commit(empty0 + 8u * s);
                if (in_chain == chain - 1 || k == blocks - 1) umma_commit(acc_full0 + 8u * acc);
            }
            __syncwarp();
        }
        // tensor memory is freed only after the MMAs in flight
        if (leader) umma_commit(drain_bar);
        __syncwarp();
        volatile uint32_t no_abort = 0;
        wait_bar(drain_bar, 0, Ctl{&no_abort, p.status});
    } else if (warp >= CDG_EPI_WARP0) {
        const int quad = warp & 3, lane = threadIdx.x % 32;
        float sum[CMU_BN];
        bool ok = true;
        for (int link = 0; link * chain < blocks; ++link) {
            const uint32_t acc = link & 1;
            if (!wait_bar(acc_full0 + 8u * acc, (link >> 1) & 1u, ctl)) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int cc = 0; cc < CMU_BN; cc += 32) {
                uint32_t r[32];
                const uint32_t at = tmem + acc * CMU_BN + cc + (static_cast<uint32_t>(quad * 32) << 16);
                tmem_ld_32x32b_x16(at, *reinterpret_cast<uint32_t(*)[16]>(&r[0]));
                tmem_ld_32x32b_x16(at + 16, *reinterpret_cast<uint32_t(*)[16]>(&r[16]));
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 32; ++q) sum[cc + q] = link ? sum[cc + q] + __uint_as_float(r[q]) : __uint_as_float(r[q]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty0 + 8u * acc);
        }
        if (ok) {
            const Epilogue e{p, b, tm * CMU_BM + quad * 32 + lane, p.first ? p.xs[b] : CMU_SCALE, sym && tn < tm};
#pragma unroll
            for (int cc = 0; cc < CMU_BN; cc += 32)
                if (tn * CMU_BN + cc < p.N) e.chunk(tn * CMU_BN + cc, sum + cc);
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * CMU_BN);
    }
}

constexpr int kSmem = 1024 + CMU_STAGES * CMU_STAGE_BYTES + 256;

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
    return cudaFuncSetAttribute(cdg::gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, cdg::kSmem);
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

cudaError_t cmu_launch_gemm(const CmuGemm &p, cudaStream_t s)
{
    const dim3 grid((p.N + CMU_BN - 1) / CMU_BN, (p.M + CMU_BM - 1) / CMU_BM, p.batch);
    cdg::gemm_kernel<<<grid, CDG_THREADS, cdg::kSmem, s>>>(p);
    return cudaGetLastError();
}
