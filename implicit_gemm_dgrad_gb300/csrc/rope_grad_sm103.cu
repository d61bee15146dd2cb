// The gradient of the norms of queries and keys with the position rotation:
// kernels (rope_device.cuh), and the sum of the weights' partial gradients.
#include "rope_device.cuh"

namespace cdg {
namespace {

// dw = the sum of a side's partial rows, 32 columns a CTA.
__global__ void __launch_bounds__(1024) rope_sum_kernel(const __grid_constant__ RopeArgs p)
{
    __shared__ float red[32][33];
    grid_dep_wait();
    const RopeSide &sd = p.side[blockIdx.y];
    if (!sd.dw) return;
    const int x = threadIdx.x & 31, y = threadIdx.x / 32, col = blockIdx.x * 32 + x;
    const int first = blockIdx.y ? p.side[0].blocks * p.side[0].ctas : 0, n = sd.blocks * sd.ctas;
    float v = 0.0f;
    if (col < p.dim)
        for (int i = y; i < n; i += 32) v += p.partial[static_cast<long long>(first + i) * p.dim + col];
    red[y][x] = v;
    __syncthreads();
    v = red[x][y];
#pragma unroll
    for (int d = 16; d; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if (x == 0 && blockIdx.x * 32 + y < p.dim) sd.dw[blockIdx.x * 32 + y] = v;
}

}  // namespace
}  // namespace cdg

cudaError_t crp_launch_grad(cdg::RopeArgs &a, int dtype, cudaStream_t s)
{
    using namespace cdg;
    cudaError_t e = cudaSuccess;
    if (a.tokens > 0)
        e = dtype == CDG_F32   ? launch_rope<float, true>(a, s)
            : dtype == CDG_F16 ? launch_rope<__half, true>(a, s)
                               : launch_rope<__nv_bfloat16, true>(a, s);
    if (e == cudaSuccess && (a.side[0].dw || a.side[1].dw))
        e = launch_early(rope_sum_kernel, dim3((a.dim + 31) / 32, 2), dim3(1024), 0, s, a);
    return e;
}
