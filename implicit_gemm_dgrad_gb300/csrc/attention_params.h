// Launch parameters shared by the host side (attention_api.cu) and the sm_103a
// kernels (attention_sm103.cu, attention_grad_sm103.cu) of the attention.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cdg_params.h"

#define CAT_TILE 128      // queries of an MMA tile, keys of a step
#define CAT_THREADS 384   // forward: 8 warps that compute, 1 that loads, 1 that issues MMAs, 2 more
#define CAT_GRAD_THREADS 640  // gradient: 16 warps that compute, 1 that loads, 1 that issues MMAs, 2 more

struct CatParams {
    CUtensorMap tmQ, tmK, tmV, tmDO;  // {dim, heads, tokens}, boxes of 64 columns x 1 head x 128 tokens, 128-byte swizzle
    const void *q_offsets, *k_offsets;  // sequences + 1 numbers each, or NULL: one sequence of all tokens
    int index_bytes, sequences;
    int q_tokens, k_tokens;
    int heads, kv_heads, group;  // group = heads / kv_heads
    int dim;                     // head width: a multiple of 8
    int slices;                  // 64-column slices of a head: 1 or 2
    int ksteps;                  // ceil(dim / 16)
    int causal, window;
    float scale, scale_log2;     // scale, scale * log2(e)
    uint32_t idesc_qk;           // 128 x 128, both operands K-major
    uint32_t idesc_pv;           // 128 x dim (up to a multiple of 16), B MN-major
    // outputs: row strides in elements
    void *o, *dq, *dk, *dv;
    long long ld_o, ld_dq, ld_dk, ld_dv;
    float *lse;                  // [heads][q_tokens]
    // gradient: the forward's o and its gradient, and for each row (- lse log2 e, sum of do o), [heads][q_tokens]
    const void *o_in, *d_o;
    long long ld_oi, ld_do;
    const float *lse_in;
    float2 *stats;
    int splits;                  // dk and dv: parts of a group's query heads, a CTA each; above 1 their fp32 sums go to
    float *partial;              // [splits][dk, dv][k_tokens][kv_heads * dim], and are added in order by a kernel of their own
    int *status;
};

size_t cat_smem_forward(int slices);
size_t cat_smem_grad(int slices);
cudaError_t cat_prepare_forward();
cudaError_t cat_prepare_grad();
// bf16: 1 for bfloat16, 0 for float16; items: CTAs of a launch (of dk and dv: without the splits)
cudaError_t cat_launch_forward(const CatParams &p, int bf16, long long items, cudaStream_t s);
cudaError_t cat_launch_stats(const CatParams &p, int bf16, cudaStream_t s);
cudaError_t cat_launch_dkv(const CatParams &p, int bf16, long long items, cudaStream_t s);
cudaError_t cat_launch_dq(const CatParams &p, int bf16, long long items, cudaStream_t s);
cudaError_t cat_launch_join(const CatParams &p, int bf16, long long items, cudaStream_t s);
