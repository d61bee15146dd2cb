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
    // fp16: what scales ds.  Of each CTA of the statistics (stat_ctas over the queries' rows,
    // then size_ctas over v's), the largest |do|^2 or |v|^2 of a row's head, and |do o|, of its finite
    // rows that a sequence holds:
    const void *v_in;
    long long ld_v;
    uint4 *sizes;
    int stat_ctas, size_ctas;
    // Parts that an item's steps are split into, a CTA each, where items are few.  Above
    // 1 their fp32 results go to `partial`, and a kernel of its own joins them in order:
    int q_splits;                // o, or dq: q_partial is [q_splits][q_tokens][heads * dim],
    float *q_partial;
    float *lse_partial;          //   of o with each part's own lse, [q_splits][heads][q_tokens]
    int k_splits;                // dk and dv: k_partial is [k_splits][dv, dk][k_tokens][kv_heads * dim]
    float *k_partial;
    int *status;
};

size_t cat_smem_forward(int slices);
size_t cat_smem_grad(int slices);
cudaError_t cat_prepare_forward();
cudaError_t cat_prepare_grad();
#define CAT_JOIN_ROWS 16  // rows and one head that a CTA of a join takes

// CTAs of the statistics, over the queries' rows (bf16 != 0) or, in fp16, over rows of either side:
// so few that the next kernels have not many sizes to read.
long long cat_stat_ctas(long long tokens, int heads, int bf16);
// bf16: 1 for bfloat16, 0 for float16; items: CTAs of a launch without the splits
cudaError_t cat_launch_forward(const CatParams &p, int bf16, long long items, long long join_items, cudaStream_t s);
cudaError_t cat_launch_stats(const CatParams &p, int bf16, cudaStream_t s);
cudaError_t cat_launch_dkv(const CatParams &p, int bf16, long long items, cudaStream_t s);
cudaError_t cat_launch_dq(const CatParams &p, int bf16, long long items, cudaStream_t s);
// joins what dk and dv, dq, or both have in parts; CTAs for keys' rows and for queries' rows
cudaError_t cat_launch_grad_join(const CatParams &p, int bf16, long long key_items, long long query_items, cudaStream_t s);
