// C-ABI of the attention and its gradient: validation, tensor maps, launches;
// the kernels are in attention_sm103.cu and attention_grad_sm103.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "../../include/cdg.h"
#include "attention_params.h"
#include "token_device.cuh"

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled()
{
    static const EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                           cudaSuccess &&
                       q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<EncodeTiledFn>(p)
                   : nullptr;
    }();
    return fn;
}

constexpr int kMaxTokens = 1 << 30;   // tokens of a call: tensor-map coordinates are 32 bits
constexpr int kMaxHeads = 1024;
constexpr int kMaxSequences = 1 << 20;

}  // namespace

struct cdg_attention_st {
    int heads, kv_heads, dim, dtype, causal, window, device, sms;
    float scale;
    bool host_only;
    int *d_status;
};

namespace {

int make_attention_plan(int heads, int kv_heads, int dim, int dtype, int causal, int window, float scale, bool host_only,
                        cdg_attention_t *out)
{
    if (!out) return CDG_ERR_INVALID_ARG;
    *out = nullptr;
    if (heads < 1 || kv_heads < 1 || heads % kv_heads || dim < 1 || (dtype != CDG_F16 && dtype != CDG_BF16 && dtype != CDG_F32) ||
        (causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal) || !std::isfinite(scale) || !(scale > 0.0f))
        return CDG_ERR_INVALID_ARG;
    if (dtype == CDG_F32 || dim % 8 || dim > 128 || heads > kMaxHeads) return CDG_ERR_UNSUPPORTED;
    cdg_attention_st *h = new (std::nothrow) cdg_attention_st();
    if (!h) return CDG_ERR_CUDA;
    h->heads = heads; h->kv_heads = kv_heads; h->dim = dim; h->dtype = dtype;
    h->causal = causal; h->window = window; h->scale = scale;
    h->host_only = host_only;
    h->sms = host_only ? 152 : cdg::sm_count();
    if (!host_only) {
        if (h->sms < 1 || cudaGetDevice(&h->device) != cudaSuccess || cat_prepare_forward() != cudaSuccess || cat_prepare_grad() != cudaSuccess ||
            cudaMalloc(&h->d_status, sizeof(int)) != cudaSuccess || cudaMemset(h->d_status, 0, sizeof(int)) != cudaSuccess) {
            if (h->d_status) cudaFree(h->d_status);
            delete h;
            return CDG_ERR_CUDA;
        }
    }
    *out = h;
    return CDG_OK;
}

bool sizes_ok(const cdg_attention_st *h, long long q_tokens, long long k_tokens, int sequences)
{
    return h && q_tokens >= 0 && k_tokens >= 0 && q_tokens < kMaxTokens && k_tokens < kMaxTokens && sequences >= 1 &&
           sequences <= kMaxSequences;
}

// One matrix of a call: tokens x (heads * dim), row stride ld.
struct Matrix {
    const void *p;
    long long ld, tokens;
    int heads;
};

int check(const cdg_attention_st *h, std::initializer_list<Matrix> all)
{
    for (const Matrix &m : all) {
        if (m.tokens == 0) continue;
        if (!m.p || m.ld < static_cast<long long>(m.heads) * h->dim) return CDG_ERR_INVALID_ARG;
        if (m.ld >= (1ll << 31)) return CDG_ERR_UNSUPPORTED;
    }
    for (const Matrix &m : all)
        if (m.tokens > 0 && (!cdg::aligned_to(m.p, 16) || m.ld % 8)) return CDG_ERR_ALIGNMENT;
    return CDG_OK;
}

cdg::Rows rows(const cdg_attention_st *h, const Matrix &m)
{
    return cdg::Rows{m.p, m.tokens, static_cast<long long>(m.heads) * h->dim, m.ld, 2};
}
cdg::Extent extent(const cdg_attention_st *h, const Matrix &m) { return rows(h, m).extent(); }
bool overlap(const cdg_attention_st *h, const Matrix &a, const Matrix &b) { return cdg::overlap(rows(h, a), rows(h, b)); }

// dim x heads x tokens, boxes of 64 columns of one head x 128 tokens.
bool encode(const cdg_attention_st *h, CUtensorMap *map, const Matrix &m)
{
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    if (m.tokens == 0) {
        std::memset(map, 0, sizeof *map);  // of a side without rows: no load uses it
        return true;
    }
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(h->dim), static_cast<cuuint64_t>(m.heads), static_cast<cuuint64_t>(m.tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(h->dim) * 2, static_cast<cuuint64_t>(m.ld) * 2};
    const cuuint32_t box[3] = {64, 1, CAT_TILE}, ones[3] = {1, 1, 1};
    return enc(map, h->dtype == CDG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
               const_cast<void *>(m.p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What every call has: sizes, offsets, heads.
int common(const cdg_attention_st *h, CatParams &p, long long q_tokens, long long k_tokens, const void *q_offsets,
           const void *k_offsets, int index_bytes, int sequences)
{
    if (!sizes_ok(h, q_tokens, k_tokens, sequences) || (index_bytes != 4 && index_bytes != 8) ||
        (sequences > 1 && (!q_offsets || !k_offsets)))
        return CDG_ERR_INVALID_ARG;
    if (!cdg::aligned_to(q_offsets, index_bytes) || !cdg::aligned_to(k_offsets, index_bytes)) return CDG_ERR_ALIGNMENT;
    std::memset(&p, 0, sizeof p);
    p.q_offsets = q_offsets;
    p.k_offsets = k_offsets;
    p.index_bytes = index_bytes;
    p.sequences = sequences;
    p.q_tokens = static_cast<int>(q_tokens);
    p.k_tokens = static_cast<int>(k_tokens);
    p.heads = h->heads;
    p.kv_heads = h->kv_heads;
    p.group = h->heads / h->kv_heads;
    p.dim = h->dim;
    p.slices = (h->dim + 63) / 64;
    p.ksteps = (h->dim + 15) / 16;
    p.causal = h->causal;
    // A window past the call's keys hides none of them: cut there, its sums with rows'
    // numbers (all below 2^30) stay inside 32 bits.
    p.window = std::min(h->window, std::max(1, p.k_tokens));
    p.scale = h->scale;
    p.scale_log2 = static_cast<float>(h->scale * 1.4426950408889634);
    // fp32 sums, operands of the type, N, M = 128; B of the second is MN-major (bit 16)
    const uint32_t ab = h->dtype == CDG_BF16 ? 1u : 0u, of = (1u << 4) | (ab << 7) | (ab << 10) | (static_cast<uint32_t>(CAT_TILE >> 4) << 24);
    p.idesc_qk = of | (static_cast<uint32_t>(CAT_TILE >> 3) << 17);
    p.idesc_pv = of | (1u << 16) | (static_cast<uint32_t>(2 * p.ksteps) << 17);
    p.status = h->d_status;
    return CDG_OK;
}

// Tiles of `rows` that sequences of `tokens` rows in all can have, times heads.
long long items(long long tokens, int sequences, int rows, int heads)
{
    return (tokens + (rows - 1) * std::min<long long>(sequences, tokens)) / rows * heads;
}

// Parts that the steps of `n` items are split into: until there is an item for
// every SM, but no part of fewer than four of an average item's `steps`.
int parts_of(long long n, long long steps, int sms)
{
    int parts = 1;
    while (n > 0 && n * parts < sms && steps >= 8ll * parts && parts < 32) parts *= 2;
    return parts;
}
// Tiles of the other side that a tile sees, on average: of sequences of `tokens`
// rows in all, within the window, half of them under a causal mask.
long long steps_of(const cdg_attention_st *h, long long tokens, int sequences)
{
    long long rows = tokens / sequences;
    if (h->causal) rows = (rows + 1) / 2;
    if (h->window) rows = std::min<long long>(rows, h->window);
    return (rows + CAT_TILE - 1) / CAT_TILE;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// The forward's workspace: o and lse of each part.
struct Workspace {
    int parts;
    size_t lse, bytes;
    Workspace(const cdg_attention_st *h, long long q_tokens, long long k_tokens, int sequences)
    {
        parts = parts_of(items(q_tokens, sequences, 2 * CAT_TILE, h->heads), steps_of(h, k_tokens, sequences), h->sms);
        const size_t rows = static_cast<size_t>(parts) * q_tokens * h->heads * 4;
        lse = up256(rows * h->dim);
        bytes = parts > 1 ? lse + up256(rows) : 256;
    }
};

// The gradient's: the rows' statistics, fp16's sizes, then the sums of the parts of dq, and of dk and dv.
struct GradWorkspace {
    int q_parts, k_parts;
    long long stat_ctas, size_ctas;
    size_t sizes, dq, dkv, bytes;
    GradWorkspace(const cdg_attention_st *h, long long q_tokens, long long k_tokens, int sequences)
    {
        q_parts = parts_of(items(q_tokens, sequences, CAT_TILE, h->heads), steps_of(h, k_tokens, sequences), h->sms);
        k_parts = parts_of(items(k_tokens, sequences, CAT_TILE, h->kv_heads), h->heads / h->kv_heads * steps_of(h, q_tokens, sequences), h->sms);
        sizes = up256(static_cast<size_t>(q_tokens) * h->heads * sizeof(float2));
        stat_ctas = cat_stat_ctas(q_tokens, h->heads, h->dtype == CDG_BF16);
        size_ctas = h->dtype == CDG_F16 ? cat_stat_ctas(k_tokens, h->kv_heads, 0) : 0;
        dq = sizes + (h->dtype == CDG_F16 ? up256(static_cast<size_t>(stat_ctas + size_ctas) * sizeof(uint4)) : 0);
        dkv = dq + (q_parts > 1 ? up256(static_cast<size_t>(q_parts) * q_tokens * h->heads * h->dim * 4) : 0);
        bytes = dkv + (k_parts > 1 ? up256(2ull * k_parts * k_tokens * h->kv_heads * h->dim * 4) : 0);
        bytes = std::max<size_t>(256, bytes);
    }
};

int usable(const cdg_attention_st *h)
{
    if (!h) return CDG_ERR_INVALID_ARG;
    if (h->host_only) return CDG_ERR_NO_DEVICE;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return CDG_ERR_CUDA;
    return dev == h->device ? CDG_OK : CDG_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

int cdg_attention_plan(int heads, int kv_heads, int dim, int dtype, int causal, int window, float scale, cdg_attention_t *out)
{
    return make_attention_plan(heads, kv_heads, dim, dtype, causal, window, scale, false, out);
}

int cdg_attention_plan_host(int heads, int kv_heads, int dim, int dtype, int causal, int window, float scale, cdg_attention_t *out)
{
    return make_attention_plan(heads, kv_heads, dim, dtype, causal, window, scale, true, out);
}

void cdg_attention_destroy(cdg_attention_t h)
{
    if (!h) return;
    if (h->d_status) cudaFree(h->d_status);
    delete h;
}

size_t cdg_attention_workspace_bytes(cdg_attention_t h, long long q_tokens, long long k_tokens, int sequences)
{
    return sizes_ok(h, q_tokens, k_tokens, sequences) ? Workspace(h, q_tokens, k_tokens, sequences).bytes : 0;
}

size_t cdg_attention_grad_workspace_bytes(cdg_attention_t h, long long q_tokens, long long k_tokens, int sequences)
{
    return sizes_ok(h, q_tokens, k_tokens, sequences) ? GradWorkspace(h, q_tokens, k_tokens, sequences).bytes : 0;
}

int cdg_attention(cdg_attention_t h, const void *q, long long ld_q, const void *k, long long ld_k, const void *v, long long ld_v,
                  long long q_tokens, long long k_tokens, const void *q_offsets, const void *k_offsets, int index_bytes,
                  int sequences, void *o, long long ld_o, float *lse, void *workspace, cdg_stream_t stream)
{
    using namespace cdg;
    if (!h) return CDG_ERR_INVALID_ARG;
    CatParams p;
    int rc = common(h, p, q_tokens, k_tokens, q_offsets, k_offsets, index_bytes, sequences);
    if (rc != CDG_OK) return rc;
    const Matrix mq{q, ld_q, q_tokens, h->heads}, mk{k, ld_k, k_tokens, h->kv_heads}, mv{v, ld_v, k_tokens, h->kv_heads},
        mo{o, ld_o, q_tokens, h->heads};
    if ((rc = check(h, {mq, mk, mv, mo})) != CDG_OK) return rc;
    if (!workspace || (q_tokens > 0 && !lse)) return CDG_ERR_INVALID_ARG;
    if (!aligned_to(lse, 4) || !aligned_to(workspace, 256)) return CDG_ERR_ALIGNMENT;
    const Extent l = cdg::extent(lse, static_cast<size_t>(q_tokens) * h->heads * 4),
                 w = cdg::extent(workspace, cdg_attention_workspace_bytes(h, q_tokens, k_tokens, sequences)),
                 offs[2] = {cdg::extent(q_offsets, static_cast<size_t>(sequences + 1) * index_bytes),
                            cdg::extent(k_offsets, static_cast<size_t>(sequences + 1) * index_bytes)};
    for (const Matrix &m : {mq, mk, mv})
        if (overlap(h, mo, m) || cdg::overlap(::extent(h, m), l) || cdg::overlap(::extent(h, m), w)) return CDG_ERR_ALIAS;
    const Extent eo = ::extent(h, mo);
    if (cdg::overlap(eo, l) || cdg::overlap(eo, w) || cdg::overlap(l, w)) return CDG_ERR_ALIAS;
    for (const Extent &f : offs)
        if (cdg::overlap(f, eo) || cdg::overlap(f, l) || cdg::overlap(f, w)) return CDG_ERR_ALIAS;
    if ((rc = usable(h)) != CDG_OK) return rc;
    if (q_tokens == 0) return CDG_OK;
    if (!encode(h, &p.tmQ, mq) || !encode(h, &p.tmK, mk) || !encode(h, &p.tmV, mv)) return CDG_ERR_CUDA;
    p.o = o;
    p.ld_o = ld_o;
    p.lse = lse;
    const Workspace ws(h, q_tokens, k_tokens, sequences);
    p.q_splits = ws.parts;
    p.q_partial = static_cast<float *>(workspace);
    p.lse_partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + ws.lse);
    const long long n = items(q_tokens, sequences, 2 * CAT_TILE, h->heads);
    if (n * p.q_splits >= (1ll << 31)) return CDG_ERR_UNSUPPORTED;
    // (few items are split, so that a join has few CTAs too)
    const long long joins = items(q_tokens, sequences, CAT_JOIN_ROWS, h->heads);
    return cat_launch_forward(p, h->dtype == CDG_BF16, n, joins, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CDG_OK : CDG_ERR_CUDA;
}

int cdg_attention_grad(cdg_attention_t h, const void *q, long long ld_q, const void *k, long long ld_k, const void *v,
                       long long ld_v, const void *o, long long ld_o, const float *lse, const void *d_o, long long ld_do,
                       long long q_tokens, long long k_tokens, const void *q_offsets, const void *k_offsets, int index_bytes,
                       int sequences, void *dq, long long ld_dq, void *dk, long long ld_dk, void *dv, long long ld_dv,
                       void *workspace, cdg_stream_t stream)
{
    using namespace cdg;
    if (!h) return CDG_ERR_INVALID_ARG;
    CatParams p;
    int rc = common(h, p, q_tokens, k_tokens, q_offsets, k_offsets, index_bytes, sequences);
    if (rc != CDG_OK) return rc;
    const Matrix mq{q, ld_q, q_tokens, h->heads}, mk{k, ld_k, k_tokens, h->kv_heads}, mv{v, ld_v, k_tokens, h->kv_heads},
        mo{o, ld_o, q_tokens, h->heads}, md{d_o, ld_do, q_tokens, h->heads};
    const Matrix out[3] = {{dq, ld_dq, q_tokens, h->heads}, {dk, ld_dk, k_tokens, h->kv_heads}, {dv, ld_dv, k_tokens, h->kv_heads}};
    if ((rc = check(h, {mq, mk, mv, mo, md, out[0], out[1], out[2]})) != CDG_OK) return rc;
    if (!workspace || (q_tokens > 0 && !lse)) return CDG_ERR_INVALID_ARG;
    if (!aligned_to(lse, 4) || !aligned_to(workspace, 256)) return CDG_ERR_ALIGNMENT;
    const Extent l = cdg::extent(lse, static_cast<size_t>(q_tokens) * h->heads * 4),
                 w = cdg::extent(workspace, cdg_attention_grad_workspace_bytes(h, q_tokens, k_tokens, sequences)),
                 offs[2] = {cdg::extent(q_offsets, static_cast<size_t>(sequences + 1) * index_bytes),
                            cdg::extent(k_offsets, static_cast<size_t>(sequences + 1) * index_bytes)};
    for (const Matrix &m : {mq, mk, mv, mo, md}) {
        for (const Matrix &g : out)
            if (overlap(h, g, m)) return CDG_ERR_ALIAS;
        if (cdg::overlap(::extent(h, m), w)) return CDG_ERR_ALIAS;
    }
    if (overlap(h, out[0], out[1]) || overlap(h, out[0], out[2]) || overlap(h, out[1], out[2])) return CDG_ERR_ALIAS;
    for (const Matrix &g : out) {
        const Extent e = ::extent(h, g);
        if (cdg::overlap(e, l) || cdg::overlap(e, w) || cdg::overlap(e, offs[0]) || cdg::overlap(e, offs[1])) return CDG_ERR_ALIAS;
    }
    if (cdg::overlap(l, w) || cdg::overlap(w, offs[0]) || cdg::overlap(w, offs[1])) return CDG_ERR_ALIAS;
    if ((rc = usable(h)) != CDG_OK) return rc;
    if (!encode(h, &p.tmQ, mq) || !encode(h, &p.tmK, mk) || !encode(h, &p.tmV, mv) || !encode(h, &p.tmDO, md)) return CDG_ERR_CUDA;
    p.dq = dq; p.ld_dq = ld_dq;
    p.dk = dk; p.ld_dk = ld_dk;
    p.dv = dv; p.ld_dv = ld_dv;
    p.o_in = o; p.ld_oi = ld_o;
    p.d_o = d_o; p.ld_do = ld_do;
    p.lse_in = lse;
    const GradWorkspace ws(h, q_tokens, k_tokens, sequences);
    p.stats = static_cast<float2 *>(workspace);
    p.v_in = v; p.ld_v = ld_v;
    p.sizes = reinterpret_cast<uint4 *>(static_cast<char *>(workspace) + ws.sizes);
    p.stat_ctas = static_cast<int>(ws.stat_ctas);
    p.size_ctas = static_cast<int>(ws.size_ctas);
    p.q_splits = ws.q_parts;
    p.k_splits = ws.k_parts;
    p.q_partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + ws.dq);
    p.k_partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + ws.dkv);
    const int bf16 = h->dtype == CDG_BF16;
    const long long nq = items(q_tokens, sequences, CAT_TILE, h->heads), nk = items(k_tokens, sequences, CAT_TILE, h->kv_heads);
    if (nq * p.q_splits >= (1ll << 31) || nk * p.k_splits >= (1ll << 31) || q_tokens * h->heads >= (1ll << 34)) return CDG_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (q_tokens > 0 && cat_launch_stats(p, bf16, s) != cudaSuccess) return CDG_ERR_CUDA;
    if (k_tokens > 0 && cat_launch_dkv(p, bf16, nk, s) != cudaSuccess) return CDG_ERR_CUDA;
    if (q_tokens > 0 && cat_launch_dq(p, bf16, nq, s) != cudaSuccess) return CDG_ERR_CUDA;
    if (cat_launch_grad_join(p, bf16, items(k_tokens, sequences, CAT_JOIN_ROWS, h->kv_heads), items(q_tokens, sequences, CAT_JOIN_ROWS, h->heads),
                             s) != cudaSuccess)
        return CDG_ERR_CUDA;
    return CDG_OK;
}

int cdg_attention_device_status(cdg_attention_t h, cdg_stream_t stream)
{
    if (!h) return CDG_ERR_INVALID_ARG;
    if (h->host_only) return CDG_ERR_NO_DEVICE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int v = 0;
    if (cudaMemcpyAsync(&v, h->d_status, sizeof v, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return CDG_ERR_CUDA;
    if (v != 0 && (cudaMemsetAsync(h->d_status, 0, sizeof(int), s) != cudaSuccess ||
                   cudaStreamSynchronize(s) != cudaSuccess))
        return CDG_ERR_CUDA;
    return v;
}

}  // extern "C"
