// Norms of queries and keys with the position rotation: C entry points, and the
// forward kernels (rope_device.cuh).
#include "rope_device.cuh"

namespace cdg {
namespace {

// Rows of partial sums that launch_width may use, at most: a CTA a block of at
// least one head, or the share.
long long partial_rows(int heads, int kv_heads) { return kGradCtas + heads + kv_heads; }

struct RopeCall {
    long long tokens;
    int heads, kv_heads, dim, dtype, rot, interleaved, norm, index_bytes;
    float factor, eps;
    const float *inv_freq, *w_q, *w_k;
    const void *positions;
};

int check_call(const RopeCall &c)
{
    if (c.tokens < 0 || c.heads < 0 || c.kv_heads < 0 || c.heads + c.kv_heads < 1 || c.dim < 1 ||
        (c.dtype != CDG_F16 && c.dtype != CDG_BF16 && c.dtype != CDG_F32) || c.rot < 0 || c.rot > c.dim || c.rot % 2 ||
        (c.interleaved != 0 && c.interleaved != 1) || (c.norm != 0 && c.norm != 1) || (c.index_bytes != 4 && c.index_bytes != 8) ||
        !std::isfinite(c.factor) || !std::isfinite(c.eps) || c.eps < 0.0f || (c.rot > 0 && !c.inv_freq) ||
        (!c.norm && (c.w_q || c.w_k)))
        return CDG_ERR_INVALID_ARG;
    if (c.dim > kMaxHead || c.heads > kMaxHeads || c.kv_heads > kMaxHeads || c.tokens >= (1ll << 31)) return CDG_ERR_UNSUPPORTED;
    if (!aligned_to(c.inv_freq, 4) || !aligned_to(c.w_q, 4) || !aligned_to(c.w_k, 4) || !aligned_to(c.positions, c.index_bytes))
        return CDG_ERR_ALIGNMENT;
    return CDG_OK;
}

RopeArgs make_args(const RopeCall &c)
{
    RopeArgs a{};
    a.positions = c.positions;
    a.inv_freq = c.inv_freq;
    a.tokens = c.tokens;
    a.index_bytes = c.index_bytes;
    a.dim = c.dim;
    a.rot = c.rot;
    a.interleaved = c.interleaved;
    a.norm = c.norm;
    a.factor = c.factor;
    a.eps = c.eps;
    a.side[0].heads = c.heads;
    a.side[1].heads = c.kv_heads;
    a.side[0].w = c.w_q;
    a.side[1].w = c.w_k;
    return a;
}

int check_rows(const Rows &r)
{
    if (r.rows == 0 || r.width == 0) return CDG_OK;
    if (!r.p || r.ld < r.width) return CDG_ERR_INVALID_ARG;
    if (r.ld >= (1ll << 31)) return CDG_ERR_UNSUPPORTED;
    return aligned_to(r.p, r.esize) ? CDG_OK : CDG_ERR_ALIGNMENT;
}

// What a call reads beside its matrices.
struct SmallInputs {
    Extent e[4];
    SmallInputs(const RopeCall &c)
        : e{extent(c.inv_freq, c.rot / 2 * 4), extent(c.w_q, c.dim * 4), extent(c.w_k, c.dim * 4),
            extent(c.positions, static_cast<size_t>(c.tokens) * c.index_bytes)}
    {
    }
    bool meet(const Extent &x) const { return overlap(x, e[0]) || overlap(x, e[1]) || overlap(x, e[2]) || overlap(x, e[3]); }
};

bool same(const Rows &a, const Rows &b) { return a.p == b.p && a.ld == b.ld; }

}  // namespace
}  // namespace cdg

extern "C" {

int cdg_rope_frequencies(int rot, double base, double stretch, long long trained, double low, double high, float *inv_freq)
{
    if (rot < 0 || rot % 2 || rot > cdg::kMaxHead || !std::isfinite(base) || !(base > 0.0) || !std::isfinite(stretch) || !(stretch > 0.0) ||
        trained < 0 || (trained > 0 && !(low >= 0.0 && low < high && std::isfinite(high))) || (rot > 0 && !inv_freq))
        return CDG_ERR_INVALID_ARG;
    for (int i = 0; i < rot / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot);
        double keep = 0.0;
        if (trained > 0) {
            const double turns = static_cast<double>(trained) * f / 6.283185307179586;
            keep = std::min(1.0, std::max(0.0, (turns - low) / (high - low)));
        }
        inv_freq[i] = static_cast<float>(f * (keep + (1.0 - keep) / stretch));
    }
    return CDG_OK;
}

int cdg_qk_rope(const void *q, long long ld_q, const void *k, long long ld_k, const void *positions, int index_bytes,
                long long tokens, int heads, int kv_heads, int dim, int dtype, const float *inv_freq, int rot, int interleaved,
                float factor, int norm, float eps, const float *w_q, const float *w_k, void *q_out, long long ld_qo, void *k_out,
                long long ld_ko, cdg_stream_t stream)
{
    using namespace cdg;
    const RopeCall c{tokens, heads, kv_heads, dim, dtype, rot, interleaved, norm, index_bytes, factor, eps, inv_freq, w_q, w_k, positions};
    int rc = check_call(c);
    if (rc != CDG_OK) return rc;
    const int es = dtype_bytes(dtype);
    const long long wq = static_cast<long long>(heads) * dim, wk = static_cast<long long>(kv_heads) * dim;
    const Rows in[2] = {{q, tokens, wq, ld_q, es}, {k, tokens, wk, ld_k, es}};
    const Rows out[2] = {{q_out, tokens, wq, ld_qo, es}, {k_out, tokens, wk, ld_ko, es}};
    for (const Rows &r : {in[0], in[1], out[0], out[1]})
        if ((rc = check_rows(r)) != CDG_OK) return rc;
    const SmallInputs small(c);
    for (int i = 0; i < 2; ++i) {
        if (out[i].width == 0) continue;
        if ((in[i].width && !same(out[i], in[i]) && overlap(out[i], in[i])) || (in[1 - i].width && overlap(out[i], in[1 - i])) ||
            small.meet(out[i].extent()))
            return CDG_ERR_ALIAS;
    }
    if (wq && wk && overlap(out[0], out[1])) return CDG_ERR_ALIAS;
    if (tokens == 0) return CDG_OK;
    RopeArgs a = make_args(c);
    for (int i = 0; i < 2; ++i) {
        a.side[i].x = in[i].p;
        a.side[i].ld_x = in[i].ld;
        a.side[i].out = const_cast<void *>(out[i].p);
        a.side[i].ld_out = out[i].ld;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == CDG_F32   ? launch_rope<float, false>(a, s)
                          : dtype == CDG_F16 ? launch_rope<__half, false>(a, s)
                                             : launch_rope<__nv_bfloat16, false>(a, s);
    return e == cudaSuccess ? CDG_OK : CDG_ERR_CUDA;
}

size_t cdg_qk_rope_grad_workspace_bytes(long long tokens, int heads, int kv_heads, int dim)
{
    if (tokens < 0 || tokens >= (1ll << 31) || heads < 0 || kv_heads < 0 || heads > cdg::kMaxHeads || kv_heads > cdg::kMaxHeads || heads + kv_heads < 1 ||
        dim < 1 || dim > cdg::kMaxHead)
        return 0;
    return static_cast<size_t>(cdg::partial_rows(heads, kv_heads)) * dim * 4;
}

int cdg_qk_rope_grad(const void *q, long long ld_q, const void *k, long long ld_k, const void *positions, int index_bytes,
                     long long tokens, int heads, int kv_heads, int dim, int dtype, const float *inv_freq, int rot,
                     int interleaved, float factor, int norm, float eps, const float *w_q, const float *w_k, const void *dq_out,
                     long long ld_dqo, const void *dk_out, long long ld_dko, void *dq, long long ld_dq, void *dk, long long ld_dk,
                     float *dw_q, float *dw_k, void *workspace, cdg_stream_t stream)
{
    using namespace cdg;
    const RopeCall c{tokens, heads, kv_heads, dim, dtype, rot, interleaved, norm, index_bytes, factor, eps, inv_freq, w_q, w_k, positions};
    int rc = check_call(c);
    if (rc != CDG_OK) return rc;
    if ((!norm && (dw_q || dw_k)) || !workspace) return CDG_ERR_INVALID_ARG;
    const int es = dtype_bytes(dtype);
    const long long wq = static_cast<long long>(heads) * dim, wk = static_cast<long long>(kv_heads) * dim;
    // (without the norm the inputs are not read)
    const Rows x[2] = {{q, tokens, norm ? wq : 0, ld_q, es}, {k, tokens, norm ? wk : 0, ld_k, es}};
    const Rows dy[2] = {{dq_out, tokens, wq, ld_dqo, es}, {dk_out, tokens, wk, ld_dko, es}};
    const Rows dx[2] = {{dq, tokens, wq, ld_dq, es}, {dk, tokens, wk, ld_dk, es}};
    for (const Rows &r : {x[0], x[1], dy[0], dy[1], dx[0], dx[1]})
        if ((rc = check_rows(r)) != CDG_OK) return rc;
    if (!aligned_to(workspace, 16) || !aligned_to(dw_q, 4) || !aligned_to(dw_k, 4)) return CDG_ERR_ALIGNMENT;
    const SmallInputs small(c);
    const Extent ws = extent(workspace, cdg_qk_rope_grad_workspace_bytes(tokens, heads, kv_heads, dim)),
                 dw[2] = {extent(dw_q, dim * 4), extent(dw_k, dim * 4)};
    auto used = [](const Rows &r) { return r.rows > 0 && r.width > 0; };
    for (int i = 0; i < 2; ++i) {
        if (!used(dx[i])) continue;
        for (int j = 0; j < 2; ++j) {
            if (used(x[j]) && overlap(dx[i], x[j])) return CDG_ERR_ALIAS;
            if (used(dy[j]) && !(i == j && same(dx[i], dy[j])) && overlap(dx[i], dy[j])) return CDG_ERR_ALIAS;
        }
    }
    if (used(dx[0]) && used(dx[1]) && overlap(dx[0], dx[1])) return CDG_ERR_ALIAS;
    for (const Rows &r : {x[0], x[1], dy[0], dy[1], dx[0], dx[1]}) {
        if (!used(r)) continue;
        const Extent e = r.extent();
        if (overlap(e, ws) || overlap(e, dw[0]) || overlap(e, dw[1])) return CDG_ERR_ALIAS;
        if ((r.p == dq || r.p == dk) && small.meet(e)) return CDG_ERR_ALIAS;
    }
    if (small.meet(ws) || small.meet(dw[0]) || small.meet(dw[1]) || overlap(ws, dw[0]) || overlap(ws, dw[1]) || overlap(dw[0], dw[1]))
        return CDG_ERR_ALIAS;
    RopeArgs a = make_args(c);
    for (int i = 0; i < 2; ++i) {
        a.side[i].x = x[i].p;
        a.side[i].ld_x = x[i].ld;
        a.side[i].dy = dy[i].p;
        a.side[i].ld_dy = dy[i].ld;
        a.side[i].out = const_cast<void *>(dx[i].p);
        a.side[i].ld_out = dx[i].ld;
    }
    a.side[0].dw = dw_q;
    a.side[1].dw = dw_k;
    a.partial = static_cast<float *>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = crp_launch_grad(a, dtype, s);
    return e == cudaSuccess ? CDG_OK : CDG_ERR_CUDA;
}

}  // extern "C"
