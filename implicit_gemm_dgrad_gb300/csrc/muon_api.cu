// C-ABI of the orthogonalised weight update: validation, planning, tensor maps
// and launches; the kernels are in muon_sm103.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "../../include/cdg.h"
#include "muon_params.h"
#include "token_device.cuh"

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime's driver entry point (no -lcuda
// symbol needed at link time).
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

// What the iteration does to a singular value x in [0, 1] (a grid of them):
// whether it stays within the bounds of cdg_muon_plan, and within those of the
// Gram form's fp16 operands (see iterate_kernel: A, Q and T times 1024, P times
// 32; P's size is also what multiplies the rounding of A).
struct Bounds {
    bool iteration, gram;
};
Bounds iteration_bounds(int steps, double a, double b, double c)
{
    Bounds ok{true, true};
    const int kPoints = 8192;
    for (int i = 0; i <= kPoints; ++i) {
        double x = static_cast<double>(i) / kPoints, p = 1.0;
        for (int s = 0; s < steps; ++s) {
            const double x2 = x * x, poly = b * x2 + c * x2 * x2, q = a + poly;
            if (!(std::fabs(poly) <= 60.0)) ok.iteration = false;
            x *= q;
            p *= q;
            if (!(std::fabs(x) <= 4.0)) ok.iteration = false;
            if (!ok.iteration) return Bounds{false, false};
            if (std::fabs(q) > 32.0 || std::fabs(q) * x2 > 32.0 || std::fabs(p) > 1000.0) ok.gram = false;
        }
    }
    return ok;
}

// Cycles a block of K takes a 256 x 256 tile of a CTA pair and a 128 x 128 tile
// of one CTA (measured: the one near the tensor cores' rate, the other at the 64
// bytes a cycle an SM loads).
constexpr int kPairCycles = 630, kSquareCycles = 512;
// Ranges of K the Gram form's X X^T is cut into, at most.
constexpr int kMaxSplits = 8;
// Blocks of K a split tile's CTA takes at least (512 x 4608: 207 us with 4, 196 us with
// 16, 232 us unsplit; 256 x 1024: 127 us with 4, 112 us unsplit).
constexpr int kMinRange = 16;

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

struct cdg_muon_st {
    int batch, rows, cols, dtype, steps, transposed, m, n, pitch_x, pitch_a, partials, gram, splits, sms;
    float a, b, c, eps;
    bool host_only;
    int *d_status;
    size_t ws_bytes;
    // byte offsets in the workspace
    size_t x[2][2], mat[2], poly[2], diag, partial, sums, xs;  // x[buffer][part], mat[part], poly[part]
    const void *cached_ws;
    CUtensorMap x_rows[2][2], x_cols[2][2], mat_rows[2], poly_rows[2], mat_cols[2], poly_cols[2];
    cdg_muon_info_t info;
};

namespace {

// num_sms = 0: this device's.  Arguments are checked before the device is asked.
int make_muon_plan(int batch, int rows, int cols, int dtype, int steps, float a, float b, float c, float eps,
                   int num_sms, bool host_only, cdg_muon_t *out)
{
    if (!out) return CDG_ERR_INVALID_ARG;
    *out = nullptr;
    if (batch < 1 || rows < 1 || cols < 1 || (dtype != CDG_F16 && dtype != CDG_BF16 && dtype != CDG_F32) || steps < 1 ||
        steps > 32 || !std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c) || !std::isfinite(eps) ||
        eps < 0.0f || num_sms < (host_only ? 1 : 0))
        return CDG_ERR_INVALID_ARG;
    const Bounds bounds = iteration_bounds(steps, a, b, c);
    if (!bounds.iteration) return CDG_ERR_INVALID_ARG;
    const int m = std::min(rows, cols), n = std::max(rows, cols);
    if (batch > 65535 || m > 32768 || n > (1 << 21)) return CDG_ERR_UNSUPPORTED;
    if (!host_only && (num_sms = cdg::sm_count()) < 1) return CDG_ERR_CUDA;
    cdg_muon_st *h = new (std::nothrow) cdg_muon_st();
    if (!h) return CDG_ERR_CUDA;
    h->batch = batch; h->rows = rows; h->cols = cols; h->dtype = dtype; h->steps = steps;
    h->a = a; h->b = b; h->c = c; h->eps = eps;
    h->host_only = host_only;
    h->transposed = rows > cols;
    h->m = m;
    h->n = n;
    h->pitch_x = (n + 7) / 8 * 8;
    h->pitch_a = (m + 7) / 8 * 8;
    const long long per = static_cast<long long>(rows) * cols;
    h->partials = static_cast<int>(std::max(1ll, std::min<long long>({(per + 2047) / 2048, CMU_MAX_PARTIALS,
                                                                      std::max(1ll, 8ll * num_sms / batch)})));
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t was = at;
        at += up256(bytes);
        return was;
    };
    const size_t nb = static_cast<size_t>(batch);
    const size_t xb = nb * m * h->pitch_x * 2, ab = nb * m * h->pitch_a * 2;
    // an fp32 plan keeps fp32 accuracy, in both calls; the Gram form does not have it
    h->gram = m <= CMU_SIDE && bounds.gram && dtype != CDG_F32;
    h->splits = std::min((n + CMU_BK - 1) / CMU_BK, kMaxSplits);
    h->sms = num_sms;
    // low parts of A and B: three products for one (fp32 updates, and small matrices without the Gram form), or P's
    const bool low = dtype == CDG_F32 || m <= CMU_SIDE;
    for (int i = 0; i < 2; ++i)
        for (int q = 0; q < 2; ++q) h->x[i][q] = take(xb);
    for (int q = 0; q < 2; ++q) {
        h->mat[q] = q == 0 || low ? take(ab) : h->mat[0];
        h->poly[q] = q == 0 || low ? take(ab) : h->poly[0];
    }
    h->diag = take(nb * m * 4);
    h->partial = take(nb * CMU_MAX_PARTIALS * 4);
    h->xs = take(nb * 4);
    h->sums = h->gram ? take(nb * h->splits * CMU_SIDE * CMU_SIDE * 4) : 0;
    h->ws_bytes = at;
    h->info.m = m;
    h->info.n = n;
    h->info.transposed = h->transposed;
    h->info.gram = h->gram;
    h->info.launches = h->gram ? 5 : 2 + 3 * steps;
    if (!host_only) {
        if (cmu_prepare_kernels() != cudaSuccess || cudaMalloc(&h->d_status, sizeof(int)) != cudaSuccess ||
            cudaMemset(h->d_status, 0, sizeof(int)) != cudaSuccess) {
            if (h->d_status) cudaFree(h->d_status);
            delete h;
            return CDG_ERR_CUDA;
        }
    }
    *out = h;
    return CDG_OK;
}

// rows x cols fp16 matrices of a batch, boxes of 64 columns x box_rows rows.
bool encode(CUtensorMap *map, void *p, int cols, int rows, int batch, int pitch, int box_rows)
{
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(batch)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch) * 2, static_cast<cuuint64_t>(pitch) * rows * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1}, ones[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, p, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int encode_maps(cdg_muon_st *h, void *workspace)
{
    if (workspace == h->cached_ws) return CDG_OK;
    char *ws = static_cast<char *>(workspace);
    bool ok = true;
    for (int q = 0; q < 2; ++q) {
        for (int i = 0; i < 2; ++i) {
            ok = ok && encode(&h->x_rows[i][q], ws + h->x[i][q], h->n, h->m, h->batch, h->pitch_x, 128);
            ok = ok && encode(&h->x_cols[i][q], ws + h->x[i][q], h->n, h->m, h->batch, h->pitch_x, 64);
        }
        ok = ok && encode(&h->mat_rows[q], ws + h->mat[q], h->m, h->m, h->batch, h->pitch_a, 128);
        ok = ok && encode(&h->poly_rows[q], ws + h->poly[q], h->m, h->m, h->batch, h->pitch_a, 128);
        ok = ok && encode(&h->mat_cols[q], ws + h->mat[q], h->m, h->m, h->batch, h->pitch_a, 64);
        ok = ok && encode(&h->poly_cols[q], ws + h->poly[q], h->m, h->m, h->batch, h->pitch_a, 64);
    }
    if (!ok) return CDG_ERR_CUDA;
    h->cached_ws = workspace;
    return CDG_OK;
}

// The form of a product of M x N outputs over K (maps of 128-row and of 64-row
// boxes of the B operand for both): of CTA pairs and square tiles the one whose
// waves take fewer cycles (2048 x 2048 all in pairs: 303 us, in squares: 282;
// 3000 x 3000: 724 and 876), and narrow tiles where square ones would occupy at
// most half of the SMs, with K split until all SMs work or a range is down to
// kMinRange blocks.
void choose_form(CmuGemm &g, bool precise, int sms, const CUtensorMap *b128, const CUtensorMap *b64)
{
    const bool sym = g.mode <= CMU_POLY;
    auto tiles = [&](int side) {
        const long long tm = (g.M + side - 1) / side, tn = (g.N + side - 1) / side;
        return (sym ? tm * (tm + 1) / 2 : tm * tn) * g.batch;
    };
    const long long t128 = tiles(128), t256 = tiles(256);
    const long long waves128 = (t128 + sms - 1) / sms, waves256 = (t256 + sms / 2 - 1) / std::max(1, sms / 2);
    const bool pair = !precise && sms >= 2 && waves256 * kPairCycles < waves128 * kSquareCycles;
    g.form = pair ? CMU_PAIR : 2 * t128 <= sms ? CMU_NARROW : CMU_SQUARE;
    g.split = 1;
    const int blocks = (g.K + CMU_BK - 1) / CMU_BK;
    if (g.form == CMU_NARROW)
        while (g.split < 8 && 2 * t128 * g.split * 2 <= sms && blocks / (2 * g.split) >= kMinRange) g.split *= 2;
    for (int q = 0; q < 2; ++q) g.tmB[q] = g.form == CMU_NARROW ? b64[q] : b128[q];
}

struct Final {
    void *out;
    int out_type;
    const float *w_in;
    float w_keep, w_step;
};

// The norm, the first X and the products; the last one writes `out`.
int run(cdg_muon_st *h, CmuPrepare p, const Final &f, void *workspace, cudaStream_t s)
{
    const int rc = encode_maps(h, workspace);
    if (rc != CDG_OK) return rc;
    char *ws = static_cast<char *>(workspace);
    auto at16 = [&](size_t off) { return reinterpret_cast<uint16_t *>(ws + off); };
    p.batch = h->batch; p.rows = h->rows; p.cols = h->cols; p.dtype = h->dtype; p.transposed = h->transposed;
    p.partials = h->partials;
    p.eps = h->eps;
    p.partial = reinterpret_cast<float *>(ws + h->partial);
    p.xs = reinterpret_cast<float *>(ws + h->xs);
    p.x_hi = at16(h->x[0][0]);
    p.x_lo = at16(h->x[0][1]);
    p.pitch_x = h->pitch_x;
    const bool precise = h->dtype == CDG_F32, gram = h->gram;
    const int parts = precise || h->m <= CMU_SIDE ? 3 : 1;
    p.has_lo = p.nesterov >= 0 || precise || (parts == 3 && !gram);
    if (cmu_launch_norm(p, s) != cudaSuccess || cmu_launch_split(p, s) != cudaSuccess) return CDG_ERR_CUDA;
    CmuGemm g;
    std::memset(&g, 0, sizeof g);
    g.batch = h->batch;
    g.xs = p.xs;
    g.parts = parts;
    g.poly_scale = CMU_SCALE;
    g.diag = reinterpret_cast<float *>(ws + h->diag);
    g.a = h->a; g.b = h->b; g.c = h->c;
    g.out = f.out; g.out_type = f.out_type; g.w_in = f.w_in; g.w_keep = f.w_keep; g.w_step = f.w_step;
    g.transposed = h->transposed; g.rows = h->rows; g.cols = h->cols;
    g.status = h->d_status;
    if (gram) {
        g.first = 1;
        g.has_lo = p.has_lo;
        g.M = g.N = h->m;
        g.K = h->n;
        g.mode = CMU_PARTIAL;
        g.form = CMU_SQUARE;
        g.split = 1;
        g.parts = p.has_lo ? 3 : 1;
        g.tiles = h->splits;
        g.partial = reinterpret_cast<float *>(ws + h->sums);
        for (int q = 0; q < 2; ++q) {
            g.tmA[q] = g.tmB[q] = g.tmE[q] = h->x_rows[0][q];
            g.tmY[q] = h->x_rows[1][q];
            g.tmT[q] = h->mat_cols[q];
        }
        if (cmu_launch_gemm(g, h->sms, s) != cudaSuccess) return CDG_ERR_CUDA;
        const CmuIterate it{h->batch, h->m, h->steps, h->splits, h->pitch_a, h->a, h->b, h->c, g.partial, g.xs,
                            at16(h->poly[0]), at16(h->poly[1]), g.diag, h->d_status};
        if (cmu_launch_iterate(it, s) != cudaSuccess) return CDG_ERR_CUDA;
        g.mode = CMU_FINAL;
        g.parts = p.has_lo ? 3 : 2;
        g.a = 0.0f;
        g.poly_scale = CMU_POLY_SCALE;
        g.N = h->n;
        g.K = h->m;
        for (int q = 0; q < 2; ++q) g.tmA[q] = h->poly_rows[q];
        choose_form(g, true, h->sms, h->x_cols[0], h->x_cols[0]);
        return cmu_launch_gemm(g, h->sms, s) == cudaSuccess ? CDG_OK : CDG_ERR_CUDA;
    }
    for (int k = 0; k < h->steps; ++k) {
        const int cur = k & 1;
        g.first = k == 0;
        g.has_lo = k > 0 || p.has_lo;
        g.mode = CMU_GRAM;
        g.M = g.N = h->m;
        g.K = h->n;
        for (int q = 0; q < 2; ++q) {
            g.tmA[q] = g.tmE[q] = h->x_rows[cur][q];
            g.tmY[q] = h->mat_rows[q];
            g.tmT[q] = h->mat_cols[q];
        }
        choose_form(g, parts != 1, h->sms, h->x_rows[cur], h->x_cols[cur]);
        if (cmu_launch_gemm(g, h->sms, s) != cudaSuccess) return CDG_ERR_CUDA;
        g.mode = CMU_POLY;
        g.K = h->m;
        for (int q = 0; q < 2; ++q) {
            g.tmA[q] = g.tmE[q] = h->mat_rows[q];
            g.tmY[q] = h->poly_rows[q];
            g.tmT[q] = h->poly_cols[q];
        }
        choose_form(g, parts != 1, h->sms, h->mat_rows, h->mat_cols);
        if (cmu_launch_gemm(g, h->sms, s) != cudaSuccess) return CDG_ERR_CUDA;
        g.mode = k == h->steps - 1 ? CMU_FINAL : CMU_UPDATE;
        g.N = h->n;
        for (int q = 0; q < 2; ++q) {
            g.tmA[q] = h->poly_rows[q];
            g.tmE[q] = h->x_rows[cur][q];
            g.tmY[q] = h->x_rows[cur ^ 1][q];
        }
        choose_form(g, parts != 1, h->sms, h->x_cols[cur], h->x_cols[cur]);
        if (cmu_launch_gemm(g, h->sms, s) != cudaSuccess) return CDG_ERR_CUDA;
    }
    return CDG_OK;
}

}  // namespace

extern "C" {

int cdg_muon_plan(int batch, int rows, int cols, int dtype, int steps, float a, float b, float c, float eps,
                  cdg_muon_t *out)
{
    return make_muon_plan(batch, rows, cols, dtype, steps, a, b, c, eps, 0, false, out);
}

int cdg_muon_plan_host(int batch, int rows, int cols, int dtype, int steps, float a, float b, float c, float eps,
                       int num_sms, cdg_muon_t *out)
{
    return make_muon_plan(batch, rows, cols, dtype, steps, a, b, c, eps, num_sms, true, out);
}

void cdg_muon_destroy(cdg_muon_t h)
{
    if (!h) return;
    if (h->d_status) cudaFree(h->d_status);
    delete h;
}

size_t cdg_muon_workspace_bytes(cdg_muon_t h) { return h ? h->ws_bytes : 0; }

int cdg_muon_get_info(cdg_muon_t h, cdg_muon_info_t *info)
{
    if (!h || !info) return CDG_ERR_INVALID_ARG;
    *info = h->info;
    return CDG_OK;
}

int cdg_muon_orthogonalize(cdg_muon_t h, const void *U, void *O, void *workspace, cdg_stream_t stream)
{
    using namespace cdg;
    if (!h || !U || !O || !workspace) return CDG_ERR_INVALID_ARG;
    if (h->host_only) return CDG_ERR_NO_DEVICE;
    if (!aligned_to(U, 16) || !aligned_to(O, 16) || !aligned_to(workspace, 256)) return CDG_ERR_ALIGNMENT;
    const size_t n = static_cast<size_t>(h->batch) * h->rows * h->cols * dtype_bytes(h->dtype);
    const Extent u = extent(U, n), o = extent(O, n), w = extent(workspace, h->ws_bytes);
    if (overlap(u, o) || overlap(u, w) || overlap(o, w)) return CDG_ERR_ALIAS;
    CmuPrepare p;
    std::memset(&p, 0, sizeof p);
    p.nesterov = -1;
    p.u = U;
    const Final f{O, h->dtype == CDG_F32 ? CDG_T_F32 : h->dtype == CDG_BF16 ? CDG_T_BF16 : CDG_T_F16, nullptr, 0.0f, 0.0f};
    return run(h, p, f, workspace, static_cast<cudaStream_t>(stream));
}

int cdg_muon_step(cdg_muon_t h, const float *W, const void *G, const float *M, float *W_out, float *M_out, float lr,
                  float momentum, float weight_decay, float update_scale, int nesterov, void *workspace,
                  cdg_stream_t stream)
{
    using namespace cdg;
    if (!h || !W || !G || !M || !W_out || !M_out || !workspace || !std::isfinite(lr) || !std::isfinite(momentum) ||
        !std::isfinite(weight_decay) || !std::isfinite(update_scale) || (nesterov != 0 && nesterov != 1))
        return CDG_ERR_INVALID_ARG;
    if (h->host_only) return CDG_ERR_NO_DEVICE;
    for (const void *q : {static_cast<const void *>(W), G, static_cast<const void *>(M), static_cast<const void *>(W_out),
                          static_cast<const void *>(M_out)})
        if (!aligned_to(q, 16)) return CDG_ERR_ALIGNMENT;
    if (!aligned_to(workspace, 256)) return CDG_ERR_ALIGNMENT;
    const size_t n = static_cast<size_t>(h->batch) * h->rows * h->cols;
    const Extent w = extent(W, n * 4), g = extent(G, n * dtype_bytes(h->dtype)), m = extent(M, n * 4),
                 wo = extent(W_out, n * 4), mo = extent(M_out, n * 4), ws = extent(workspace, h->ws_bytes);
    if ((W_out != W && overlap(wo, w)) || (M_out != M && overlap(mo, m)) || overlap(wo, g) || overlap(wo, m) ||
        overlap(wo, mo) || overlap(mo, g) || overlap(mo, w))
        return CDG_ERR_ALIAS;
    for (const Extent &e : {w, g, m, wo, mo})
        if (overlap(ws, e)) return CDG_ERR_ALIAS;
    CmuPrepare p;
    std::memset(&p, 0, sizeof p);
    p.nesterov = nesterov;
    p.momentum = momentum;
    p.u = G;
    p.m_in = M;
    p.m_out = M_out;
    const Final f{W_out, CDG_T_F32, W, static_cast<float>(1.0 - static_cast<double>(lr) * weight_decay),
                  static_cast<float>(static_cast<double>(lr) * update_scale)};
    return run(h, p, f, workspace, static_cast<cudaStream_t>(stream));
}

int cdg_muon_device_status(cdg_muon_t h, cdg_stream_t stream)
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
