// Launch parameters shared by the host side (muon_api.cu) and the sm_103a
// kernels (muon_sm103.cu) of the orthogonalised weight update.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cdg_params.h"

// Fixed-point-like scales (powers of two) of the fp16 operands: X, A = X X^T
// and B = b A + c A^2 are stored times 1024, so that values of norm about 1
// keep their 11 bits down to 6e-8 of it.
#define CMU_SCALE 1024.0f
#define CMU_MAX_PARTIALS 512  // partial sums of squares a matrix
// A CTA's share of a stage: 128 rows of A and 128 rows (or columns) of B, 64 of K.
#define CMU_BK 64
#define CMU_STAGES 5
#define CMU_HALF_BYTES (128 * CMU_BK * 2)
#define CMU_STAGING_BYTES (2 * CMU_HALF_BYTES)  // per group of eight epilogue warps: 128 x 64 fp16, twice
#define CMU_BAR_BYTES 512
// Two-part products move their sums from tensor memory to registers after this
// many K blocks (see gemm_kernel); one-part products once.
#define CMU_CHAIN 2

// One batched product C[b] = opA[b] opB[b]^T over K, fp32 sums, and what its
// epilogue makes of it.
enum CmuMode {
    CMU_GRAM = 0,    // A = X X^T (symmetric)
    CMU_POLY = 1,    // B = b A + c A A^T (symmetric), its diagonal apart
    CMU_UPDATE = 2,  // X' = (a + diag B) X + (B - diag B) X
    CMU_FINAL = 3,   // the last update: O, or W
    CMU_PARTIAL = 4  // fp32 partial sums of X X^T over one of several ranges of K (one tile a matrix)
};

// Output tiles of a product: 256 x 256 by CTA pairs, 128 x 128, or 128 x 64
// with K split over the CTAs of a cluster.
enum CmuForm { CMU_PAIR = 0, CMU_SQUARE = 1, CMU_NARROW = 2 };

// The whole iteration of a matrix of up to 128 rows on its Gram matrix: see
// iterate_kernel.
#define CMU_SIDE 128
#define CMU_POLY_SCALE 32.0f  // P, whose eigenvalues reach a^steps, is stored times 32
struct CmuIterate {
    int batch, m, steps, splits, pitch_a;
    float a, b, c;
    const float *partial;  // [batch][splits][128][128]: X X^T, X times xs
    const float *xs;
    uint16_t *poly, *poly_lo;
    float *diag;
    int *status;
};

struct CmuGemm {
    // High and low parts of: the operands ({k, rows, batch}, boxes {64, 128, 1};
    // tmB of an update {n, k, batch}, boxes {64, 64, 1}), the epilogue's input
    // and its output (boxes {64, 128, 1}), and the output's mirror image
    // (symmetric products, boxes {64, 64, 1}).
    CUtensorMap tmA[2], tmB[2], tmE[2], tmY[2], tmT[2];
    int mode;
    int form;         // CMU_PAIR, CMU_SQUARE, CMU_NARROW
    int split;        // NARROW: CTAs of a cluster that share a tile's K
    int tiles_m, tiles;  // tiles along M; tiles (PARTIAL: ranges of K) a matrix
    int parts;        // 1: high x high; 2: and low x high before it; 3: and high x low between
    int M, N, K, batch;
    int first;        // X is still times xs[b] instead of CMU_SCALE
    int has_lo;       // X has a low part
    const float *xs;
    float *diag;      // diagonal of B, [batch][M]
    float *partial;   // PARTIAL: [batch][tiles][128][128]
    float a, b, c, poly_scale;  // poly_scale: B is stored times it
    // FINAL: O (dtype) or W_out; transposed: element (i, j) of X is element (j, i) of O
    int out_type, transposed, rows, cols;
    void *out;
    const float *w_in;
    float w_keep, w_step;  // W_out = w_keep W - w_step O
    int *status;
};

struct CmuPrepare {
    int batch, rows, cols, dtype, transposed, partials;
    int nesterov;         // -1: U itself; 0, 1: momentum
    float momentum, eps;
    const void *u;        // U or G
    const float *m_in;
    float *m_out;
    float *partial;       // [batch][CMU_MAX_PARTIALS]
    float *xs;            // [batch]
    uint16_t *x_hi, *x_lo;
    int pitch_x, has_lo;
};

cudaError_t cmu_prepare_kernels();
cudaError_t cmu_launch_norm(const CmuPrepare &p, cudaStream_t stream);
cudaError_t cmu_launch_split(const CmuPrepare &p, cudaStream_t stream);
cudaError_t cmu_launch_iterate(const CmuIterate &p, cudaStream_t stream);
cudaError_t cmu_launch_gemm(const CmuGemm &p, int sms, cudaStream_t stream);
