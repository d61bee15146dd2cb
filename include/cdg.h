/*
 * cdg.h -- Conv2d backward-data (dgrad) on one NVIDIA GB300 (sm_103a).
 *
 * The operation (apache/tvm PR #10110, "[CUTLASS] Conv2d dgrad", opening
 * description: "Conv2d dgrad"; the stride-2 case is the "strided dgrad" of the
 * benchmark comment on the same page):
 *
 *     dX[n,h,w,c] = sum over k, r, s and every (p, q) with
 *                   h = p*stride - pad + r*dil,  w = q*stride - pad + s*dil,
 *                   0 <= p < P, 0 <= q < Q,   of  dY[n,p,q,k] * W[k,r,s,c]
 *
 * the gradient of a cross-correlation Conv2d with respect to its input.
 * P = floor((H + 2*pad - dil*(R-1) - 1)/stride) + 1, Q likewise with W and S.
 * Inputs are fp16 or bf16; every product is accumulated in fp32 (the page's
 * closing remark that training needs fp32 accumulation).  Optionally the
 * result is gated by a saved activation x, out = (x > 0) ? dX : +0.0 (the
 * dgrad "activation fusion" of the page's last comments).
 *
 * Layouts: dY  NHWC  [N][P][Q][K]
 *          W   KRSC  [K][R][S][C]      (the forward filter, as stored)
 *          dX  NHWC  [N][H][W][C]      (fp16/bf16 like dY, or fp32)
 *          x   NHWC  [N][H][W][C]      (same type as dY)
 * All tensors are dense and contiguous.  Every pointer passed to prepack or
 * dgrad is a DEVICE pointer, 16-byte aligned.
 *
 * Ownership: the caller owns all tensors and streams; the library never
 * allocates, frees or retains caller memory.  A handle owns its host plan
 * and a 4-byte device status word.  Calls are asynchronous on the given stream.
 *
 * Errors: every function returns a cdg_status_t; nothing aborts or throws
 * across this interface.  On any error other than CDG_ERR_CUDA nothing has
 * been launched.
 *
 * Thread safety: a handle may be used from one thread at a time; calls on one
 * handle from different streams must not overlap on the GPU (they share the
 * handle's status word and its cached descriptors).
 */
#ifndef CDG_H
#define CDG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct cdg_plan_st *cdg_handle_t;
/* A cudaStream_t, passed as an opaque pointer (NULL = the legacy default stream). */
typedef void *cdg_stream_t;

typedef enum {
    CDG_OK = 0,
    CDG_ERR_INVALID_ARG = 1,  /* bad size, NULL pointer, unknown flag            */
    CDG_ERR_UNSUPPORTED = 2,  /* valid but outside what the kernels handle:       */
                              /* C or K not a multiple of 8, stride > 4,          */
                              /* R*S > 128, tensor dims beyond TMA limits         */
    CDG_ERR_ALIGNMENT = 3,    /* a tensor pointer is not 16-byte aligned          */
    CDG_ERR_ALIAS = 4,        /* dX overlaps dY, the packed weights or x          */
    CDG_ERR_CUDA = 5,         /* a CUDA runtime/driver call or launch failed      */
    CDG_ERR_TIMEOUT = 6,      /* a kernel gave up a bounded pipeline wait         */
    CDG_ERR_NO_DEVICE = 7,    /* the handle was planned without a device          */
    CDG_ERR_SCRATCH_TOO_SMALL = 8 /* cdg_dgrad_noalloc: packed weights exceed     */
                                  /* CDG_NOALLOC_MAX_WEIGHT_BYTES                 */
} cdg_status_t;

/* CDG_F32 is taken by the token operators and the weight update (below) only. */
typedef enum { CDG_F16 = 0, CDG_BF16 = 1, CDG_F32 = 2 } cdg_dtype_t;

/* Epilogue flags (bit set). */
enum {
    CDG_EPI_RELU_BWD = 1,     /* gate by the saved activation: out = (x > 0) ? v : +0.0 */
    CDG_EPI_OUT_F32 = 2,      /* write dX as fp32 instead of the input type             */
    CDG_EPI_RELU_BWD_BITS = 4, /* the same gate from a packed bit mask (one bit per     */
                              /* element, see cdg_pack_relu_mask): out = bit ? v : +0.0 */
                              /* (not together with CDG_EPI_RELU_BWD)                   */
    CDG_EPI_SUM = 8,          /* also the per-channel sums of the output (cdg_dgrad_sums) */
    CDG_EPI_SUM_X = 16,       /* CDG_EPI_SUM plus the per-channel sums of out * x where   */
                              /* the gate passes; needs CDG_EPI_RELU_BWD                 */
    CDG_EPI_GELU_BWD = 32,    /* GELU backward: out = v * f'(x), x the GELU's saved      */
                              /* input (same layout and type as for CDG_EPI_RELU_BWD),   */
                              /* f(x) = x (1 + erf(x / sqrt 2)) / 2                      */
    CDG_EPI_SILU_BWD = 64     /* SiLU backward: out = v * f'(x), f(x) = x / (1 + e^-x)   */
                              /* (at most one of RELU_BWD, RELU_BWD_BITS, GELU_BWD,      */
                              /* SILU_BWD)                                               */
};

/*
 * Plan one dgrad shape on the current CUDA device.
 *   N, H, W    batch and dX spatial size (the forward input size)
 *   C, K       dX channels and dY channels (forward in / out channels)
 *   R, S       filter size; stride, pad, dil apply to both axes, pad symmetric
 *   dtype      CDG_F16 or CDG_BF16 for dY, W and x
 *   epilogue   CDG_EPI_* bit set
 * On success *out receives a handle (free it with cdg_destroy).  Validation:
 * all sizes >= 1 (pad >= 0), P and Q >= 1, C % 8 == 0, K % 8 == 0, stride <= 4,
 * R*S <= 128.  The plan derives P and Q, splits a strided problem into its
 * stride^2 phase sub-convolutions (each dX pixel residue class (h mod stride,
 * w mod stride) receives a fixed subset of the filter taps), chooses tiles and
 * allocates the 4-byte device status word.
 */
int cdg_plan(int N, int H, int W, int C, int K, int R, int S,
             int stride, int pad, int dil, int dtype, int epilogue, cdg_handle_t *out);

/*
 * The same planning without touching any GPU: num_sms stands in for the
 * device's SM count.  The handle answers the query functions below; prepack
 * and dgrad on it return CDG_ERR_NO_DEVICE.  For inspecting the planner.
 */
int cdg_plan_host(int N, int H, int W, int C, int K, int R, int S,
                  int stride, int pad, int dil, int dtype, int epilogue,
                  int num_sms, cdg_handle_t *out);

/* Release a handle (NULL is ignored).  Synchronises nothing. */
void cdg_destroy(cdg_handle_t h);

/* dY's spatial extents P and Q. */
int cdg_get_output_dims(cdg_handle_t h, int *P, int *Q);

/* Bytes the packed-weight buffer must have (R*S*C*K elements of dtype). */
size_t cdg_packed_weight_bytes(cdg_handle_t h);

/*
 * Planner description, for logs and tests.
 */
typedef struct {
    int P, Q;
    int num_phases;       /* stride^2                                            */
    int phase_taps[16];   /* taps of phase (ph, pw) at index ph*stride + pw       */
    int tile_m;           /* dX pixels per tile (GEMM M tile)                      */
    int tile_n;           /* channels per tile (GEMM N tile)                       */
    int tile_k;           /* dY channels per pipeline stage (GEMM K block)         */
    int a_mode;           /* 0: 4-D boxes over dY per tap, 1: dY rows as a matrix, */
                          /* 2: one halo box per K block for all taps, weights     */
                          /*    streamed per tap (opt-in),                         */
                          /* 3: halo boxes with every weight tile resident in      */
                          /*    shared memory (chosen when the filter fits)        */
    int box_w, box_h, box_n; /* output tile box (a_mode 0 and 2)                   */
    int stages;           /* shared-memory pipeline depth                          */
    int work_items;       /* (phase, m-tile, n-tile) items in one launch           */
    int grid;             /* persistent CTAs                                       */
    int smem_bytes;       /* dynamic shared memory per CTA                         */
    int tmem_cols;        /* tensor-memory columns per CTA                         */
    int cta_pair;         /* 1: CTA pairs share 256-row tiles (2-SM MMA)            */
    int mma_warps;        /* MMA-issuing warps per CTA: 2 splits the work items and */
                          /* the pipeline stages between two issuers (N tile <= 128) */
    int tuned;            /* 1 once cdg_autotune has chosen this plan              */
} cdg_plan_info_t;

int cdg_plan_get_info(cdg_handle_t h, cdg_plan_info_t *info);

/*
 * Re-lay the forward filter W (KRSC, dtype, device) into the packed operand
 * the dgrad kernel reads: Wpacked[r*S + s][c][k] = W[k][r][s][c], i.e. for
 * every tap a C x K matrix with K contiguous.  Wpacked must hold
 * cdg_packed_weight_bytes(h) bytes and not overlap W.  Asynchronous on stream.
 */
int cdg_prepack_weights(cdg_handle_t h, const void *W_krsc, void *Wpacked, cdg_stream_t stream);

/*
 * dX = dgrad(dY, W) for the planned shape, one kernel launch, asynchronous
 * on stream.  relu_mask is the saved activation x for a plan with
 * CDG_EPI_RELU_BWD (NHWC like dX, input dtype), the packed mask for
 * CDG_EPI_RELU_BWD_BITS (cdg_pack_relu_mask's layout), the activation's saved
 * input for CDG_EPI_GELU_BWD or CDG_EPI_SILU_BWD (NHWC like dX, input
 * dtype), else NULL; it must not overlap dX.  Every element of dX is written, including pixels no
 * filter tap reaches (+0.0); dX is never read, so its prior contents do not
 * matter.  dY, Wpacked and x are only read.  No workspace, no allocation.
 * A device-side pipeline timeout (which a correct launch never hits) is
 * reported by cdg_device_status, not here.
 */
int cdg_dgrad(cdg_handle_t h, const void *dY, const void *Wpacked, void *dX,
              const void *relu_mask, cdg_stream_t stream);

/*
 * dgrad with the per-channel sums of its output fused into the epilogue (the
 * epilogue fusion of the Bolt reading notes: a reduction over the output is
 * taken where the output is made, instead of by a second pass that re-reads
 * it).  For a plan made with CDG_EPI_SUM, after dX = dgrad(dY, W) (gated as
 * the plan says):
 *
 *     sums[c]     = sum over n, h, w of out[n,h,w,c]
 *     sums[C + c] = sum over n, h, w with x[n,h,w,c] > 0 of out[n,h,w,c] * x[n,h,w,c]
 *                   (CDG_EPI_SUM_X only)
 *
 * taken from the fp32 values before they are rounded to dX's type.  sums[c]
 * is the bias gradient of a bias added before the ReLU, and BatchNorm's beta
 * gradient; with x the BatchNorm output y = gamma*xhat + beta (the ReLU's
 * input, or relu(y), which gives the same terms), BatchNorm's gamma gradient
 * is (sums[C + c] - beta[c]*sums[c]) / gamma[c].  Positions the gate masks add
 * nothing, whatever x holds there.
 *
 *   sums       device, fp32, C (CDG_EPI_SUM) or 2*C (CDG_EPI_SUM_X) values,
 *              overwritten
 *   workspace  device, cdg_sums_workspace_bytes(h) bytes, overwritten: each
 *              CTA of the launch adds its tiles' column sums into a row of its
 *              own, and a second kernel adds the rows in order
 *
 * Two kernel launches on stream.  The result does not depend on scheduling:
 * every partial sum is taken in a fixed order, so repeated calls give the
 * same bits.  Other arguments and errors as for cdg_dgrad; sums and workspace
 * must be 16-byte aligned and overlap no other tensor (CDG_ERR_ALIAS).
 * cdg_dgrad, cdg_dgrad_noalloc and cdg_autotune refuse plans made with the
 * sum flags (CDG_ERR_INVALID_ARG, CDG_ERR_INVALID_ARG, CDG_ERR_UNSUPPORTED).
 */
int cdg_dgrad_sums(cdg_handle_t h, const void *dY, const void *Wpacked, void *dX, const void *relu_mask, float *sums,
                   void *workspace, cdg_stream_t stream);

/* Bytes of the workspace cdg_dgrad_sums needs: (SM count) x (1 or 2) x C x 4;
 * 0 for a plan without the sum flags. */
size_t cdg_sums_workspace_bytes(cdg_handle_t h);

/*
 * Synchronise stream, then read and clear the handle's device status word:
 * CDG_OK, or CDG_ERR_TIMEOUT if a launch since the last call gave up a
 * bounded wait (its dX is then incomplete).
 */
int cdg_device_status(cdg_handle_t h, cdg_stream_t stream);

/*
 * How long any single pipeline wait of this plan's kernel may take before the
 * launch gives up: it then records CDG_ERR_TIMEOUT (read by
 * cdg_device_status), leaves every loop, waits (again bounded) for its own
 * copies and tensor-core work in flight, releases its tensor memory and
 * returns, leaving dX incomplete.  A correct launch never comes near the
 * default of 4 s; a caller with a watchdog of its own may lower it.
 * ns in [1e5, 6e10] (0.1 ms .. 60 s), else CDG_ERR_INVALID_ARG.  Host only;
 * applies to launches made after the call.
 */
int cdg_plan_set_wait_limit(cdg_handle_t h, unsigned long long ns);

/*
 * TEST ONLY.  stage >= 0: every launch of this plan withholds one operand
 * load -- in each CTA, the pipeline stage with that sequence number gets
 * neither its tensor copies nor their byte count -- so the MMA warp's bounded
 * wait for it runs out and the launch takes the timeout path above (status
 * CDG_ERR_TIMEOUT, dX incomplete).  This exercises the failure path without
 * any fault: every wait in the kernel is bounded.  stage = -1 restores normal
 * launches.  Plans in the halo operand mode or with CTA pairs return
 * CDG_ERR_UNSUPPORTED (their loaders do not take the option).  Host only.
 */
int cdg_plan_withhold_load_for_test(cdg_handle_t h, int stage);

/*
 * Plan-time autotuning, in the manner of cuDNN's Find (the pages' comparison of
 * cuDNN's Get and Find algorithm selection): run the dgrad of this plan's shape
 * under each configuration the planner can produce for it (the planner's own
 * choice; without or with CTA pairs; one MMA warp; with or without halo
 * operand boxes; halo boxes with CTA pairs; phases in order; 128- and
 * 192-channel N tiles), reps timed launches
 * each after one untimed launch, and keep the fastest in the handle
 * (cdg_plan_get_info then reports it, with tuned = 1).  Configurations that
 * come out identical are timed once.  Each timed launch follows a write of a
 * scratch buffer twice the L2 size, so candidates are compared with cold
 * caches, as layers run inside a network step.  The planner's own choice is
 * kept unless another configuration is at least 2 % faster.
 *
 *   dY, Wpacked, dX, relu_mask   as for cdg_dgrad; dX is overwritten (with the
 *                                correct result) many times
 *   reps                         timed launches per configuration, 1..1000
 *   best_ms                      if not NULL, receives the best mean launch time
 *
 * Synchronises stream.  Allocates a 4-byte status word per candidate plan and
 * the flush buffer (all freed before returning).  On CDG_ERR_CUDA or
 * CDG_ERR_TIMEOUT the handle keeps its previous plan.
 */
int cdg_autotune(cdg_handle_t h, const void *dY, const void *Wpacked, void *dX, const void *relu_mask,
                 cdg_stream_t stream, int reps, float *best_ms);

/*
 * Pack the ReLU-backward mask of a saved activation x (NHWC, pixels = N*H*W
 * rows of C channels, dtype CDG_F16 or CDG_BF16) for a plan with
 * CDG_EPI_RELU_BWD_BITS.  Layout: each pixel's C channels as bits, the row
 * padded to whole 16-byte units (cdg_relu_mask_bytes(1, C) bytes a pixel);
 * channel c of pixel p is bit c % 8 of byte p*row + c/8, set when x > 0
 * (x <= 0, -0.0 and NaN give 0); padding bits are 0.  For C a multiple of 128
 * this is exactly one bit per element; the padding lets the dgrad fetch a
 * tile's mask with the same tensor copies as its output, and for C < 128 it
 * still cuts the gate's reads 8x against x.  This variant of the pages'
 * ReLU-backward epilogue fusion is an addition of this library (the pages gate
 * with the activation itself).  C % 8 == 0; x and bits 16-byte aligned, not
 * overlapping; bits holds cdg_relu_mask_bytes(pixels, C) bytes, all of which
 * are written.  Asynchronous on stream.
 */
int cdg_pack_relu_mask(const void *x, void *bits, long long pixels, int C, int dtype, cdg_stream_t stream);

/* Bytes of a packed ReLU mask of `pixels` pixels of C channels (see
 * cdg_pack_relu_mask), or -1 for pixels < 0, C <= 0 or C % 8 != 0.  Host only. */
long long cdg_relu_mask_bytes(long long pixels, int C);

/* Static text for a status code. */
const char *cdg_status_string(int status);

/*
 * dgrad for callers that cannot allocate device memory -- code that runs
 * where cudaMalloc is off limits (inside a memory pool that must not grow,
 * a real-time loop that may not block on the allocator, an embedding runtime
 * that owns all device memory).  This entry point has no counterpart in the
 * pages the method is described on; it is an addition of this library.
 *
 * It computes exactly what cdg_prepack_weights followed by cdg_dgrad
 * computes, but takes the forward filter W in its stored KRSC layout and
 * needs neither a packed-weight buffer nor a device status word from the
 * caller: both live in one scratch array compiled into the library
 * (a file-scope __device__ array that every GPU which loads the library keeps
 * until the process exits).  It calls no cudaMalloc, no cudaFree and no
 * allocating library routine.
 *
 *   h          a plan from cdg_plan, or from cdg_plan_host (which touches no
 *              device; pass the device's SM count as num_sms)
 *   dY, dX, relu_mask   as for cdg_dgrad (device pointers, 16-byte aligned)
 *   W_krsc     the forward filter [K][R][S][C], device pointer
 *
 * Limit: the packed weights (R*S*C*K elements of 2 bytes) must fit in
 * CDG_NOALLOC_MAX_WEIGHT_BYTES (8 MiB: 4,194,304 weights, enough for every
 * ResNet-50 convolution); larger filters return CDG_ERR_SCRATCH_TOO_SMALL
 * before anything is launched.
 *
 * The first call on a device finds the scratch array's device address
 * (cudaGetSymbolAddress, with that device current) and raises the kernels'
 * shared-memory limit; make that first call before any stream capture.
 *
 * Every call on a device shares the one scratch array, which keeps the last
 * call's packed weights; each call clears the status word and re-packs W on
 * its stream first.  Calls whose work overlaps on the GPU (different streams,
 * or different host threads) race on the scratch array and give wrong
 * results: serialise them.  A device-side pipeline timeout is recorded in the
 * scratch status word, not returned here: read it with
 * cdg_dgrad_noalloc_status.
 *
 * A plan from cdg_plan_host that chose CTA pairs has its persistent grid
 * checked against the device (how many pairs fit at once) on its first
 * cdg_dgrad_noalloc call, and reduced if needed.
 */
#define CDG_NOALLOC_MAX_WEIGHT_BYTES (8u << 20)
int cdg_dgrad_noalloc(cdg_handle_t h, const void *dY, const void *W_krsc, void *dX, const void *relu_mask,
                      cdg_stream_t stream);

/*
 * The status word cdg_dgrad_noalloc launches report into, on the current
 * device: synchronise stream, read the word and clear it.  Returns CDG_OK, or
 * CDG_ERR_TIMEOUT if a cdg_dgrad_noalloc launch since the last read gave up a
 * bounded wait (its dX is then incomplete), or CDG_ERR_CUDA.  Allocates
 * nothing (the word is in the library's scratch array).  Because every
 * cdg_dgrad_noalloc call on a device shares the word, read it after each call
 * (or each batch of serialised calls) whose result matters.
 */
int cdg_dgrad_noalloc_status(cdg_stream_t stream);

/*
 * Back-to-back dgrads in one persistent kernel: the backward of a
 * bottleneck's 1x1 -> 3x3 forward pair (conv1 1x1 C1 -> C2, then the
 * activation, then conv2 R2 x S2 C2 -> K2), which runs as
 *
 *     g   = act_bwd(dgrad(dY2, W2), x2)     (conv2's dgrad, gated)
 *     dX1 = dgrad_1x1(g, W1)                 (conv1's dgrad)
 *
 * This is the persistent kernel fusion of the Bolt reading notes (page 5 of
 * the pages, "Persistent kernel (GEMM/Conv) fusion"), with threadblock
 * residence: each CTA computes a tile of g over all C2 channels (ThreadBlock_N
 * = the first dgrad's output channels) and keeps it on chip -- in tensor
 * memory, where it is the A operand of the second GEMM -- so g is never
 * read back from HBM.  The second dgrad is 1x1, stride 1, so a tile of dX1
 * needs exactly the same pixels of g.  g itself is written only if asked
 * (conv1's weight gradient needs it).
 *
 *   conv2: stride 1, pad2, dil2, R2 x S2, C2 = 64 input channels (this kernel),
 *          K2 output channels (dY2's), dY2 NHWC [N][P][Q][K2] with
 *          P = H + 2*pad2 - dil2*(R2-1), W2 KRSC [K2][R2][S2][C2];
 *          its weights and a halo tile of dY2 must fit in shared memory
 *          together with W1 (CDG_ERR_UNSUPPORTED otherwise)
 *   conv1: 1x1, stride 1, pad 0, C1 <= 256 input channels (C1 % 8 == 0),
 *          W1 KRSC [C2][1][1][C1]
 *   x2     the saved tensor of the activation between them, NHWC [N][H][W][C2]:
 *          flags CDG_EPI_RELU_BWD (its output or input; g = (x2 > 0) ? v : +0.0),
 *          CDG_EPI_GELU_BWD or CDG_EPI_SILU_BWD (its input; g = v * f'(x2)),
 *          or none of them (no activation: x2 = NULL)
 *   g      NHWC [N][H][W][C2], written only with CDG_FUSED_WRITE_G (else NULL)
 *   dX1    NHWC [N][H][W][C1]
 * All in dtype (dX1 and g in dtype too); fp32 accumulation in both GEMMs; g
 * is rounded to dtype before the second GEMM, exactly as if it went through
 * memory.  Weights are packed once with cdg_fused_prepack_weights.
 */
typedef struct cdg_fused_st *cdg_fused_t;
#define CDG_FUSED_WRITE_G 256

int cdg_fused_plan(int N, int H, int W, int C1, int C2, int K2, int R2, int S2, int pad2, int dil2, int dtype,
                   int flags, cdg_fused_t *out);
/* The same planning without a device (num_sms stands in for the SM count). */
int cdg_fused_plan_host(int N, int H, int W, int C1, int C2, int K2, int R2, int S2, int pad2, int dil2, int dtype,
                        int flags, int num_sms, cdg_fused_t *out);
void cdg_fused_destroy(cdg_fused_t f);
/* Bytes of the two packed weight buffers (W2: R2*S2*C2*K2, W1: C1*C2 elements). */
int cdg_fused_packed_weight_bytes(cdg_fused_t f, size_t *w2_bytes, size_t *w1_bytes);
/* Pack W2 and W1 (device, KRSC) into W2p and W1p; asynchronous on stream. */
int cdg_fused_prepack_weights(cdg_fused_t f, const void *W2_krsc, const void *W1_krsc, void *W2p, void *W1p,
                              cdg_stream_t stream);
/* One launch on stream.  Errors as for cdg_dgrad (CDG_ERR_ALIAS when an
 * output overlaps an input or the other output).  No allocation. */
int cdg_dgrad_fused(cdg_fused_t f, const void *dY2, const void *W2p, const void *x2, const void *W1p, void *g,
                    void *dX1, cdg_stream_t stream);
/* The first dgrad's planner description (halo tiles, grid, stages), with the
 * fused kernel's shared memory and tensor-memory columns. */
int cdg_fused_get_info(cdg_fused_t f, cdg_plan_info_t *info);
/* Synchronise stream, read and clear the fused plan's device status word. */
int cdg_fused_device_status(cdg_fused_t f, cdg_stream_t stream);

/*
 * Weight gradient (wgrad) of the same cross-correlation Conv2d, the
 * follow-up the apache/tvm PR #10110 page ("[CUTLASS] Conv2d dgrad") names
 * for dgrad, "wgrad + parallel split-k" (merge comment).  The page gives no
 * formula; this library computes the definition
 *
 *   dW[k,r,s,c] = sum over n, p, q of
 *                 dY[n,p,q,k] * x[n, p*stride - pad + r*dil, q*stride - pad + s*dil, c]
 *
 * with x read as zero outside the image.  dY NHWC [N][P][Q][K] and the
 * forward input x NHWC [N][H][W][C] in dtype; dW KRSC [K][R][S][C] in dtype,
 * or fp32 with out_f32 = 1.  fp32 accumulation.  The reduction over the
 * N*P*Q positions is split into `splits` parts that run in parallel; their
 * fp32 partials go to a caller-provided workspace and are added in a fixed
 * order, so results are deterministic.
 */
typedef struct cdg_wgrad_st *cdg_wgrad_t;

typedef struct {
    int P, Q;
    int tile_m;           /* dY channels per tile (GEMM M tile, 128)             */
    int tile_n;           /* x channels per tile and tap                          */
    int taps_per_item;    /* taps whose tiles share one MMA along N (narrow C)    */
    int splits;           /* reduction splits                                     */
    int pos_box[3];       /* positions per block along q, p, n (product 64)      */
    int blocks;           /* position blocks of 64 in the reduction              */
    int stages;           /* shared-memory pipeline depth                         */
    int work_items;       /* (split, tap group, m-tile, n-tile) items in one launch */
    int grid;             /* persistent CTAs                                      */
    int smem_bytes;       /* dynamic shared memory per CTA                        */
    int tmem_cols;        /* tensor-memory columns per CTA                        */
    int x_major;          /* 1 (1x1 filters, K <= 64, C > 64): M tiles pair two   */
                          /* 64-channel slices of x and N runs over the dY        */
                          /* channels, so that no M row is idle; tile_m/tile_n    */
                          /* then count x channels / dY channels                  */
} cdg_wgrad_info_t;

/*
 * Plan one wgrad shape on the current device.  Arguments as for cdg_plan
 * (H, W are x's sizes); out_f32 0 or 1; splits = 0 lets the planner choose
 * (enough work items to fill the SMs), k >= 1 asks for k (capped at the
 * number of position blocks).  Errors: CDG_ERR_INVALID_ARG for bad sizes or
 * flags, CDG_ERR_UNSUPPORTED when C or K is not a multiple of 8, stride > 4,
 * R*S > 128, or H or W is smaller than the stride.  Free with
 * cdg_wgrad_destroy.
 */
int cdg_wgrad_plan(int N, int H, int W, int C, int K, int R, int S, int stride, int pad, int dil, int dtype,
                   int out_f32, int splits, cdg_wgrad_t *out);

/* The same planning without a device (num_sms stands in for the SM count);
 * cdg_wgrad on such a handle returns CDG_ERR_NO_DEVICE. */
int cdg_wgrad_plan_host(int N, int H, int W, int C, int K, int R, int S, int stride, int pad, int dil, int dtype,
                        int out_f32, int splits, int num_sms, cdg_wgrad_t *out);

void cdg_wgrad_destroy(cdg_wgrad_t h);

/* Bytes of the fp32 workspace cdg_wgrad needs: splits * K * R * S * C * 4. */
size_t cdg_wgrad_workspace_bytes(cdg_wgrad_t h);

int cdg_wgrad_get_info(cdg_wgrad_t h, cdg_wgrad_info_t *info);

/*
 * dW = wgrad(dY, x): two kernel launches on stream (the split GEMM, then the
 * ordered reduction), asynchronous.  All pointers are device pointers,
 * 16-byte aligned; workspace holds cdg_wgrad_workspace_bytes(h) bytes and is
 * overwritten; dW may not overlap dY, x or the workspace, nor the workspace
 * dY or x (CDG_ERR_ALIAS).  dY and x are only read.  No allocation.  A
 * device-side pipeline timeout is reported by cdg_wgrad_device_status.
 */
int cdg_wgrad(cdg_wgrad_t h, const void *dY, const void *x, void *dW, void *workspace, cdg_stream_t stream);

/* Synchronise stream, then read and clear the plan's device status word. */
int cdg_wgrad_device_status(cdg_wgrad_t h, cdg_stream_t stream);

/*
 * Token operators: the two ends of a training step whose layers' gradients
 * cdg_dgrad and cdg_wgrad compute -- the log probabilities of given tokens
 * with the gradient of the logits (the first dY), and the embedding lookup
 * with its gradient -- and the forms that serving takes them in.
 *
 * None of these needs a plan or synchronises; every call is asynchronous on
 * stream and allocates nothing.  Sizes of zero rows or tokens launch nothing.
 * Matrices have unit column stride and a row stride `ld` in elements (at least
 * the row length); rows may start at any element (pointers aligned to the
 * element; no 16-byte rule).  dtype is CDG_F16, CDG_BF16 or CDG_F32.  Token
 * numbers are int32 (index_bytes = 4) or int64 (8); a number outside
 * [0, vocab) -- -1, -100 -- names no token.  Results do not depend on
 * scheduling: repeated calls give the same bits.
 *
 * cdg_token_logprobs: with z = scale * logits[i], p = softmax(z),
 *
 *     lse[i]     = log sum over j of exp(z_j)
 *     logp[i]    = z_t - lse[i], t = targets[i]; 0 where there is no token
 *     entropy[i] = - sum over j of p_j log p_j   (p_j = 0 adds nothing)
 *     top_ids[i][0..top), top_logp[i][0..top):
 *                  the `top` largest logits, largest first, equal ones by
 *                  lowest number, and their log probabilities
 *
 * Sums are fp32.  Logits of -inf (masked tokens) have probability 0.  A row of
 * -inf alone has lse = logp = top_logp = -inf, entropy 0 and top_ids 0, 1, ...
 * A row that holds NaN or +inf answers NaN everywhere (logp: where there is a
 * token), and top_ids -1.
 *   scale       > 0, finite (1 / temperature)
 *   vocab       at most 2^30
 *   top         0 .. 32, at most vocab
 *   targets and logp may both be NULL; lse and entropy may be NULL; top_ids and
 *   top_logp are NULL exactly when top = 0.  fp32 outputs, int32 top_ids,
 *   dense, none overlapping another or the logits (CDG_ERR_ALIAS).
 */
int cdg_token_logprobs(const void *logits, long long ld, const void *targets, int index_bytes, long long rows,
                       int vocab, int dtype, float scale, int top, float *logp, float *lse, float *entropy,
                       int *top_ids, float *top_logp, cdg_stream_t stream);

/*
 * The gradient of cdg_token_logprobs: for the row gradients g = g_logp[i] and
 * h = g_entropy[i] of logp and entropy,
 *
 *     dlogits[i][j] = scale * (g (1[j = t] - p_j) - h p_j (log p_j + entropy[i]))
 *
 * with log p_j = z_j - lse[i]; lse and entropy as cdg_token_logprobs wrote
 * them.  A row without a token has g = 0; a row of -inf alone gets zeros.
 * p_j is as exact as an fp32 lse holds it (|lse| 2^-24, relative) and at most
 * 1: a row of nothing but finite masks gets a bounded gradient, not 1 / vocab.
 * g_entropy may be NULL (h = 0; entropy may then be NULL too).  dlogits has
 * the logits' dtype and may be the logits themselves (same pointer, same
 * stride); any other overlap is CDG_ERR_ALIAS.
 */
int cdg_token_logprobs_grad(const void *logits, long long ld, const void *targets, int index_bytes, long long rows,
                            int vocab, int dtype, float scale, const float *lse, const float *entropy,
                            const float *g_logp, const float *g_entropy, void *dlogits, long long ld_d,
                            cdg_stream_t stream);

/*
 * cdg_embed: out[i][:] = scale * table[tokens[i]][:], rounded once; a row of
 * zeros where there is no token.  table is vocab x dim, out count x dim, both
 * dtype.  out must not overlap the table or the tokens.  dim at most 2^24.
 */
int cdg_embed(const void *table, long long ld_table, const void *tokens, int index_bytes, long long count, int vocab,
              int dim, int dtype, float scale, void *out, long long ld_out, cdg_stream_t stream);

/*
 * The gradient of cdg_embed with respect to the table:
 *
 *     dtable[v][:] = scale * (sum of dout[i][:] over the i with tokens[i] = v)
 *
 * added in ascending order of i within parts of a fixed size, the parts in
 * order, in fp32, and rounded once to dtype, or kept fp32 with out_f32 = 1.  accumulate = 0
 * writes every row of dtable (zeros where no token points); accumulate = 1
 * adds the sums to the rows that tokens point to and leaves the others alone
 * (a table tied to an output layer already holds that layer's gradient).
 *   workspace   device, cdg_embed_grad_workspace_bytes(count, vocab, dim)
 *               bytes, 16-byte aligned, overwritten
 * dtable and workspace overlap each other and the inputs nowhere
 * (CDG_ERR_ALIAS).  count below 2^30, dim at most 2^24; above some millions of
 * tokens the sort's time grows with the square of count (2^24: about 4 ms).
 */
int cdg_embed_grad(const void *dout, long long ld_dout, const void *tokens, int index_bytes, long long count,
                   int vocab, int dim, int dtype, float scale, void *dtable, long long ld_dtable, int out_f32,
                   int accumulate, void *workspace, cdg_stream_t stream);

/* Bytes of cdg_embed_grad's workspace; 0 for sizes it refuses.  Host only. */
size_t cdg_embed_grad_workspace_bytes(long long count, int vocab, int dim);

/*
 * The weight update from an orthogonalised gradient (the Muon optimiser's
 * step): what consumes cdg_wgrad's dW, a K x (R*S*C) matrix as it is stored.
 *
 * cdg_muon_orthogonalize: for every rows x cols matrix U of a batch, `steps`
 * Newton-Schulz products with the quintic (a, b, c),
 *
 *     X = U / (|U|_F + eps)
 *     steps times:  A = X X^T,  X = a X + (b A + c A^2) X
 *
 * on the smaller side (X^T X for rows > cols), which drives the singular
 * values of U towards 1 and keeps its singular vectors.  U and O are dtype
 * (CDG_F16, CDG_BF16 or CDG_F32), dense, batch x rows x cols; O may not
 * overlap U.  Products run on the tensor cores on fp16 operands with fp32
 * sums; X is held as a high and a low fp16 part and the diagonal of b A + c A^2
 * in fp32, so that O is within 2e-3 of the iteration in exact arithmetic
 * (relative, Frobenius, five steps; up to 1.8e-3 where all singular values are
 * equal, else mostly below 1e-3), beside its own rounding.  With CDG_F32 every
 * operand is two fp16 parts, at three products for one, and O is within 1e-5.
 * |U|_F must be representable: its square is summed in fp32.  A zero U gives a
 * zero O, whatever eps is; a U with a NaN or an infinity gives NaN.
 *
 * cdg_muon_step: the whole update of fp32 weights W from a gradient G (dtype)
 * and its momentum M (fp32), all batch x rows x cols, dense:
 *
 *     M_out = momentum * M + G
 *     U     = G + momentum * M_out  (nesterov = 1),  M_out (nesterov = 0)
 *     W_out = (1 - lr * weight_decay) * W - lr * update_scale * orthogonalize(U)
 *
 * M_out and the sum for W_out are fp32; the orthogonalised update is as exact
 * as cdg_muon_orthogonalize's for the same dtype, so that of an fp32 G keeps fp32
 * accuracy, at 1.6 to 4.5 times the time of a 16-bit plan's.
 * M_out may be M, and W_out may be W; no other overlap (CDG_ERR_ALIAS).
 *
 * A plan holds one shape.  Calls on one plan must not overlap on the GPU if
 * they share the workspace (device, cdg_muon_workspace_bytes bytes, 256-byte
 * aligned, overwritten).  Pointers of U, O, G, M and W are 16-byte aligned.
 * A device-side pipeline timeout (which a correct launch never hits) is
 * reported by cdg_muon_device_status.
 */
typedef struct cdg_muon_st *cdg_muon_t;

/* batch, rows, cols >= 1; steps 1 .. 32; eps >= 0.  (a, b, c) must keep
 * [0, 1] bounded over the steps: every iterate of the scalar map
 * x -> a x + b x^3 + c x^5 within 4, and |b x^2 + c x^4| <= 60
 * (CDG_ERR_INVALID_ARG otherwise). */
int cdg_muon_plan(int batch, int rows, int cols, int dtype, int steps, float a, float b, float c, float eps,
                  cdg_muon_t *out);
/* The same planning without a device (num_sms stands in for the SM count). */
int cdg_muon_plan_host(int batch, int rows, int cols, int dtype, int steps, float a, float b, float c, float eps,
                       int num_sms, cdg_muon_t *out);
void cdg_muon_destroy(cdg_muon_t h);
size_t cdg_muon_workspace_bytes(cdg_muon_t h);

typedef struct {
    int m, n;             /* the smaller and the larger side                      */
    int transposed;       /* 1: rows > cols, the kernels hold U^T                 */
    int gram;             /* 1: the steps run on X X^T alone, on one SM a matrix    */
    int launches;         /* kernel launches of one cdg_muon_orthogonalize        */
} cdg_muon_info_t;
int cdg_muon_get_info(cdg_muon_t h, cdg_muon_info_t *info);

int cdg_muon_orthogonalize(cdg_muon_t h, const void *U, void *O, void *workspace, cdg_stream_t stream);
int cdg_muon_step(cdg_muon_t h, const float *W, const void *G, const float *M, float *W_out, float *M_out, float lr,
                  float momentum, float weight_decay, float update_scale, int nesterov, void *workspace,
                  cdg_stream_t stream);
/* Synchronise stream, then read and clear the plan's device status word. */
int cdg_muon_device_status(cdg_muon_t h, cdg_stream_t stream);

/*
 * Attention over packed sequences and its gradient: the block between the two
 * ends of a token model's training step.
 *
 * q is q_tokens x (heads * dim), k and v are k_tokens x (kv_heads * dim), rows
 * of all heads one after the other; query head h reads key and value head
 * h / (heads / kv_heads).  Sequence s has the rows q_offsets[s] ..
 * q_offsets[s + 1] of q and k_offsets[s] .. k_offsets[s + 1] of k and v.  For
 * its query i of ql and key j of kl, r = i + kl - ql (the last query sees the
 * last key), i sees j where
 *
 *     causal = 0: always;   causal = 1: j <= r;   window = w > 0: also j > r - w
 *
 * cdg_attention:       s_ij = scale q_i . k_j over the keys that i sees,
 *     lse_i = log sum_j exp(s_ij),   o_i = sum_j exp(s_ij - lse_i) v_j
 * A query that sees no key has o = 0 and lse = -inf.
 *
 * cdg_attention_grad:  with p_ij = exp(s_ij - lse_i) from the given lse, and
 *     ds_ij = p_ij (do_i . v_j - do_i . o_i),
 *     dv_j = sum_i p_ij do_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j
 * dk and dv are sums over the query heads of their group too.  Rows that no
 * sequence holds are neither read into a result nor written.
 *
 * All matrices are dtype (CDG_F16 or CDG_BF16); products have fp32 sums, p and
 * ds are rounded to dtype as their operands; row sums, lse (heads x q_tokens,
 * natural log) and do . o are fp32.  Repeated calls give the same bits.  The
 * gradient rounds fp16's p and ds at powers of two times their value, so that
 * those of many keys or small do keep their bits: p is held to 2^-36 or 2^-11 of
 * itself, ds to 2^-35 of max |do| max |v| + max |do . o| over the call's heads and
 * rows that are finite and a sequence's, or 2^-11 of itself.  It therefore takes
 * an lse for which p stays below 2^5 (the forward's: 1).
 * A NaN or an infinity in a row of a sequence may reach other results of that
 * sequence and head, masked or not, and none of another sequence or head
 * (group of heads, for k and v).
 *   dim        a multiple of 8, at most 128; heads a multiple of kv_heads, at most 1024
 *   ld_*       row strides in elements, multiples of 8; matrices 16-byte aligned.
 *              Matrices of one stride may lie side by side in the rows of one
 *              buffer, inputs and outputs alike; no other overlap of an output (CDG_ERR_ALIAS)
 *   q_offsets, k_offsets   device, sequences + 1 int32 (index_bytes = 4) or
 *              int64 (8) numbers, ascending; both may be NULL for one sequence of
 *              all rows.  Numbers outside [0, tokens] are cut to it, and a
 *              sequence that ends before it begins is empty; sequences that
 *              overlap leave their rows' results undefined
 *   tokens     below 2^30, sequences at most 2^20
 *   workspace  device, 256-byte aligned, cdg_attention_workspace_bytes or
 *              cdg_attention_grad_workspace_bytes bytes, overwritten
 *
 * A plan holds the heads and the mask, and belongs to the device that was
 * current when it was made (CDG_ERR_INVALID_ARG on another).  Calls on one plan
 * may overlap on the GPU unless they share a workspace or an output.  No call
 * allocates or synchronises.  A device-side pipeline timeout (which a correct
 * launch never hits) is reported by cdg_attention_device_status.
 */
typedef struct cdg_attention_st *cdg_attention_t;

/* window 0 (none), or > 0 with causal = 1 (one past every key hides nothing); scale > 0, finite. */
int cdg_attention_plan(int heads, int kv_heads, int dim, int dtype, int causal, int window, float scale,
                       cdg_attention_t *out);
/* The same without a device: for the checks and sizes. */
int cdg_attention_plan_host(int heads, int kv_heads, int dim, int dtype, int causal, int window, float scale,
                            cdg_attention_t *out);
void cdg_attention_destroy(cdg_attention_t h);
/* Bytes of workspace; 0 for sizes that are refused. */
size_t cdg_attention_workspace_bytes(cdg_attention_t h, long long q_tokens, long long k_tokens, int sequences);
size_t cdg_attention_grad_workspace_bytes(cdg_attention_t h, long long q_tokens, long long k_tokens, int sequences);

int cdg_attention(cdg_attention_t h, const void *q, long long ld_q, const void *k, long long ld_k, const void *v,
                  long long ld_v, long long q_tokens, long long k_tokens, const void *q_offsets, const void *k_offsets,
                  int index_bytes, int sequences, void *o, long long ld_o, float *lse, void *workspace,
                  cdg_stream_t stream);
int cdg_attention_grad(cdg_attention_t h, const void *q, long long ld_q, const void *k, long long ld_k, const void *v,
                       long long ld_v, const void *o, long long ld_o, const float *lse, const void *d_o,
                       long long ld_do, long long q_tokens, long long k_tokens, const void *q_offsets,
                       const void *k_offsets, int index_bytes, int sequences, void *dq, long long ld_dq, void *dk,
                       long long ld_dk, void *dv, long long ld_dv, void *workspace, cdg_stream_t stream);
/* Synchronise stream, then read and clear the plan's device status word. */
int cdg_attention_device_status(cdg_attention_t h, cdg_stream_t stream);

/*
 * Norms of queries and keys for each head with the position rotation in the
 * same pass, and their gradient.  For every token t and head of q (tokens x
 * heads * dim) and of k (tokens x kv_heads * dim), x the head's dim values:
 *
 *     norm = 1:  z = x / sqrt(mean(x^2) + eps) * w;     norm = 0:  z = x
 *     angle_i = positions[t] * inv_freq[i], i < rot / 2
 *     (y_a, y_b) = factor * (z_a cos - z_b sin, z_b cos + z_a sin)
 *         interleaved = 0:  a = i, b = i + rot / 2;     1:  a = 2 i, b = 2 i + 1
 *     y = z behind the first rot values
 *
 * and the gradient, for dy, with n = x / sqrt(mean(x^2) + eps) and dz = dy
 * turned back: dw = sum over tokens and heads of dz n, dn = dz w,
 * dx = (dn - n mean(dn n)) / sqrt(mean(x^2) + eps); dx = dz without the norm.
 *
 * Matrices are dtype (CDG_F16, CDG_BF16, CDG_F32) with row strides ld_* (below
 * 2^31), aligned to the element; inv_freq, w_q, w_k, dw_q and dw_k are fp32.
 * Computed in fp32 (a head's sum of squares has to be representable), rounded
 * once; a frequency is held to 2^-64 of a turn, so that angles are as exact as
 * fp32 holds them at positions up to 2^38.  An infinite or NaN frequency makes its
 * pairs NaN, and may others of the rotated part.  16-bit results use cosines and sines
 * good to 2^-20.  Repeated calls give the same bits.
 *   heads, kv_heads   either may be 0 (that side's pointers are not used)
 *   dim        at most 256;  rot even, 0 .. dim (0: no rotation, inv_freq may be NULL)
 *   positions  int32 or int64 (index_bytes 4, 8), any value; NULL: the token's number
 *   w_q, w_k   NULL: ones; NULL without the norm
 *   outputs    may be the input of the same side (same pointer, same stride): q_out
 *              q, dq dq_out; matrices of one stride may lie side by side in the
 *              rows of one buffer; no other overlap (CDG_ERR_ALIAS)
 *   q, k       of the gradient: not read without the norm (may be NULL)
 *   dw_q, dw_k NULL: not wanted
 *   workspace  of the gradient: device, cdg_qk_rope_grad_workspace_bytes bytes,
 *              16-byte aligned, overwritten
 */
int cdg_qk_rope(const void *q, long long ld_q, const void *k, long long ld_k, const void *positions, int index_bytes,
                long long tokens, int heads, int kv_heads, int dim, int dtype, const float *inv_freq, int rot,
                int interleaved, float factor, int norm, float eps, const float *w_q, const float *w_k, void *q_out,
                long long ld_qo, void *k_out, long long ld_ko, cdg_stream_t stream);
int cdg_qk_rope_grad(const void *q, long long ld_q, const void *k, long long ld_k, const void *positions,
                     int index_bytes, long long tokens, int heads, int kv_heads, int dim, int dtype,
                     const float *inv_freq, int rot, int interleaved, float factor, int norm, float eps,
                     const float *w_q, const float *w_k, const void *dq_out, long long ld_dqo, const void *dk_out,
                     long long ld_dko, void *dq, long long ld_dq, void *dk, long long ld_dk, float *dw_q, float *dw_k,
                     void *workspace, cdg_stream_t stream);
/* Bytes of cdg_qk_rope_grad's workspace; 0 for sizes it refuses.  Host only. */
size_t cdg_qk_rope_grad_workspace_bytes(long long tokens, int heads, int kv_heads, int dim);

/*
 * inv_freq (host, rot / 2 numbers) for cdg_qk_rope: f_i = base^(-2 i / rot),
 * stretched for contexts longer than the `trained` tokens a model has seen: a
 * frequency that makes `low` turns or fewer over them is divided by `stretch`,
 * one that makes `high` turns or more is kept, and those between are blended
 * linearly in their turns.  trained = 0: all are divided.  stretch = 1: none.
 */
int cdg_rope_frequencies(int rot, double base, double stretch, long long trained, double low, double high,
                         float *inv_freq);

#ifdef __cplusplus
}
#endif

#endif /* CDG_H */
