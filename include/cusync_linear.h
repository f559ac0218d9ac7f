/*
 * cusync_linear.h -- C ABI of the layers around the chains of cusync.h: single products with
 * everything that surrounds them in one kernel, the norm in front of them, 8-bit rows and
 * checkpoints, and their gradients.
 *
 *   norm         S = X + R;  y = w * S / sqrt(mean(S^2) + eps), in bf16 or 8 bits
 *   norm_grad    its gradients
 *   linear       Y = act(X x W + bias) + R, from bf16 or 8-bit operands; the
 *                pre-activations as an 8-bit checkpoint
 *   linear_grad  its gradients, from that checkpoint and X (bf16 or 8-bit rows)
 *
 * Conventions:
 *  - Tensors are contiguous, row-major, device-resident, 16-byte aligned and owned by the
 *    caller.  Activations, weights and parameters are bf16; weights have the reduction
 *    dimension contiguous ("[out, in]"), as in cusync.h.
 *  - 8-bit rows: q [rows, cols] e4m3 and scales [rows] fp32; row r stands for
 *    scales[r] * q[r] (a scale below 2^-126 in magnitude may count as 0).
 *  - 8-bit checkpoint of pre-activations z [M, parts, N] (parts: 2 for SwiGLU, gate then up,
 *    else 1): Zq [M, parts, N] e4m3 and Ze [M, parts, ceil(N / 32)] one byte for each 32
 *    columns (the last block may be shorter): z ~ Zq * 2^(Ze - 127), the smallest such power by
 *    which the block's finite values fit into +-448, at least 2^-126.
 *  - Values that are infinite or NaN become NaN in 8 bits (e4m3 has no infinity) and do not count
 *    for a scale.  The gradient at a pre-activation whose checkpoint is NaN is NaN, ReLU's too.
 *  - Calls enqueue kernels on the caller's stream, on the current device, and return; they
 *    allocate nothing, keep nothing between calls and can be recorded by stream capture.  A
 *    device's first cusync_norm_grad with rows, and its first cusync_linear or cusync_linear_grad
 *    with rows, sets the attributes of the kernels of the norms and of the linear layers; that, and CUDA's
 *    loading of a kernel at its first launch, may also happen in a capture, at the host's time.
 *    A `work` buffer belongs to one call at a time: two calls (or two captured graphs) that may
 *    run at the same time need buffers of their own.
 *  - Results do not depend on timing: the same inputs give the same bytes.  Calls of different
 *    sizes, with another num_sms or for other outputs (dX without dWt, dbias alone) may take different
 *    kernels, whose results differ by roundings.
 *  - cusync_norm holds for all finite S and w, and any finite eps that is not negative (elements that
 *    pass below 2^-126 on the way, beside much larger ones, lose bits).  Elsewhere these intermediate results are in 32 bits, whatever the result's own range: w * dY and w * dY * S in
 *    cusync_norm_grad, dY * up in the gradient of SwiGLU, e4m3 sums times a Ws beyond 2^+-80.  Sigmoids
 *    below 2^-126 (gates below -87.3) count as 0.
 *  - Outputs may not overlap inputs or one another, except where a function says so.
 *  - Sizes the kernels do not cover return CUSYNC_ERR_UNSUPPORTED; there is no fallback.
 */
#ifndef CUSYNC_LINEAR_H_
#define CUSYNC_LINEAR_H_

#include "cusync.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ norm */

typedef enum {
  CUSYNC_NORM_RMS = 0, /* y = w * S / sqrt(mean(S^2) + eps) */
  CUSYNC_NORM_NONE = 1 /* y = S: the addition and the 8-bit rows alone (w is not read) */
} cusync_norm_kind_t;

#define CUSYNC_NORM_MAX_D 32768

typedef struct {
  int64_t M;       /* rows (0 is allowed) */
  int64_t D;       /* columns: a multiple of 8, at most CUSYNC_NORM_MAX_D */
  int32_t kind;    /* cusync_norm_kind_t */
  float eps;       /* finite, not negative */
  int32_t num_sms; /* SMs that the gradient's grid is made for; 0 = all.  cusync_norm takes all that are free */
  int32_t _pad0;
} cusync_norm_desc_t;

typedef struct {
  int64_t grad_work_bytes; /* cusync_norm_grad */
} cusync_norm_info_t;

/* Pure host computation.  INVALID_ARG / UNSUPPORTED for a bad descriptor. */
cusync_status_t cusync_norm_info(const cusync_norm_desc_t* d, cusync_norm_info_t* out);

/* X [M, D]; R [M, D] or NULL (S = X then); w [D].  Outputs, each NULL where it is not
 * wanted (at least one is): S [M, D], the sum rounded to bf16; Y [M, D], y in bf16; Q
 * [M, D] and Qs [M], y as 8-bit rows (both or neither): Qs = max|y| / 448, at least 2^-126.
 * y is computed from the sum before its rounding.  S may be X or R (that buffer itself). */
cusync_status_t cusync_norm(const cusync_norm_desc_t* d, const void* X, const void* R, const void* w, void* S,
                            void* Y, void* Q, float* Qs, cusync_stream_t stream);

/* Gradients at S [M, D] (what cusync_norm wrote, or its X where it had no R) for dY [M, D]:
 * dX [M, D], which is R's gradient too, and dw [D] (NULL: not wanted).  dS [M, D] or NULL is the
 * gradient that reaches S along the residual path: it is added to dX, which may be dY or dS (that
 * buffer itself).  work: grad_work_bytes of scratch.  UNSUPPORTED for CUSYNC_NORM_NONE. */
cusync_status_t cusync_norm_grad(const cusync_norm_desc_t* d, const void* S, const void* w, const void* dY,
                                 const void* dS, void* work, void* dX, void* dw, cusync_stream_t stream);

/* ------------------------------------------------------------------ linear */

typedef enum {
  CUSYNC_LINEAR_NONE = 0,
  CUSYNC_LINEAR_RELU = 1,
  CUSYNC_LINEAR_GELU = 2,  /* GeLU_tanh */
  CUSYNC_LINEAR_SWIGLU = 3 /* silu(X x Wgate + b) * (X x Wup + b'); Wt [2*N, K]: Wgate^T's rows, then
                              Wup^T's; bias [2*N] */
} cusync_linear_act_t;

typedef enum {
  CUSYNC_LINEAR_BF16 = 0,
  CUSYNC_LINEAR_E4M3 = 1 /* X as 8-bit rows (linear: Wt too, a scale for each output column) */
} cusync_linear_dtype_t;

/* columns that share an exponent in a checkpoint */
#define CUSYNC_LINEAR_BLOCK 32

typedef struct {
  int64_t M;       /* rows of X (0 is allowed) */
  int64_t K;       /* columns of X: a multiple of 8 (E4M3: of 16) */
  int64_t N;       /* columns of Y: a multiple of 8 */
  int32_t act;     /* cusync_linear_act_t */
  int32_t dtype;   /* cusync_linear_dtype_t */
  int32_t num_sms; /* SMs that grids of persistent kernels are made for; 0 = all.  It does not keep others free:
                      products of few tiles and the gradients at the pre-activations take a block for
                      each piece of work, on all SMs */
  int32_t _pad0;
} cusync_linear_desc_t;

typedef struct {
  int64_t work_bytes;      /* cusync_linear */
  int64_t grad_work_bytes; /* cusync_linear_grad */
  int64_t parts;           /* 2 for SwiGLU, else 1 */
  int64_t blocks;          /* ceil(N / 32): Ze is [M, parts, blocks] */
} cusync_linear_info_t;

/* Pure host computation.  INVALID_ARG / UNSUPPORTED for a bad descriptor. */
cusync_status_t cusync_linear_info(const cusync_linear_desc_t* d, cusync_linear_info_t* out);

/* Y [M, N] of X [M, K] and Wt [parts*N, K] (E4M3: with Xs [M] and Ws [parts*N]; BF16: Xs and Ws
 * are NULL), bias [parts*N] or NULL, R [M, N] or NULL.  Sums, activation and additions in 32 bits,
 * one rounding.  Zq and Ze (both, or neither): the checkpoint of the pre-activations, bias
 * included.  Y may be R (that buffer itself).  work: work_bytes of scratch. */
cusync_status_t cusync_linear(const cusync_linear_desc_t* d, const void* X, const float* Xs, const void* Wt,
                              const float* Ws, const void* bias, const void* R, void* work, void* Y, void* Zq,
                              uint8_t* Ze, cusync_stream_t stream);

/* Gradients of cusync_linear for dY [M, N] (R's gradient is dY itself): dX [M, K], dWt
 * [parts*N, K] and dbias [parts*N] in bf16; each NULL where it is not wanted, at least one
 * is.  Zq and Ze: the checkpoint (NULL for act NONE).  Wt [parts*N, K] is always bf16 (needed
 * for dX).  X (needed for dWt): bf16, or E4M3: 8-bit rows with Xs.  The gradient at the
 * pre-activations is rounded to bf16 before the products that read it (with dWt of 8-bit rows:
 * times the fraction of the row's scale, a factor of at most 2); dbias is summed before that
 * rounding.  work: grad_work_bytes of scratch. */
cusync_status_t cusync_linear_grad(const cusync_linear_desc_t* d, const void* X, const float* Xs, const void* Wt,
                                   const void* Zq, const uint8_t* Ze, const void* dY, void* work, void* dX,
                                   void* dWt, void* dbias, cusync_stream_t stream);

/* Synchronise `stream` and read the error word of the last cusync_linear, cusync_linear_grad or
 * cusync_norm_grad call that used `work`: OK, or DEVICE if a device-internal wait gave up (the outputs of that call
 * are not valid).  code may be NULL.  UNSUPPORTED while the stream is being captured. */
cusync_status_t cusync_linear_check(const void* work, cusync_stream_t stream, uint32_t* code);

#ifdef __cplusplus
}
#endif
#endif /* CUSYNC_LINEAR_H_ */
