/*
 * cusync_moe.h -- C ABI of the mixture-of-experts layer: the MLP chains of cusync.h with
 * `experts` sets of weights, of which a router picks `top_k` for every token.
 *
 *   route      scores, groups, top-k, weights          and its gradient
 *   plan       which rows each expert computes
 *   mlp        Y[t] = sum_j weights[t,j] * MLP_{ids[t,j]}(X[t])   and its gradients
 *
 * Conventions:
 *  - Tensors are contiguous, row-major, device-resident, 16-byte aligned and owned by the
 *    caller.  Activations and expert weights are bf16, expert weights with the reduction
 *    dimension contiguous ("[out, in]"), as in cusync.h.
 *  - Calls enqueue kernels on the caller's stream, on the current device, and return; they
 *    allocate nothing, keep nothing between calls and can be recorded by stream capture (a
 *    device's first call with tokens sets the attributes that kernels need: make it before a
 *    capture; which call it is does not matter, CUDA loads other kernels at their first launch,
 *    also in a capture).
 *    A `plan` or `work` buffer belongs to one call at a time: two calls (or two captured
 *    graphs) that may run at the same time need buffers of their own.
 *  - Results do not depend on timing: the same inputs give the same bytes.  Calls of different
 *    sizes may take different kernels, whose results differ by roundings.
 *  - An id outside [0, experts) is an assignment to no expert: it adds nothing, and its
 *    gradient is zero.  The same expert may be chosen twice by a token; both count.
 *  - Sizes the kernels do not cover return CUSYNC_ERR_UNSUPPORTED; there is no fallback.
 */
#ifndef CUSYNC_MOE_H_
#define CUSYNC_MOE_H_

#include "cusync.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  CUSYNC_MOE_SOFTMAX = 0, /* over all experts of a token */
  CUSYNC_MOE_SIGMOID = 1  /* of each expert alone */
} cusync_moe_score_t;

typedef enum {
  CUSYNC_MOE_GELU = 0,  /* h = GeLU_tanh(X x W1); W1t [experts, N1, D] */
  CUSYNC_MOE_SWIGLU = 1 /* h = silu(X x Wgate) * (X x Wup); W1t [experts, 2*N1, D]: an
                           expert's Wgate^T rows, then its Wup^T rows */
} cusync_moe_act_t;

#define CUSYNC_MOE_MAX_EXPERTS 1024
#define CUSYNC_MOE_MAX_TOP_K 32
#define CUSYNC_MOE_MAX_GROUPS 32
/* T * top_k at most */
#define CUSYNC_MOE_MAX_ASSIGNMENTS 16777216
/* an expert's rows start at a multiple of this in the dispatch order */
#define CUSYNC_MOE_TILE_ROWS 128

typedef struct {
  int64_t T;           /* tokens (0 is allowed) */
  int64_t D;           /* model width: a multiple of 8 (mlp only) */
  int64_t N1;          /* an expert's hidden width: a multiple of 8 (mlp only) */
  int32_t experts;     /* 1 .. CUSYNC_MOE_MAX_EXPERTS */
  int32_t top_k;       /* 1 .. CUSYNC_MOE_MAX_TOP_K, at most group_limit * experts / groups */
  int32_t act;         /* cusync_moe_act_t */
  int32_t score;       /* cusync_moe_score_t */
  int32_t groups;      /* experts form this many equal groups of neighbours; 0 = 1 */
  int32_t group_limit; /* groups a token may use; 0 = all */
  int32_t group_top;   /* a group's rank is the sum of its 1 or 2 largest keys; 0 = 1 */
  int32_t renorm;      /* weights divided by the sum of the chosen scores */
  float scale;         /* factor on the weights (finite) */
  int32_t logits_f32;  /* logits and their gradient: 1 = fp32, 0 = bf16 */
  int32_t num_sms;     /* SMs that the grids of persistent kernels (the products, the router, the
                          MLP of few tokens) are made for; 0 = all */
  int32_t _pad0;
} cusync_moe_desc_t;

/* Buffer sizes, and where a plan's arrays start (in 32-bit words from its beginning). */
typedef struct {
  int64_t plan_bytes;
  int64_t work_bytes;      /* cusync_moe_mlp (0 where D or N1 is 0) */
  int64_t grad_work_bytes; /* cusync_moe_mlp_grad */
  int64_t slots;           /* rows of the dispatch order, every expert's tail included */
  int64_t counts;          /* [experts] assignments of each expert */
  int64_t offsets;         /* [experts + 1] first slot of each expert; then the end */
  int64_t slot_of;         /* [T, top_k] slot of an assignment, -1 = none */
  int64_t row_of;          /* [slots] assignment t * top_k + j of a slot, -1 = none */
} cusync_moe_info_t;

/* Pure host computation.  INVALID_ARG / UNSUPPORTED for a bad descriptor. */
cusync_status_t cusync_moe_info(const cusync_moe_desc_t* d, cusync_moe_info_t* out);

/* ids [T, top_k] int32 and weights [T, top_k] fp32 of logits [T, experts] (fp32 or bf16).
 *   s = softmax or sigmoid of the logits; key = s + bias (bias [experts] fp32, or NULL)
 *   groups > 1: only experts of the group_limit groups with the largest rank remain
 *   ids = the top_k largest keys, largest first; weights = scale * s[ids] (renorm: over
 *   the sum of the chosen s).  Scores grow with their logits: without a bias, and where ranks
 *   are single keys, experts go by their logits alone.
 * Equal keys, and equal ranks of groups, go to the lowest index; keys that 32 bits cannot
 * tell apart are compared in 64.  A logit of -inf or NaN, or a bias of -inf or NaN, is never
 * chosen; a bias of +inf comes before all others.  A logit of +inf has the score that it
 * tends to: 1 for sigmoid; for softmax an equal share with the token's other +inf, where all
 * other scores are 0.  A group with fewer keys left than its rank adds up ranks last.  Where
 * nothing is left to choose the id is -1 and the weight 0. */
cusync_status_t cusync_moe_route(const cusync_moe_desc_t* d, const void* logits, const float* bias, int32_t* ids,
                                 float* weights, cusync_stream_t stream);

/* dlogits [T, experts] (the logits' type) from dweights [T, top_k] fp32, with the ids that
 * cusync_moe_route gave for these logits (the bias has no gradient: it only selects). */
cusync_status_t cusync_moe_route_grad(const cusync_moe_desc_t* d, const void* logits, const int32_t* ids,
                                      const float* dweights, void* dlogits, cusync_stream_t stream);

/* The dispatch order of ids [T, top_k]: expert by expert, an expert's assignments in the
 * order of ids, each expert from a multiple of CUSYNC_MOE_TILE_ROWS.  Writes the arrays of
 * cusync_moe_info_t into plan (plan_bytes). */
cusync_status_t cusync_moe_plan(const cusync_moe_desc_t* d, const int32_t* ids, void* plan, cusync_stream_t stream);

/* Y [T, D] bf16 of X [T, D], W1t [experts, N1 or 2*N1, D], W2t [experts, D, N1], ids and
 * weights (fp32) [T, top_k].  work: work_bytes of scratch.  Y may not overlap an input. */
cusync_status_t cusync_moe_mlp(const cusync_moe_desc_t* d, const void* X, const void* W1t, const void* W2t,
                               const int32_t* ids, const float* weights, void* work, void* Y, cusync_stream_t stream);

/* Gradients of cusync_moe_mlp for dY [T, D]: dX [T, D], dW1t and dW2t (the weights' shapes;
 * every expert's is written, zero where no token chose it) in bf16, dweights [T, top_k] in
 * fp32.  The hidden layer is computed again from X: nothing of the forward pass is needed.
 * dweights are sums of products of fp32 values that the matrix unit has summed over D; it cuts
 * what lies behind 24 bits instead of rounding it, so they are up to about 3e-9 * D of their
 * value too small for dense normal operands (6e-6 at D = 2048), and exact where the sums are.
 * work: grad_work_bytes of scratch. */
cusync_status_t cusync_moe_mlp_grad(const cusync_moe_desc_t* d, const void* X, const void* W1t, const void* W2t,
                                    const int32_t* ids, const float* weights, const void* dY, void* work, void* dX,
                                    void* dW1t, void* dW2t, float* dweights, cusync_stream_t stream);

/* Synchronise `stream` and read the error word of the last call that used `buffer` (a plan
 * or work buffer): OK, or DEVICE if a device-internal wait gave up (the outputs of that
 * call are not valid).  code may be NULL.  UNSUPPORTED while the stream is being captured. */
cusync_status_t cusync_moe_check(const void* buffer, cusync_stream_t stream, uint32_t* code);

#ifdef __cplusplus
}
#endif
#endif /* CUSYNC_MOE_H_ */
