/*
 * muon_grad.h - C ABI of the list operators around the optimizer step on one gfx950 GPU: the
 * global gradient norm, clipping by it, and AdamW over a list of tensors (same library, same
 * conventions and status codes as muon.h).
 *
 * Why they are here: a training step takes the norm of all its gradients and scales them by
 * it before any optimizer runs.  muon_step and shampoo_step update the matrices; embeddings,
 * output heads, norm vectors and biases are many tensors of both types that AdamW updates
 * (MatrixFSDP summary, Methodology §1: the non-matrix parameters keep standard AdamW).
 *
 * What is computed:
 *   norm    L2: n = sqrt(sum over all tensors and elements of g^2); inf: n = max |g|.  An
 *           infinity gives inf, a NaN gives NaN (of either kind of norm).
 *   clip    c = min(1, max_norm / (n + 1e-6)), NaN where n is NaN; g <- c g.
 *   AdamW   with w = master if there is one, else param, gs = c g (c = 1 without clipping)
 *           and t = step >= 1:
 *             m <- b1 m + (1-b1) gs;  v <- b2 v + (1-b2) gs^2;
 *             w <- w - lr ((m / (1-b1^t)) / (sqrt(v / (1-b2^t)) + eps) + weight_decay decay w);
 *             param <- w, rounded to param's type.
 *   muon_step_clipped runs muon_step with M <- beta M + c G.
 * The norm is a float in device memory, so clipping needs no transfer to the host.  Where
 * several ranks own parts of the gradients, each takes its part's norm, the caller reduces
 * them (sum of squares, or maximum), and every rank clips by the reduced value.
 * shampoo_step and muon_step_noalloc take no clip: scale their gradients in place first.
 *
 * Precision: the squares and sums of the L2 norm are 64-bit, in a fixed order (results are
 * bitwise reproducible), so no gradient is too small or too large for it; the norm is rounded
 * to fp32 once (inf above the fp32 range).  c and its product with g are fp32; a bf16
 * gradient is rounded (to nearest even) once, on store.  AdamW runs in fp32, and a bf16 param
 * is rounded once.  Without a master that rounding loses updates below half a bf16 step.
 * The betas of adamw_hparams are floats, and are taken as what they are: 0.9999f is
 * 0.99989998.., so 1 - 0.9999f, and v with it, is 1.7e-4 off what 0.9999 gives.  The _double
 * entry points take 64-bit hyperparameters; m and v then follow the betas given.
 *
 * Lists: a list is laid out once (muon_grad_list_init, adamw_list_init: the tensors'
 * addresses and sizes, and a map of their parts, go to the caller's workspace) and then used
 * by any number of calls, as long as the tensors stay where they are; their values may
 * change.  The layout is enqueued on the stream given (through kernel arguments: no host
 * buffer, no copy, so it may be captured, and the list is then for calls on streams of the same
 * capture only, MUON_EINVAL elsewhere: its table is not there before a replay); uses on another
 * stream must be ordered after it by the caller.  Calls of a list, replays of graphs that hold
 * them among these, come one after another (two at once need two lists): two norms at once mix
 * their partial results, and what they write is undefined.  Later calls are right again.  A list
 * is used on the device it was laid out on.
 */
#ifndef MUON_GRAD_H
#define MUON_GRAD_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One gradient: n contiguous elements of `dtype`, aligned to their size.  n may be 0 (grad may
 * then be NULL). */
typedef struct muon_grad {
  void* grad;
  int64_t n;
  int32_t dtype;    /* muon_dtype */
  int32_t reserved; /* must be 0 */
} muon_grad;

/* One parameter tensor of n contiguous elements: param, m, v and master are updated in place,
 * grad is read only.  All aligned to their element size. */
typedef struct adamw_tensor {
  void* param;
  const void* grad;
  float* m;
  float* v;
  float* master;       /* fp32 master copy of a bf16 param, or NULL */
  int64_t n;
  int32_t param_dtype; /* muon_dtype */
  int32_t grad_dtype;  /* muon_dtype */
  float decay;         /* factor on the weight decay of this tensor (0: none), finite */
  int32_t reserved;    /* must be 0 */
} adamw_tensor;

/* A laid-out list: opaque, filled by the init call, copied freely. */
typedef struct muon_grad_list {
  uint64_t opaque[8];
} muon_grad_list;
typedef struct adamw_list {
  uint64_t opaque[8];
} adamw_list;

/* What to clip by: the norm (a float in device memory, read when the kernels run) and the
 * limit. */
typedef struct muon_clip {
  const float* norm;
  float max_norm;   /* finite, >= 0 */
  int32_t reserved; /* must be 0 */
} muon_clip;

typedef enum muon_norm_kind { MUON_NORM_L2 = 0, MUON_NORM_INF = 1 } muon_norm_kind;

/* Bytes of device workspace a list needs.  Host only, no HIP call.  MUON_EINVAL for sizes,
 * dtypes, NULL or misaligned pointers, MUON_EALIAS when gradients of a muon_grad list overlap
 * each other, or an output of an adamw_tensor list overlaps another output or any gradient;
 * at most 2^20 tensors and 2^40 elements. */
int muon_grad_list_size(const muon_grad* grads, int32_t count, size_t* bytes);
int adamw_list_size(const adamw_tensor* tensors, int32_t count, size_t* bytes);

/* Lay out a list in `workspace` (device memory of at least the size above, 256-byte aligned,
 * owned by the caller, kept as long as the list is used and written by nothing else) and fill
 * *list.  count == 0 is a list of no tensors (its norm is 0).  Errors as the size calls,
 * MUON_ENOSPC, and MUON_EALIAS when the workspace overlaps a tensor of the list. */
int muon_grad_list_init(const muon_grad* grads, int32_t count, void* workspace, size_t workspace_bytes,
                        void* hip_stream, muon_grad_list* list);
int adamw_list_init(const adamw_tensor* tensors, int32_t count, void* workspace, size_t workspace_bytes,
                    void* hip_stream, adamw_list* list);

/* *capture <- the identity of the graph capture that hip_stream takes part in, 0 for none:
 * what tells whether a list that was laid out in a capture can be used on the stream.
 * Enqueues nothing.  MUON_EINVAL for a capture that was broken off. */
int muon_stream_capture(void* hip_stream, uint64_t* capture);

/* *norm <- the norm of all gradients of the list (4-byte aligned device memory that is no part
 * of a gradient; MUON_EALIAS when it lies in the list's workspace, for this and the calls
 * below).  kind: muon_norm_kind. */
int muon_grad_norm(const muon_grad_list* list, int32_t kind, float* norm, void* hip_stream);

/* Scale every gradient of the list by the coefficient of `clip`, in place.  Where the
 * coefficient is 1 nothing is read or written.  clip->norm is no part of a gradient. */
int muon_grad_clip(const muon_grad_list* list, const muon_clip* clip, void* hip_stream);

/* muon_grad_norm, then muon_grad_clip by its result. */
int muon_grad_clip_norm(const muon_grad_list* list, int32_t kind, float max_norm, float* norm, void* hip_stream);

/* Hyperparameters of AdamW in 64 bits: lr, eps and weight_decay are rounded to fp32, the betas,
 * in [0, 1), are not (nor 1 - beta). */
typedef struct adamw_hparams_double {
  double lr;
  double beta1;
  double beta2;
  double eps;
  double weight_decay;
  int32_t step;
  int32_t reserved; /* must be 0 */
} adamw_hparams_double;

/* adamw_step (muon.h) with 64-bit hyperparameters. */
int adamw_step_double(float* p, const float* g, float* m, float* v, int64_t n, const adamw_hparams_double* hp,
                      void* hip_stream);

/* AdamW over the list.  hp as adamw_step; clip may be NULL (no clipping), and clip->norm is no
 * part of a tensor that the list updates. */
int adamw_list_step(const adamw_list* list, const adamw_hparams* hp, const muon_clip* clip, void* hip_stream);
int adamw_list_step_double(const adamw_list* list, const adamw_hparams_double* hp, const muon_clip* clip,
                           void* hip_stream);

/* muon_step whose gradients are scaled by the coefficient of `clip` as the momentum reads
 * them: M <- beta M + c G, in fp32, the gradients unchanged.  clip NULL is muon_step;
 * MUON_EALIAS when clip->norm lies in a param, a momentum or the workspace. */
int muon_step_clipped(const muon_matrix* mats, int32_t count, const muon_hparams* hp, const muon_clip* clip,
                      void* workspace, size_t workspace_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* MUON_GRAD_H */
