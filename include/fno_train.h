/*
 * libfno's training operators: what a training run takes beside the blocks of fno.h.
 *
 * A layer norm, a group norm with its activation, and dropout between blocks, each with its
 * gradients, the global norm and clipping of the gradients that the blocks return, and the AdamW
 * update.  They need no plan.  Ownership, streams, the timer
 * and errors are fno.h's.  Unlike its calls these accept data pointers at any multiple of the
 * element size (fields cut out of larger ones, parameters packed into one buffer); float32 vectors
 * (gamma, beta, the statistics and the record) at 4 bytes, workspaces and tables at 16.  float32,
 * bfloat16 and IEEE half data (fno_dtype); every statistic, sum and state is float32 or wider, and
 * a half-format result is rounded to nearest-even once.
 */
#ifndef LIBFNO_FNO_TRAIN_H
#define LIBFNO_FNO_TRAIN_H

#include "fno.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Layer norm over the channels of a field [batch][channels][npts], at each point:
 *   mu = mean_c x;  r = 1 / sqrt(mean_c (x - mu)^2 + eps);  y = gamma[c] (x - mu) r + beta[c]
 * npts = 1 is the row form: `batch` rows of `channels` entries.  Strides are in elements, from
 * one batch entry to the next; inside an entry the data is packed.  The strides of inputs may be
 * anything >= 0 (0: one entry for all), those of outputs at least channels * npts. */
typedef struct fno_layer_norm_desc {
  int32_t dtype;          /* fno_dtype of x, y, grad_y, grad_x                        */
  int32_t reserved;       /* must be 0                                               */
  int64_t batch;          /* >= 0; with batch or npts 0 there are no rows             */
  int64_t channels;       /* >= 1, below 2^31                                        */
  int64_t npts;           /* >= 0                                                    */
  int64_t x_stride;       /* of x                                                    */
  int64_t y_stride;       /* of y (forward), of grad_y (backward)                    */
  int64_t grad_x_stride;  /* of grad_x (the forward does not look at it)             */
  double eps;             /* finite, >= 0                                            */
} fno_layer_norm_desc;

/* gamma and beta (float32 [channels]) may be NULL: 1 and 0.  stats (nullable) receives float32
 * [2][batch * npts]: mu, then r, for the backward.  y may be x (the same pointer and stride).  A
 * non-finite x makes its own row non-finite and no other. */
fno_status fno_layer_norm_fwd(const fno_layer_norm_desc* desc, const void* x, const float* gamma,
                              const float* beta, void* y, float* stats, void* stream);

/* Bytes of workspace of fno_layer_norm_bwd on this descriptor (0 for small fields, which need
 * none: workspace may then be NULL). */
fno_status fno_layer_norm_workspace_bytes(const fno_layer_norm_desc* desc, size_t* bytes);

/* Backward from the forward's x and stats.  With h = (x - mu) r and g = gamma grad_y:
 *   grad_x = r (g - mean_c g - h mean_c(g h)),
 *   grad_gamma[c] = sum grad_y h,  grad_beta[c] = sum grad_y  (over batch and npts; float32).
 * Outputs may be NULL to skip them; they are overwritten (grad_gamma and grad_beta with zeros
 * when there are no rows), and the same bits run to run.  grad_x may be grad_y or x (the same
 * pointer and stride). */
fno_status fno_layer_norm_bwd(const fno_layer_norm_desc* desc, const void* x, const float* gamma,
                              const float* stats, const void* grad_y, void* grad_x,
                              float* grad_gamma, float* grad_beta, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Dropout from a counter: the mask is a function of the numbers here and of each element's index,
 * so that nothing is stored and a backward pass drops what its forward dropped.  With
 * T = round(65536 p), element i of a tensor (counted through the packed tensor in memory order,
 * wherever its entries lie) is dropped, 0, where its 16 bits are below T, and is multiplied by
 * 65536 / (65536 - T) elsewhere.  Its bits are half (the lower for even i) of word (i % 8) / 2 of
 * Philox4x32-10 of the counter (i / 8, draw + *counter) under the key seed, each 64 bits with the
 * low word first.  Different draws under a seed are different masks. */
typedef struct fno_dropout {
  double p;                 /* 0 <= p, T <= 65535; T = 0 drops nothing                        */
  uint64_t seed;
  uint64_t draw;            /* of this layer and step                                         */
  const uint64_t* counter;  /* on the device, read when the call runs, 8-byte aligned: what a */
                            /* captured graph moves on between its replays; NULL: 0           */
} fno_dropout;

typedef struct fno_dropout_desc {
  int32_t dtype;            /* fno_dtype of x, residual and y                                 */
  int32_t reserved;         /* must be 0                                                      */
  int64_t batch, elems;     /* >= 0: entries, packed elements of an entry                     */
  int64_t x_stride;         /* elements between entries of x, of grad_y in the backward: >= 0 */
  int64_t residual_stride;  /* of residual: >= 0                                              */
  int64_t y_stride;         /* of y, of grad_x in the backward: >= elems                      */
} fno_dropout_desc;

/* y = residual + dropped x (residual NULL: 0).  y may be x or residual (the same pointer and
 * stride). */
fno_status fno_dropout_fwd(const fno_dropout_desc* desc, const fno_dropout* drop, const void* x,
                           const void* residual, void* y, void* stream);
/* grad_x = dropped grad_y (the residual's gradient is grad_y itself); grad_x may be grad_y. */
fno_status fno_dropout_bwd(const fno_dropout_desc* desc, const fno_dropout* drop,
                           const void* grad_y, void* grad_x, void* stream);

typedef enum fno_activation {
  FNO_ACT_NONE = 0,
  FNO_ACT_GELU = 1, /* u/2 (1 + erf(u/sqrt 2)) */
  FNO_ACT_SILU = 2  /* u / (1 + e^-u)          */
} fno_activation;

/* Group norm over fields [batch][channels][npts], or channels last [batch][npts][channels], with an
 * activation and dropout in the same pass.  For each entry and each of the `groups` runs of
 * channels / groups channels, over all points, m = npts channels / groups entries:
 *   mu = sum x / m;  r = 1 / sqrt(sum (x - mu)^2 / m + eps);
 *   y = drop(act(gamma[c] (x - mu) r + beta[c]))
 * npts = 1 (the same memory either way) is the form of tokens with a norm for each head.  Strides
 * as in fno_layer_norm_desc. */
typedef struct fno_group_norm_desc {
  int32_t dtype;          /* fno_dtype of x, y, grad_y, grad_x                    */
  int32_t channels_last;  /* 0 or 1                                              */
  int32_t activation;     /* fno_activation                                      */
  int32_t reserved;       /* must be 0                                           */
  int64_t batch;          /* >= 0, below 2^31; without entries or points: no rows */
  int64_t channels;       /* >= 1, below 2^30                                    */
  int64_t groups;         /* >= 1, divides channels                              */
  int64_t npts;           /* >= 0                                                */
  int64_t x_stride;       /* of x                                                */
  int64_t y_stride;       /* of y (forward), of grad_y (backward)                */
  int64_t grad_x_stride;  /* of grad_x (the forward does not look at it)         */
  double eps;             /* finite, >= 0; added as a float32                    */
} fno_group_norm_desc;

/* Bytes of workspace of the two calls on this descriptor (either may be 0, its workspace then
 * NULL; fwd and bwd nullable).  Does not look at grad_x_stride either. */
fno_status fno_group_norm_workspace_bytes(const fno_group_norm_desc* desc, size_t* fwd,
                                          size_t* bwd);

/* drop NULL: no dropout.  gamma and beta (float32 [channels]) may be NULL: 1 and 0.  stats
 * (nullable) receives float32 [2][batch][groups]: mu, then r, for the backward (0 and 0 where there
 * are no points).  y may be x (the same pointer and stride).  A non-finite x makes its own group of its entry non-finite, where that
 * is not dropped, and no other. */
fno_status fno_group_norm_fwd(const fno_group_norm_desc* desc, const fno_dropout* drop,
                              const void* x, const float* gamma, const float* beta, void* y,
                              float* stats, void* workspace, size_t workspace_bytes, void* stream);

/* Backward from the forward's x, stats and mask.  With h = (x - mu) r and
 * g = act'(gamma h + beta) drop(grad_y):
 *   grad_x = r (gamma g - sum(gamma g) / m - h sum(gamma g h) / m)  (sums over the group),
 *   grad_gamma[c] = sum g h,  grad_beta[c] = sum g  (over batch and npts; float32).
 * Outputs may be NULL to skip them; they are overwritten (grad_gamma and grad_beta with zeros when
 * there are no rows), and the same bits run to run.  grad_x may be grad_y or x (the same pointer
 * and stride). */
fno_status fno_group_norm_bwd(const fno_group_norm_desc* desc, const fno_dropout* drop,
                              const void* x, const float* gamma, const float* beta,
                              const float* stats, const void* grad_y, void* grad_x,
                              float* grad_gamma, float* grad_beta, void* workspace,
                              size_t workspace_bytes, void* stream);

/* One entry of a tensor list: `elems` packed elements.  A complex64 tensor is a float32 one of
 * twice its elements. */
typedef struct fno_tensor {
  void* data;        /* NULL only with elems 0 */
  int64_t elems;     /* 0 .. 2^36              */
  int32_t dtype;     /* fno_dtype              */
  int32_t reserved;  /* must be 0              */
} fno_tensor;

/* A list of tensors that one call goes over (gradients, parameters, moments), made once for
 * buffers that stay: a host object, and a device table of their addresses and of the chunks that
 * the work is cut into, in memory of the caller's (16-byte aligned, fno_tensor_list_bytes).  The
 * table is uploaded on `stream`, which must not be capturing; calls on other streams are ordered
 * after that by the caller, who keeps table and tensors until the calls have run.  Making a list
 * launches nothing; any number of calls may use one list at a time. */
typedef struct fno_tensor_list fno_tensor_list;
fno_status fno_tensor_list_bytes(int64_t count, const fno_tensor* tensors, size_t* bytes);
fno_status fno_tensor_list_create(int64_t count, const fno_tensor* tensors, void* table,
                                  size_t table_bytes, void* stream, fno_tensor_list** out);
fno_status fno_tensor_list_destroy(fno_tensor_list* list); /* host only; NULL accepted */

/* Bytes of workspace of fno_grad_norm and fno_clip_grad_norm on a list. */
fno_status fno_grad_norm_workspace_bytes(const fno_tensor_list* grads, size_t* bytes);

/* The global norm of a list of gradients that carry the loss scale grad_scale (1 without one):
 *   norm = sqrt(sum over all elements of g^2) / grad_scale,
 *   factor = min(1, max_norm / norm) / grad_scale   (NaN when a gradient is infinite or NaN),
 * written to the device floats record[0] = norm, record[1] = factor.  The sum, the norm and the
 * factor are taken in float64 (no float32 gradient over- or underflows them) in a fixed order and
 * rounded at the end: the norm of finite gradients may come out as infinity, above float32's
 * range, beside a factor that is right.  max_norm > 0, INFINITY for no clipping; grad_scale finite
 * and > 0.  A tensor that is listed twice counts twice (but what a call writes, clipped gradients,
 * parameters or moments, may be listed once only). */
fno_status fno_grad_norm(const fno_tensor_list* grads, float max_norm, float grad_scale,
                         float* record, void* workspace, size_t workspace_bytes, void* stream);

/* fno_grad_norm, then out = factor * g for every tensor.  out lists as many tensors of the same
 * elems, each of its gradient's dtype or float32 (where half gradients lose their loss scale
 * without underflow), each its gradient itself or apart from all gradients.  With a factor of
 * exactly 1 a tensor that is its own output is left as it is; a gradient that is infinite or NaN
 * makes every output NaN. */
fno_status fno_clip_grad_norm(const fno_tensor_list* grads, const fno_tensor_list* out,
                              float max_norm, float grad_scale, float* record, void* workspace,
                              size_t workspace_bytes, void* stream);

typedef struct fno_adamw_desc {
  double lr;            /* finite                                                 */
  double beta1, beta2;  /* in [0, 1)                                              */
  double eps;           /* finite, >= 0                                           */
  double weight_decay;  /* finite                                                 */
  int64_t step;         /* t >= 1: this update's number, for the bias corrections */
} fno_adamw_desc;

/* One AdamW update of a list of float32 parameters, in place, from gradients of any dtype:
 *   g' = factor g (record[1] of fno_grad_norm; record NULL: g' = g)
 *   m = beta1 m + (1 - beta1) g';  v = beta2 v + (1 - beta2) g'^2
 *   p = p - lr weight_decay p - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * (m = exp_avg, v = exp_avg_sq, float32).  What desc holds goes into the launch as values: a
 * captured call replays this one update, number, rate and all.  When record's factor is not finite
 * the update is skipped: nothing is written, so that a loss-scaled run needs no synchronisation to
 * drop such a step. */
fno_status fno_adamw(const fno_tensor_list* params, const fno_tensor_list* grads,
                     const fno_tensor_list* exp_avg, const fno_tensor_list* exp_avg_sq,
                     const fno_adamw_desc* desc, const float* record, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBFNO_FNO_TRAIN_H */
