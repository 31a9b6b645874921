/*
 * libfno's training operators: what a training run takes beside the blocks of fno.h.
 *
 * A layer norm between blocks with its gradients, the global norm and clipping of the gradients
 * that the blocks return, and the AdamW update.  They need no plan.  Ownership, streams, the timer
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
