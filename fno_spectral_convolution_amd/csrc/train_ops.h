// Declarations shared by the training operators' kernels and their entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "fno_train.h"

namespace fno {

// ---- layer norm (kernels_layernorm.hip) ------------------------------------------------------
struct NormArgs {
  int64_t batch, npts;
  int channels;
  int64_t x_stride, y_stride, gx_stride;  // elements between batch entries
  float eps;
  bool stream;  // the output goes past the caches (set by the launches)
};
hipError_t launch_layer_norm_fwd(const NormArgs& a, int dtype, const void* x, const float* gamma,
                                 const float* beta, void* y, float* stats, hipStream_t s);
// rows of partial sums that the backward writes for the weight gradients, each [2][channels] floats
int layer_norm_parts(const NormArgs& a, int dtype);
// the whole backward; part: layer_norm_parts rows (unused when both weight gradients are NULL);
// without rows only the weight gradients' zeros
hipError_t launch_layer_norm_bwd(const NormArgs& a, int dtype, const void* x, const float* gamma,
                                 const float* stats, const void* gy, void* gx, float* ggamma,
                                 float* gbeta, float* part, hipStream_t s);

// the sums over `parts` rows [2][channels] of partial sums, in a fixed order: row 0's to ggamma, row
// 1's to gbeta (nullable)
hipError_t launch_weight_sums(int channels, int parts, const float* part, float* ggamma,
                              float* gbeta, hipStream_t s);

// ---- dropout (kernels_dropout.hip) -----------------------------------------------------------
struct DropArgs {
  uint32_t threshold;  // of 65536; 0: nothing is dropped
  float scale;         // 65536 / (65536 - threshold)
  uint64_t seed, draw;
  const uint64_t* counter;  // on the device, added to draw; nullable
};
struct DropoutArgs {
  DropArgs drop;
  int64_t batch, per;                   // entries, elements of an entry
  int64_t x_stride, r_stride, y_stride; // elements between entries
  bool stream;                          // the output goes past the caches (set by the launch)
};
hipError_t launch_dropout(const DropoutArgs& a, int dtype, const void* x, const void* residual,
                          void* y, hipStream_t s);

// ---- group norm (kernels_groupnorm.hip) ------------------------------------------------------
struct GroupArgs {
  int64_t batch, npts;
  int channels, groups;
  bool last;  // channels last: [batch][npts][channels]
  int act;    // fno_activation
  int64_t x_stride, y_stride, gx_stride;  // elements between batch entries
  float eps;
  DropArgs drop;
};
size_t group_norm_fwd_bytes(const GroupArgs& a, int dtype);
size_t group_norm_bwd_bytes(const GroupArgs& a, int dtype);
hipError_t launch_group_norm_fwd(const GroupArgs& a, int dtype, const void* x, const float* gamma,
                                 const float* beta, void* y, float* stats, void* ws,
                                 hipStream_t s);
hipError_t launch_group_norm_bwd(const GroupArgs& a, int dtype, const void* x, const float* gamma,
                                 const float* beta, const float* stats, const void* gy, void* gx,
                                 float* ggamma, float* gbeta, void* ws, hipStream_t s);

// ---- tensor lists (kernels_optim.hip) --------------------------------------------------------
// A list's device table: its entries, then the entry that holds each chunk.  Chunks are kChunk
// elements of one tensor (its last one fewer); they are the grain at which work is shared out.
constexpr int64_t kChunk = 2048;
struct TensorEntry {
  void* data;
  int64_t elems;
  uint32_t first;  // its first chunk
  int32_t dtype;
};
struct TensorTable {
  const TensorEntry* entry;
  const uint32_t* of_chunk;
  uint32_t chunks;
  int64_t bytes;  // of all its tensors
};
// how the partial sums of squares become a record
struct NormRecord {
  int nparts;
  float max_norm, grad_scale;
};
// most partial sums of the norm: eight work-groups of four waves fill a compute unit
constexpr int kNormParts = 2048;

// one partial sum of squares per work-group into part[0 .. groups); again: the call's next launch
// reads the tensors once more
hipError_t launch_norm_part(const TensorTable& t, int groups, double* part, bool again,
                            hipStream_t s);
hipError_t launch_norm_finish(const double* part, const NormRecord& r, float* record,
                              hipStream_t s);
// writes the record too
hipError_t launch_clip(const TensorTable& t, const TensorTable& out, const double* part,
                       const NormRecord& r, float* record, hipStream_t s);

struct AdamArgs {
  float beta1, beta2, one_minus_beta1, one_minus_beta2;
  float decay;       // lr weight_decay
  float step_size;   // lr / (1 - beta1^t)
  float inv_bias2;   // 1 / sqrt(1 - beta2^t)
  float eps;
};
hipError_t launch_adamw(const TensorTable& params, const TensorTable& grads,
                        const TensorTable& exp_avg, const TensorTable& exp_avg_sq,
                        const AdamArgs& a, const float* record, hipStream_t s);

}  // namespace fno
