// Declarations shared by the training operators' kernels and their entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "fno.h"

namespace fno {

// ---- layer norm (kernels_layernorm.hip) ------------------------------------------------------
struct NormArgs {
  int64_t batch, npts;
  int channels;
  int64_t x_stride, y_stride, gx_stride;  // elements between batch entries
  float eps;
};
hipError_t launch_layer_norm_fwd(const NormArgs& a, int dtype, const void* x, const float* gamma,
                                 const float* beta, void* y, float* stats, hipStream_t s);
// rows of partial sums that the backward writes for the weight gradients, each [2][channels] floats
int layer_norm_parts(const NormArgs& a, int dtype);
// part: layer_norm_parts rows (unused when both weight gradients are NULL)
hipError_t launch_layer_norm_bwd(const NormArgs& a, int dtype, const void* x, const float* gamma,
                                 const float* stats, const void* gy, void* gx, float* part,
                                 hipStream_t s);
hipError_t launch_layer_norm_finish(const NormArgs& a, int nparts, const float* part,
                                    float* ggamma, float* gbeta, hipStream_t s);

// ---- tensor lists (kernels_optim.hip) --------------------------------------------------------
// A list travels in kernel arguments (at most 4 KB a launch), `Cap` tensors at a time: no device
// table to upload or to go stale.  Work is cut into chunks of kChunk elements that do not cross a
// tensor's end; first[k] is the first chunk of tensor k.
constexpr int64_t kChunk = 8192;
template <int Lists, int Cap>
struct TensorTable {
  void* ptr[Lists][Cap];
  int64_t elems[Cap];
  uint32_t first[Cap + 1];
  uint8_t dtype[Cap];  // of list 0 in the low four bits, of list 1 in the high ones
  int32_t count;
};
constexpr int kNormTensors = 100;   // tensors a launch: gradients and outputs
constexpr int kAdamTensors = 80;    // parameters, gradients, two moments
typedef TensorTable<2, kNormTensors> NormTable;
typedef TensorTable<4, kAdamTensors> AdamTable;
static_assert(sizeof(NormTable) <= 3800 && sizeof(AdamTable) <= 3800, "kernel argument space");
constexpr int kNormParts = 1024;    // partial sums a launch

// one partial sum of squares per work-group into part[0 .. groups)
hipError_t launch_norm_part(const NormTable& t, int groups, double* part, hipStream_t s);
hipError_t launch_norm_finish(const double* part, int nparts, float max_norm, float grad_scale,
                              float* record, hipStream_t s);
hipError_t launch_clip(const NormTable& t, int groups, const float* record, hipStream_t s);

struct AdamArgs {
  float beta1, beta2, one_minus_beta1, one_minus_beta2;
  float decay;       // 1 - lr weight_decay
  float step_size;   // lr / (1 - beta1^t)
  float inv_bias2;   // 1 / sqrt(1 - beta2^t)
  float eps;
};
hipError_t launch_adamw(const AdamTable& t, int groups, const AdamArgs& a, const float* record,
                        hipStream_t s);

}  // namespace fno
