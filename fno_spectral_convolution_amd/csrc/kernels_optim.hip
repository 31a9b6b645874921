// The global gradient norm over a list of tensors, clipping, and the AdamW update.
#include "train_device.h"
#include "train_ops.h"

namespace fno {
namespace {

constexpr int kThreads = 256;

// the tensor that holds chunk `c` of the list: the last k with first[k] <= c
template <int Lists, int Cap>
__device__ __forceinline__ int tensor_of(const TensorTable<Lists, Cap>& t, uint32_t c) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// fixed-order sum of one double per thread; every thread gets it
__device__ __forceinline__ double group_sum(double v, double* s_red) {
  const int tid = threadIdx.x;
  __syncthreads();
  s_red[tid] = v;
  __syncthreads();
  for (int w = kThreads / 2; w > 0; w >>= 1) {
    if (tid < w) s_red[tid] += s_red[tid + w];
    __syncthreads();
  }
  return s_red[0];
}

template <typename T>
__device__ __forceinline__ double sum_squares(const T* p, int n) {
  double a = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const double g = (double)to_float(p[i]);
    a += g * g;
  }
  return a;
}

__global__ __launch_bounds__(kThreads) void k_norm_part(NormTable t, double* part) {
  __shared__ double s_red[kThreads];
  double a = 0.0;
  for (uint32_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int k = tensor_of(t, c);
    const int64_t at = (int64_t)(c - t.first[k]) * kChunk, left = t.elems[k] - at;
    const int n = (int)(left < kChunk ? left : kChunk);
    const int d = t.dtype[k] & 15;
    if (d == FNO_DTYPE_F32) a += sum_squares(static_cast<const float*>(t.ptr[0][k]) + at, n);
    else if (d == FNO_DTYPE_BF16) a += sum_squares(static_cast<const __bf16*>(t.ptr[0][k]) + at, n);
    else a += sum_squares(static_cast<const _Float16*>(t.ptr[0][k]) + at, n);
  }
  a = group_sum(a, s_red);
  if (threadIdx.x == 0) part[blockIdx.x] = a;
}

__global__ __launch_bounds__(kThreads) void k_norm_finish(const double* part, int nparts,
                                                          float max_norm, float grad_scale,
                                                          float* record) {
  __shared__ double s_red[kThreads];
  double a = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kThreads) a += part[i];
  a = group_sum(a, s_red);
  if (threadIdx.x == 0) {
    const double norm = sqrt(a) / (double)grad_scale;
    double f = norm > (double)max_norm ? (double)max_norm / norm : 1.0;
    if (!(norm < (double)INFINITY)) f = (double)NAN;
    record[0] = (float)norm;
    record[1] = (float)(f / (double)grad_scale);
  }
}

template <typename T, typename U>
__device__ __forceinline__ void scale_chunk(const T* p, U* o, int n, float f) {
  for (int i = threadIdx.x; i < n; i += kThreads) o[i] = from_float<U>(to_float(p[i]) * f);
}

__global__ __launch_bounds__(kThreads) void k_clip(NormTable t, const float* record) {
  const float f = record[1];
  for (uint32_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int k = tensor_of(t, c);
    const int64_t at = (int64_t)(c - t.first[k]) * kChunk, left = t.elems[k] - at;
    const int n = (int)(left < kChunk ? left : kChunk);
    const int d = t.dtype[k] & 15, o = t.dtype[k] >> 4;
    if (f == 1.0f && t.ptr[0][k] == t.ptr[1][k]) continue;
    if (d == FNO_DTYPE_F32) {
      scale_chunk(static_cast<const float*>(t.ptr[0][k]) + at,
                  static_cast<float*>(t.ptr[1][k]) + at, n, f);
    } else if (d == FNO_DTYPE_BF16) {
      const __bf16* p = static_cast<const __bf16*>(t.ptr[0][k]) + at;
      if (o == FNO_DTYPE_F32) scale_chunk(p, static_cast<float*>(t.ptr[1][k]) + at, n, f);
      else scale_chunk(p, static_cast<__bf16*>(t.ptr[1][k]) + at, n, f);
    } else {
      const _Float16* p = static_cast<const _Float16*>(t.ptr[0][k]) + at;
      if (o == FNO_DTYPE_F32) scale_chunk(p, static_cast<float*>(t.ptr[1][k]) + at, n, f);
      else scale_chunk(p, static_cast<_Float16*>(t.ptr[1][k]) + at, n, f);
    }
  }
}

template <typename T>
__device__ __forceinline__ void adamw_chunk(float* p, const T* g, float* m, float* v, int n,
                                            const AdamArgs& a, float f) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const float gi = to_float(g[i]) * f;
    const float mi = a.beta1 * m[i] + a.one_minus_beta1 * gi;
    const float vi = a.beta2 * v[i] + a.one_minus_beta2 * gi * gi;
    m[i] = mi;
    v[i] = vi;
    p[i] = a.decay * p[i] - a.step_size * mi / (sqrtf(vi) * a.inv_bias2 + a.eps);
  }
}

__global__ __launch_bounds__(kThreads) void k_adamw(AdamTable t, AdamArgs a, const float* record) {
  const float f = record ? record[1] : 1.0f;
  if (!(fabsf(f) < INFINITY)) return;  // the gradients were not finite: no update
  for (uint32_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int k = tensor_of(t, c);
    const int64_t at = (int64_t)(c - t.first[k]) * kChunk, left = t.elems[k] - at;
    const int n = (int)(left < kChunk ? left : kChunk);
    const int d = t.dtype[k] >> 4;
    float* p = static_cast<float*>(t.ptr[0][k]) + at;
    float* m = static_cast<float*>(t.ptr[2][k]) + at;
    float* v = static_cast<float*>(t.ptr[3][k]) + at;
    if (d == FNO_DTYPE_F32)
      adamw_chunk(p, static_cast<const float*>(t.ptr[1][k]) + at, m, v, n, a, f);
    else if (d == FNO_DTYPE_BF16)
      adamw_chunk(p, static_cast<const __bf16*>(t.ptr[1][k]) + at, m, v, n, a, f);
    else
      adamw_chunk(p, static_cast<const _Float16*>(t.ptr[1][k]) + at, m, v, n, a, f);
  }
}

}  // namespace

hipError_t launch_norm_part(const NormTable& t, int groups, double* part, hipStream_t s) {
  hipLaunchKernelGGL(k_norm_part, dim3(groups), dim3(kThreads), 0, s, t, part);
  return hipGetLastError();
}

hipError_t launch_norm_finish(const double* part, int nparts, float max_norm, float grad_scale,
                              float* record, hipStream_t s) {
  hipLaunchKernelGGL(k_norm_finish, dim3(1), dim3(kThreads), 0, s, part, nparts, max_norm,
                     grad_scale, record);
  return hipGetLastError();
}

hipError_t launch_clip(const NormTable& t, int groups, const float* record, hipStream_t s) {
  hipLaunchKernelGGL(k_clip, dim3(groups), dim3(kThreads), 0, s, t, record);
  return hipGetLastError();
}

hipError_t launch_adamw(const AdamTable& t, int groups, const AdamArgs& a, const float* record,
                        hipStream_t s) {
  hipLaunchKernelGGL(k_adamw, dim3(groups), dim3(kThreads), 0, s, t, a, record);
  return hipGetLastError();
}

}  // namespace fno
