// Layer norm over the channels of a field [batch][channels][npts], forward and backward.
#include "train_ops.h"

namespace fno {
namespace {

constexpr int kColParts = 64;  // partial sums of each channel's weight gradients

// One thread per point (b, p); three sweeps over its channels, which are npts elements apart.
template <typename T>
__global__ void k_ln_fwd_points(NormArgs a, const T* x, const float* gamma, const float* beta,
                                T* y, float* stats) {
  const int64_t rows = a.batch * a.npts;
  for (int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < rows;
       r += (int64_t)gridDim.x * blockDim.x) {
    const int64_t b = r / a.npts, p = r - b * a.npts;
    const T* xr = x + b * a.x_stride + p;
    T* yr = y + b * a.y_stride + p;
    float sum = 0.f, sq = 0.f;
    for (int c = 0; c < a.channels; ++c) sum += to_float(xr[c * a.npts]);
    const float mean = sum / (float)a.channels;
    for (int c = 0; c < a.channels; ++c) {
      const float d = to_float(xr[c * a.npts]) - mean;
      sq += d * d;
    }
    const float rstd = 1.0f / sqrtf(sq / (float)a.channels + a.eps);
    for (int c = 0; c < a.channels; ++c) {
      const float h = (to_float(xr[c * a.npts]) - mean) * rstd;
      yr[c * a.npts] = from_float<T>((gamma ? gamma[c] : 1.f) * h + (beta ? beta[c] : 0.f));
    }
    if (stats) {
      stats[r] = mean;
      stats[rows + r] = rstd;
    }
  }
}

template <typename T>
__global__ void k_ln_bwd_points(NormArgs a, const T* x, const float* gamma, const float* stats,
                                const T* gy, T* gx) {
  const int64_t rows = a.batch * a.npts;
  for (int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < rows;
       r += (int64_t)gridDim.x * blockDim.x) {
    const int64_t b = r / a.npts, p = r - b * a.npts;
    const T* xr = x + b * a.x_stride + p;
    const T* gr = gy + b * a.y_stride + p;
    T* o = gx + b * a.gx_stride + p;
    const float mean = stats[r], rstd = stats[rows + r];
    float s1 = 0.f, s2 = 0.f;
    for (int c = 0; c < a.channels; ++c) {
      const float g = to_float(gr[c * a.npts]) * (gamma ? gamma[c] : 1.f);
      s1 += g;
      s2 += g * ((to_float(xr[c * a.npts]) - mean) * rstd);
    }
    s1 /= (float)a.channels;
    s2 /= (float)a.channels;
    for (int c = 0; c < a.channels; ++c) {
      const float g = to_float(gr[c * a.npts]) * (gamma ? gamma[c] : 1.f);
      const float h = (to_float(xr[c * a.npts]) - mean) * rstd;
      o[c * a.npts] = from_float<T>(rstd * (g - s1 - h * s2));
    }
  }
}

// Work-group (part, c): the sums of grad_y h and grad_y over the part's points of channel c.
template <typename T>
__global__ void k_ln_cols(NormArgs a, const T* x, const float* stats, const T* gy, float* part) {
  __shared__ float s_red[2][256];
  const int64_t rows = a.batch * a.npts;
  const int tid = threadIdx.x;
  for (int c = blockIdx.y; c < a.channels; c += gridDim.y) {
    float sg = 0.f, sb = 0.f;
    for (int64_t r = (int64_t)blockIdx.x * 256 + tid; r < rows; r += (int64_t)gridDim.x * 256) {
      const int64_t b = r / a.npts, at = (r - b * a.npts) + c * a.npts;
      const float g = to_float(gy[b * a.y_stride + at]);
      const float h = (to_float(x[b * a.x_stride + at]) - stats[r]) * stats[rows + r];
      sg += g * h;
      sb += g;
    }
    __syncthreads();
    s_red[0][tid] = sg;
    s_red[1][tid] = sb;
    __syncthreads();
    for (int w = 128; w > 0; w >>= 1) {
      if (tid < w) {
        s_red[0][tid] += s_red[0][tid + w];
        s_red[1][tid] += s_red[1][tid + w];
      }
      __syncthreads();
    }
    if (tid < 2) part[((int64_t)blockIdx.x * 2 + tid) * a.channels + c] = s_red[tid][0];
  }
}

__global__ void k_ln_finish(int channels, int nparts, const float* part, float* ggamma,
                            float* gbeta) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= 2 * channels) return;
  float* out = i < channels ? ggamma : gbeta;
  if (!out) return;
  float s = 0.f;
  for (int k = 0; k < nparts; ++k) s += part[(int64_t)k * 2 * channels + i];
  out[i < channels ? i : i - channels] = s;
}

int point_groups(const NormArgs& a) {
  const int64_t rows = a.batch * a.npts, g = (rows + 255) / 256;
  return (int)(g < 4096 ? g : 4096);
}

template <typename T>
hipError_t fwd_t(const NormArgs& a, const void* x, const float* gamma, const float* beta, void* y,
                 float* stats, hipStream_t s) {
  hipLaunchKernelGGL(k_ln_fwd_points<T>, dim3(point_groups(a)), dim3(256), 0, s, a,
                     static_cast<const T*>(x), gamma, beta, static_cast<T*>(y), stats);
  return hipGetLastError();
}

template <typename T>
hipError_t bwd_t(const NormArgs& a, const void* x, const float* gamma, const float* stats,
                 const void* gy, void* gx, float* part, hipStream_t s) {
  // the column sums first: grad_x may overwrite x or grad_y
  if (part) {
    const int cols = a.channels < 32768 ? a.channels : 32768;
    hipLaunchKernelGGL(k_ln_cols<T>, dim3(kColParts, cols), dim3(256), 0, s, a,
                       static_cast<const T*>(x), stats, static_cast<const T*>(gy), part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (gx)
    hipLaunchKernelGGL(k_ln_bwd_points<T>, dim3(point_groups(a)), dim3(256), 0, s, a,
                       static_cast<const T*>(x), gamma, stats, static_cast<const T*>(gy),
                       static_cast<T*>(gx));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm_fwd(const NormArgs& a, int dtype, const void* x, const float* gamma,
                                 const float* beta, void* y, float* stats, hipStream_t s) {
  if (dtype == FNO_DTYPE_F32) return fwd_t<float>(a, x, gamma, beta, y, stats, s);
  if (dtype == FNO_DTYPE_BF16) return fwd_t<__bf16>(a, x, gamma, beta, y, stats, s);
  return fwd_t<_Float16>(a, x, gamma, beta, y, stats, s);
}

int layer_norm_parts(const NormArgs& a, int) {
  return a.batch * a.npts > 0 ? kColParts : 0;
}

hipError_t launch_layer_norm_bwd(const NormArgs& a, int dtype, const void* x, const float* gamma,
                                 const float* stats, const void* gy, void* gx, float* part,
                                 hipStream_t s) {
  if (dtype == FNO_DTYPE_F32) return bwd_t<float>(a, x, gamma, stats, gy, gx, part, s);
  if (dtype == FNO_DTYPE_BF16) return bwd_t<__bf16>(a, x, gamma, stats, gy, gx, part, s);
  return bwd_t<_Float16>(a, x, gamma, stats, gy, gx, part, s);
}

hipError_t launch_layer_norm_finish(const NormArgs& a, int nparts, const float* part,
                                    float* ggamma, float* gbeta, hipStream_t s) {
  hipLaunchKernelGGL(k_ln_finish, dim3((2 * (int64_t)a.channels + 255) / 256), dim3(256), 0, s,
                     a.channels, nparts, part, ggamma, gbeta);
  return hipGetLastError();
}

}  // namespace fno
