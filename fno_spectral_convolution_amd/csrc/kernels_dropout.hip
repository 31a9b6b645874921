// Dropout by itself: y = residual + drop(x), and its backward, the same mask on grad_y.
//
// Each thread takes one Philox block at a time, eight elements.  Entries may lie `stride` apart;
// the mask goes by the packed index, so that a view has the mask of its packed copy.
#include <algorithm>

#include "dropout_device.h"
#include "train_device.h"
#include "train_ops.h"

namespace fno {
namespace {

// Eight elements as one or two vectors.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  constexpr int M = 16 / (int)sizeof(T);
#pragma unroll
  for (int k = 0; k < 8; k += M) {
    float q[M];
    unpack<T, M>(load_raw<T, M, true>(p + k), q);
#pragma unroll
    for (int e = 0; e < M; ++e) f[k + e] = q[e];
  }
}

// SOLE: one entry of data.  Otherwise an entry's first and last block may be shared with its
// neighbours; each takes its own elements of them.
template <typename T, bool SOLE>
__global__ __launch_bounds__(256) void k_dropout(DropoutArgs a, const T* x, const T* residual,
                                                 T* y) {
  const Dropper drop(a.drop);
  const int64_t per_blocks = SOLE ? (a.per + 7) / 8 : (a.per + 7) / 8 + 1;
  const int64_t total = SOLE ? per_blocks : a.batch * per_blocks;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += step) {
    int64_t b = 0, k = t;
    if (!SOLE) {
      b = total <= 0xffffffff ? (int64_t)((uint32_t)t / (uint32_t)per_blocks) : t / per_blocks;
      k = t - b * per_blocks;
    }
    const int64_t first = b * a.per, block = (first >> 3) + k;
    const int64_t j = 8 * block - first;  // of the block's first element in its entry
    const T* p = x + b * a.x_stride + j;
    const T* r = residual ? residual + b * a.r_stride + j : nullptr;
    T* o = y + b * a.y_stride + j;
    if (j >= 0 && j + 8 <= a.per) {
      float f[8], add[8];
      load8(p, f);
      if (r) load8(r, add);
      if (a.drop.threshold) drop.apply<8>(f, drop.bits(block));
      if (r) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += add[e];
      }
      constexpr int M = 16 / (int)sizeof(T);
#pragma unroll
      for (int e = 0; e < 8; e += M) {
        float q[M];
#pragma unroll
        for (int i = 0; i < M; ++i) q[i] = f[e + i];
        store_pack<T, M>(o + e, q, a.stream);
      }
    } else if (j + 8 > 0 && j < a.per) {
      const uint32_t m = a.drop.threshold ? drop.bits(block) : 0xff;
      for (int e = 0; e < 8; ++e)
        if (j + e >= 0 && j + e < a.per) {
          float v = m >> e & 1 ? to_float(p[e]) * drop.scale : 0.f;
          if (r) v += to_float(r[e]);
          o[e] = from_float<T>(v);
        }
    }
  }
}

template <typename T>
hipError_t go(DropoutArgs a, const T* x, const T* residual, T* y, hipStream_t s) {
  if (a.x_stride == a.per && a.y_stride == a.per && (!residual || a.r_stride == a.per)) {
    a.per *= a.batch;
    a.batch = 1;
  }
  a.stream = a.batch * a.per * (int64_t)sizeof(T) > ((int64_t)256 << 20) && a.batch == 1 &&
             reinterpret_cast<uintptr_t>(y) % 128 == 0;
  const int64_t tasks = a.batch == 1 ? (a.per + 7) / 8 : a.batch * ((a.per + 7) / 8 + 1);
  const int64_t groups = std::min<int64_t>((tasks + 255) / 256, 4096);
  if (a.batch == 1)
    hipLaunchKernelGGL((k_dropout<T, true>), dim3(groups), dim3(256), 0, s, a, x, residual, y);
  else
    hipLaunchKernelGGL((k_dropout<T, false>), dim3(groups), dim3(256), 0, s, a, x, residual, y);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, int dtype, const void* x, const void* residual,
                          void* y, hipStream_t s) {
  const auto run = [&](auto t) {
    typedef decltype(t) T;
    return go<T>(a, static_cast<const T*>(x), static_cast<const T*>(residual), static_cast<T*>(y),
                 s);
  };
  if (dtype == FNO_DTYPE_F32) return run(0.f);
  return dtype == FNO_DTYPE_BF16 ? run((__bf16)0.f) : run((_Float16)0.f);
}

}  // namespace fno
