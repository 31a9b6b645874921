// Dropout by itself: y = residual + drop(x), and its backward, the same mask on grad_y.
//
// A thread takes eight elements at a time, what one block of the generator serves.  The mask goes by
// the packed index, so that entries that lie apart have the mask of their packed copy.
//
// Bound by memory: 134 million bfloat16 elements onto a residual 125 us, 6.5 TB/s; float32 261 (6.2)
// and without the residual 175 (6.1).  The generator and what makes bits of it are 21 vector
// instructions an element, about half the time of the bfloat16 pass, and hide behind the loads.  Few
// elements are the launch: 8 x 1024 bfloat16 2.5 us of kernel in a call of 7.5.
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

// One entry of data.  float32: a wave takes 512 elements as two vectors a lane, 256 elements apart,
// so that neighbours load neighbours; lanes 2 j and 2 j + 1 then make one block each for both.  (With a
// lane's eight elements in a row 134 million of them took 411 us onto a residual, 3.9 TB/s.)
template <typename T>
__global__ __launch_bounds__(256) void k_dropout(DropoutArgs a, const T* x, const T* residual, T* y) {
  constexpr int M = 16 / (int)sizeof(T), V = 8 / M;  // elements and number of a thread's vectors
  const Dropper drop(a.drop);
  const int64_t step = (int64_t)gridDim.x * 2048;
  const int lane = threadIdx.x % 64;
  for (int64_t base = ((int64_t)blockIdx.x * 4 + threadIdx.x / 64) * 512; base < a.per; base += step) {
    const int64_t i = base + lane * M;
    if (base + 512 <= a.per) {
      Raw<T, M> q[V], r[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        q[k] = load_raw<T, M, true>(x + i + k * 256);
        if (residual) r[k] = load_raw<T, M, true>(residual + i + k * 256);
      }
      uint32_t m = 0;
      if (a.drop.threshold) {
        if constexpr (V == 1) m = drop.bits((uint64_t)i >> 3);
        else m = drop.masks<M, V>((uint64_t)i, 256, true);
      }
#pragma unroll
      for (int k = 0; k < V; ++k) {
        float f[M];
        unpack<T, M>(q[k], f);
        if (a.drop.threshold) drop.apply<M>(f, m >> 4 * k);
        if (residual) {
#pragma unroll
          for (int e = 0; e < M; ++e) f[e] += element<T, M>(r[k], e);
        }
        store_pack<T, M>(y + i + k * 256, f, a.stream);
      }
    } else {
      for (int64_t j = base + lane; j < a.per; j += 64) {
        float v = to_float(x[j]);
        if (a.drop.threshold) v = drop.bits((uint64_t)j >> 3) >> (j & 7) & 1 ? v * drop.scale : 0.f;
        if (residual) v += to_float(residual[j]);
        y[j] = from_float<T>(v);
      }
    }
  }
}

// Entries that lie apart: a thread takes a block of eight elements at a time.  An entry's first and
// last block may be shared with its neighbours; each takes its own elements of them.  A lane's float32
// vectors lie next to each other here: eight entries of 16.8 million backward 209 us, packed 189 (bfloat16
// 87).
template <typename T>
__global__ __launch_bounds__(256) void k_dropout_entries(DropoutArgs a, int64_t blocks,
                                                         const T* x, const T* residual, T* y) {
  const Dropper drop(a.drop);
  const int64_t total = a.batch * blocks, step = (int64_t)gridDim.x * 256;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += step) {
    const int64_t b = total <= 0xffffffff ? (int64_t)((uint32_t)t / (uint32_t)blocks) : t / blocks;
    const int64_t first = b * a.per, block = (first >> 3) + t - b * blocks;
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
        store_pack<T, M>(o + e, q);
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
  // Outputs that fill half of the 256 MB cache behind the L2s go past it, where they are whole lines:
  // 205 MB of float32 onto a residual 97 us against 104, 268 MB of bf16 126 against 131, 102 MB the
  // same.  A work-group for every 2048 elements: 134 million bf16 126 us, 145 with 4096 work-groups.
  a.stream = a.per * (int64_t)sizeof(T) > ((int64_t)128 << 20) &&
             reinterpret_cast<uintptr_t>(y) % 128 == 0;
  const auto groups = [](int64_t n) { return dim3((unsigned)std::min<int64_t>(n, 1 << 20)); };
  if (a.batch == 1) {
    hipLaunchKernelGGL(k_dropout<T>, groups((a.per + 2047) / 2048), dim3(256), 0, s, a, x, residual,
                       y);
  } else {
    const int64_t blocks = (a.per + 7) / 8 + 1;
    hipLaunchKernelGGL(k_dropout_entries<T>, groups((a.batch * blocks + 255) / 256), dim3(256), 0, s,
                       a, blocks, x, residual, y);
  }
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
