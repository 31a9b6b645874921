// Device helpers of the training operators: element types, unaligned vectors, wave sums.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fno {

// ---- element types ---------------------------------------------------------------------------
// float32, bfloat16 and IEEE half data as float; half results are rounded to nearest-even.
template <typename T>
__device__ __forceinline__ float to_float(T v) {
  return (float)v;
}
template <typename T>
__device__ __forceinline__ T from_float(float v) {
  return (T)v;
}

// `N` packed elements at any multiple of the element size, as one load or store of N * sizeof(T)
// bytes: the global memory instructions take 16 bytes at any address (gfx950 runs in unaligned
// access mode), so odd row lengths and views need no code of their own.
template <typename T, int N>
struct RawVector {
  typedef T type __attribute__((ext_vector_type(N)));
  typedef type unaligned __attribute__((aligned(sizeof(T))));
};
template <typename T>
struct RawVector<T, 1> {
  typedef T type;
  typedef T unaligned;
};
template <typename T, int N>
using Raw = typename RawVector<T, N>::type;

template <typename T, int N>
__device__ __forceinline__ float element(const Raw<T, N>& q, int i) {
  if constexpr (N == 1) return to_float(q);
  else return to_float<T>(q[i]);
}
template <typename T, int N>
__device__ __forceinline__ void unpack(const Raw<T, N>& q, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = element<T, N>(q, i);
}
template <typename T, int N>
__device__ __forceinline__ Raw<T, N> pack(const float* f) {
  Raw<T, N> q;
  if constexpr (N == 1) {
    q = from_float<T>(f[0]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = from_float<T>(f[i]);
  }
  return q;
}

// Fields that are read or written once go past the caches (nontemporal) where `Stream`.
template <typename T, int N, bool Stream = false>
__device__ __forceinline__ Raw<T, N> load_raw(const T* p) {
  typedef typename RawVector<T, N>::unaligned V;
  if constexpr (Stream) return __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
  else return *reinterpret_cast<const V*>(p);
}
template <typename T, int N>
__device__ __forceinline__ void load_pack(const T* p, float (&f)[N]) {
  unpack<T, N>(load_raw<T, N>(p), f);
}
template <typename T, int N>
__device__ __forceinline__ void store_pack(T* p, const float (&f)[N], bool stream = false) {
  typedef typename RawVector<T, N>::unaligned V;
  const V q = pack<T, N>(f);
  if (stream) {
    // the empty statements keep the compiler from folding the two stores into a plain one
    asm volatile("");
    __builtin_nontemporal_store(q, reinterpret_cast<V*>(p));
    asm volatile("");
  } else {
    *reinterpret_cast<V*>(p) = q;
  }
}

// The same through pointers that the compiler cannot tell to be global (they come out of memory):
// as such they would be read with flat instructions, which also occupy the LDS.
template <typename T>
using Global = T __attribute__((address_space(1)))*;
template <typename T, int N, bool Stream = false>
__device__ __forceinline__ Raw<T, N> load_global(Global<const T> p) {
  typedef typename RawVector<T, N>::unaligned V;
  if constexpr (Stream) return __builtin_nontemporal_load((Global<const V>)p);
  else return *(Global<const V>)p;
}
template <typename T, int N>
__device__ __forceinline__ void store_global(Global<T> p, const float (&f)[N], bool stream) {
  constexpr int M = N * (int)sizeof(T) > 16 ? 16 / (int)sizeof(T) : N;
  typedef typename RawVector<T, M>::unaligned V;
#pragma unroll
  for (int k = 0; k < N; k += M) {
    const V q = pack<T, M>(f + k);
    if (stream) {
      asm volatile("");  // as in store_pack
      __builtin_nontemporal_store(q, (Global<V>)(p + k));
      asm volatile("");
    } else {
      *(Global<V>)(p + k) = q;
    }
  }
}

// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return __builtin_amdgcn_readfirstlane(v);
}
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)uniform((uint32_t)((uint64_t)v >> 32)) << 32 | uniform((uint32_t)v));
}

// ---- sums over lanes ---------------------------------------------------------------------------
template <int Ctrl>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), Ctrl, 0xf, 0xf, true));
}
// v of lane ^ 16 (ROW 16) or lane ^ 32 (ROW 32) added to v; both lanes add the same two numbers
template <int Row>
__device__ __forceinline__ float add_across(float v) {
  const unsigned u = __float_as_uint(v);
  const auto r = Row == 16 ? __builtin_amdgcn_permlane16_swap(u, u, false, false)
                           : __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sum over the aligned groups of N lanes (8, 16, 32 or 64), the same bits in every lane: six
// vector instructions for a wave and no trip through LDS.  Quad permutes reach lanes ^ 1 and ^ 2;
// with whole quads equal the half-row mirror stands for lane ^ 4, then the row mirror for ^ 8.
template <int N>
__device__ __forceinline__ float lane_sum(float v) {
  v += dpp<0xb1>(v);
  v += dpp<0x4e>(v);
  v += dpp<0x141>(v);
  if (N >= 16) v += dpp<0x140>(v);
  if (N >= 32) v = add_across<16>(v);
  if (N >= 64) v = add_across<32>(v);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}
// Sum over the lanes of a wave that share lane % N (N = 8, 16, 32; 64: v itself).
template <int N>
__device__ __forceinline__ float stride_sum(float v) {
  if (N <= 8) v += dpp<0x128>(v);  // rotation of the row by 8
  if (N <= 16) v = add_across<16>(v);
  if (N <= 32) v = add_across<32>(v);
  return v;
}

}  // namespace fno
