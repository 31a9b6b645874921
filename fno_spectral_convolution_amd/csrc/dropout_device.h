// Dropout masks from a counter: nothing is stored, the backward makes the forward's mask again.
//
// Element i of a tensor has 16 bits of its own and is dropped where they are below the threshold
// T = round(65536 p); what is kept is multiplied by 65536 / (65536 - T), the inverse of the share
// that is kept in fact.  The bits come from Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel
// random numbers: as easy as 1, 2, 3", SC 2011): ten rounds on the counter (i / 8, draw), 64 bits
// each, under the key `seed` give four words, eight elements' bits.  16 bits and not 32: ten rounds
// cost about 110 vector cycles, and four elements to a block would hold half-precision fields to
// the vector units' rate instead of the memory's.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "train_ops.h"

namespace fno {

struct Words {
  uint32_t w[4];
};

// a ^ b ^ c in one instruction
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

__device__ __forceinline__ Words philox4x32(uint64_t block, uint64_t draw, uint32_t k0,
                                            uint32_t k1) {
  uint32_t a = (uint32_t)block, b = (uint32_t)(block >> 32), c = (uint32_t)draw,
           d = (uint32_t)(draw >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = (uint64_t)a * 0xD2511F53u, q = (uint64_t)c * 0xCD9E8D57u;
    a = xor3((uint32_t)(q >> 32), b, k0);
    b = (uint32_t)q;
    c = xor3((uint32_t)(p >> 32), d, k1);
    d = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{a, b, c, d}};
}

// A draw's mask: what a kernel makes of DropArgs once.
struct Dropper {
  uint32_t threshold, k0, k1;
  float scale;
  uint64_t draw;

  __device__ __forceinline__ explicit Dropper(const DropArgs& a)
      : threshold(a.threshold), k0((uint32_t)a.seed), k1((uint32_t)(a.seed >> 32)),
        scale(a.scale), draw(a.draw) {
    if (a.counter) draw += *a.counter;
  }
  __device__ __forceinline__ Words block(uint64_t k) const {
    // the rounds' keys are sums on the scalar unit, made where they are used: kept through a loop
    // they would take twenty registers and more
    uint32_t a = k0, b = k1;
    asm volatile("" : "+s"(a), "+s"(b));
    return philox4x32(k, draw, a, b);
  }
  // bit e: whether element e of block k is kept
  __device__ __forceinline__ uint32_t bits(uint64_t k) const {
    const Words w = block(k);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m |= ((uint16_t)w.w[j] >= (uint16_t)threshold ? 1u << 2 * j : 0u) |
           (w.w[j] >= threshold << 16 ? 2u << 2 * j : 0u);
    return m;
  }
  // the same for the N elements from i on (N <= 8), which may lie in two blocks
  template <int N>
  __device__ __forceinline__ uint32_t mask(uint64_t i) const {
    const int at = (int)(i & 7), blocks = N > 1 && at + N > 8 ? 2 : 1;
    uint32_t m = 0;
#pragma unroll 1
    for (int j = 0; j < blocks; ++j) m |= bits((i >> 3) + j) << 8 * j;
    m >>= at;
    // made before the elements are touched: the generator's registers are free again by then
    asm volatile("" : "+v"(m));
    return m;
  }
  // The masks of K vectors of N <= 4 elements, `step` elements apart from i on, four bits each.
  // paired: the lanes of a pair (2 j, 2 j + 1) are both there and share each vector's block, the even
  // one its first half; each then makes every other block for both.
  template <int N, int K>
  __device__ __forceinline__ uint32_t masks(uint64_t i, int64_t step, bool paired) const {
    uint32_t m = 0;
    if (N == 4 && K % 2 == 0 && paired) {
      const uint32_t odd = threadIdx.x & 1;
      if (odd) i += step;
#pragma unroll 1
      for (int k = 0; k < K; k += 2, i += 2 * step) {
        const uint32_t own = bits(i >> 3);
        const uint32_t other = __builtin_amdgcn_mov_dpp(own, 0xb1, 0xf, 0xf, true);  // of lane ^ 1
        const uint32_t first = odd ? other : own, second = odd ? own : other;
        m |= (first >> 4 * odd & 15) << 4 * k | (second >> 4 * odd & 15) << 4 * (k + 1);
      }
    } else {
#pragma unroll 1
      for (int k = 0; k < K; ++k, i += step) m |= (mask<N>(i) & 15) << 4 * k;
    }
    return m;
  }
  // What is dropped is 0, whatever it was.
  template <int N>
  __device__ __forceinline__ void apply(float (&v)[N], uint32_t m) const {
#pragma unroll
    for (int e = 0; e < N; ++e)
      v[e] = __int_as_float(__float_as_int(v[e] * scale) & __builtin_amdgcn_sbfe(m, e, 1));
  }
};

}  // namespace fno
