// Group norm with an activation and dropout, forward and backward, over fields [batch][channels][npts]
// and channels-last data [batch][npts][channels].  With m = channels of a group * npts:
//
//   forward   mu = sum x / m,  r = 1 / sqrt(sum (x - mu)^2 / m + eps)   over a group of an entry
//             u = gamma r (x - mu) + beta,  y = drop(act(u))
//   backward  g = act'(u) drop(grad_y),  h = r (x - mu),  grad_gamma = sum g h,  grad_beta = sum g,
//             grad_x = r (gamma g - sum(gamma g) / m - h sum(gamma g h) / m)
//
// The activation, its slope and the mask are computed again from x and the element's index where
// they are needed: nothing but x and the statistics goes from the forward to the backward.  The
// variance comes from deviations about a mean, never from E[x^2] - E[x]^2: each thread keeps count,
// mean and squared deviations of what it has seen, and two of these join as
// M2 = M2_a + M2_b + n_a n_b / (n_a + n_b) (mean_a - mean_b)^2 (Chan, Golub, LeVeque 1979).  Sums are
// float32 in a fixed order, without atomics, of chains that stay short whatever the sizes: a chain of n
// like terms may be off by n / 3 units of 2^-24.  Each pass rounds once, where it stores.
#pragma once

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "dropout_device.h"
#include "pointwise.h"
#include "train_device.h"
#include "train_ops.h"

namespace fno {

constexpr int kBlock = 256, kWaves = kBlock / 64;

// ---- activations ---------------------------------------------------------------------------------
__device__ __forceinline__ float sigmoid(float u) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u * -1.4426950408889634f));
}
// one branch for all of a vector: every lane takes the same
template <int N>
__device__ __forceinline__ void activate(float (&u)[N], int act) {
  if (act == FNO_ACT_GELU) {
#pragma unroll
    for (int e = 0; e < N; ++e) u[e] = gelu_as(u[e]);
  } else if (act == FNO_ACT_SILU) {
#pragma unroll
    for (int e = 0; e < N; ++e) u[e] *= sigmoid(u[e]);
  }
}
// g *= act'(u)
template <int N>
__device__ __forceinline__ void slope(float (&g)[N], const float (&u)[N], int act) {
  if (act == FNO_ACT_GELU) {
#pragma unroll
    for (int e = 0; e < N; ++e) g[e] *= gelu_grad_as(u[e]);
  } else if (act == FNO_ACT_SILU) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float s = sigmoid(u[e]);
      g[e] *= s * fmaf(u[e], 1.0f - s, 1.0f);
    }
  }
}

// ---- sums and moments ----------------------------------------------------------------------------
// Both sums over the work-group, the same bits in every thread.  `s` is not written again before the
// next barrier but one.
template <int WAVES>
__device__ __forceinline__ float2 block_sum(float a, float b, float2* s) {
  a = lane_sum<64>(a);
  b = lane_sum<64>(b);
  if (WAVES == 1) return make_float2(a, b);
  if (threadIdx.x % 64 == 0) s[threadIdx.x / 64] = make_float2(a, b);
  __syncthreads();
  float2 t = s[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) {
    t.x += s[w].x;
    t.y += s[w].y;
  }
  return t;
}

// Sum over aligned groups of `lanes` lanes, a power of two that all lanes agree on, in each of them
// (as lane_sum).
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  if (lanes >= 2) v += dpp<0xb1>(v);
  if (lanes >= 4) v += dpp<0x4e>(v);
  if (lanes >= 8) v += dpp<0x141>(v);
  if (lanes >= 16) v += dpp<0x140>(v);
  if (lanes >= 32) v = add_across<16>(v);
  if (lanes >= 64) v = add_across<32>(v);
  return v;
}

// Count, mean, and the sum of squared deviations over the m entries of the whole group: a share of
// its variance, which stays in range where the sum by itself would pass float32's.
struct Moments {
  float n, mean, var;
};
// Squared deviations and their sum may pass float32's range where the variance does not.  They are taken
// of deviations times `down`, a power of two with down^2 <= 1 / m, so that their sum stays below the
// variance; times `up`, below 4, it is the sum divided by m.  Neither rounds.  Made by the host: a
// division and the steps after it were 2% of a call of many small groups.
struct Scale {
  float inv_m, down, up, back;  // 1 / m; back = 1 / down
  Scale() = default;
  explicit Scale(const GroupArgs& a)
      : inv_m(1.0f / ((float)(a.channels / a.groups) * (float)a.npts)) {
    int exponent;
    std::frexp(inv_m, &exponent);  // 1 / m >= 2^(exponent - 1)
    const int half = (2 - exponent) / 2;
    down = std::ldexp(1.f, -half);
    back = std::ldexp(1.f, half);
    up = std::ldexp(inv_m, 2 * half);
  }
  __device__ __forceinline__ float deviation(float x, float mean) const {
    return fmaf(x, down, -mean * down);
  }
};
__device__ __forceinline__ void join(Moments& a, float n, float mean, float var, float inv_m) {
  const float all = a.n + n, share = n > 0.f ? n * __builtin_amdgcn_rcpf(all) : 0.f;
  const float d = mean - a.mean;
  a.mean += d * share;
  a.var += var + (d * (share * (a.n * inv_m))) * d;
  a.n = all;
}
// All threads' moments, the same bits in every one.
template <int WAVES>
__device__ __forceinline__ Moments block_moments(const Moments& m, float inv_m,
                                                 float2 (&s)[2][WAVES]) {
  if (WAVES > 1) __syncthreads();
  const float2 t = block_sum<WAVES>(m.n, m.n * m.mean, s[0]);
  Moments r;
  r.n = t.x;
  r.mean = t.y / t.x;
  const float d = m.mean - r.mean;
  r.var = block_sum<WAVES>(m.n > 0.f ? m.var + (d * (m.n * inv_m)) * d : 0.f, 0.f, s[1]).x;
  return r;
}

// Calls f(masked) with a constant: whether any lane of the wave has elements that are not its own
// (most waves have none, and are spared a select an element).
template <typename F>
__device__ __forceinline__ void by_mask(bool masked, F&& f) {
  if (masked) f(std::true_type());
  else f(std::false_type());
}

// Division by a number that the host knows: three instructions where a division takes thirty in a
// row, which is what small calls are made of.  q = (n + high word of n mul) >> shift with
// shift = ceil(log2 d), mul = 2^32 (2^shift - d) / d + 1 (Granlund, Montgomery 1994), n below 2^31.
struct Divider {
  uint32_t d, mul, shift;
  Divider() = default;
  explicit Divider(int64_t by) : d((uint32_t)std::max<int64_t>(1, by)), shift(0) {
    while (((uint64_t)1 << shift) < d) ++shift;
    mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t of(uint32_t n) const {
    return (__umulhi(n, mul) + n) >> shift;
  }
  __device__ __forceinline__ int64_t of(int64_t n) const {
    return n >> 31 ? n / d : (int64_t)of((uint32_t)n);
  }
};

template <typename T, int VEC>
__device__ __forceinline__ void store_own(T* o, const float (&f)[VEC], int lo,
                                          bool stream = false) {
  if (lo == 0) {
    store_pack<T, VEC>(o, f, stream);
  } else {
#pragma unroll
    for (int e = 1; e < VEC; ++e)
      if (e >= lo) o[e] = from_float<T>(f[e]);
  }
}

// What both backward passes need of an element: h = (x - mu) r, g = act'(u) drop(grad_y), by its mask.
template <typename T, int VEC>
__device__ __forceinline__ void backward_terms(const GroupArgs& a, const Dropper& drop,
                                               const Raw<T, VEC>& rx, const Raw<T, VEC>& rg,
                                               const float (&mu)[VEC], const float (&rs)[VEC],
                                               const float (&ga)[VEC], const float (&be)[VEC],
                                               uint32_t mask, float (&h)[VEC],
                                               float (&g)[VEC]) {
  unpack<T, VEC>(rx, h);
  unpack<T, VEC>(rg, g);
#pragma unroll
  for (int e = 0; e < VEC; ++e) h[e] = (h[e] - mu[e]) * rs[e];
  if (a.drop.threshold) drop.apply<VEC>(g, mask);
  if (a.act != FNO_ACT_NONE) {
    float u[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) u[e] = fmaf(h[e], ga[e], be[e]);
    slope(g, u, a.act);
  }
}
template <int N>
__device__ __forceinline__ void fill(float (&f)[N], float v) {
#pragma unroll
  for (int e = 0; e < N; ++e) f[e] = v;
}

// ---- between the backward's passes -----------------------------------------------------------------
// From the first pass's partial rows [2][channels]: the weights' gradients, and for each group the
// means of gamma g and gamma g h.  In a launch of their own, the first work-groups for the means; where
// there is little to add up, in the second pass's launch, whose work-groups make the means that they
// need and are followed by those for the weights.
constexpr int kSumCols = 16;
struct Rows {
  int64_t n;
  const float* at;
};
struct Between {
  Rows sums;              // for the weights
  int64_t groups;         // work-groups before those of the weights
  const float* part;      // the first pass's rows
  float2* means;
  float *ggamma, *gbeta;  // nullable
  Divider by_groups;
  bool own;               // no launch of their own
};
// The weights' gradients, kSumCols columns at a time, by the work-groups from z.groups on.
__device__ __forceinline__ void weight_sums(const GroupArgs& a, const Between& z) {
  constexpr int kSlices = kBlock / kSumCols;
  __shared__ float s_col[kSlices][kSumCols];
  const int col = threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols;
  const int64_t width = 2 * (int64_t)a.channels;
  for (int64_t base = (blockIdx.x - z.groups) * kSumCols; base < width;
       base += (gridDim.x - z.groups) * kSumCols) {
    const int64_t i = base + col;
    float s = 0.f;  // (chains of up to 128 rows)
    if (i < width)
#pragma unroll 8
      for (int64_t k = slice; k < z.sums.n; k += kSlices) s += z.sums.at[k * width + i];
    s_col[slice][col] = s;
    __syncthreads();
    if (slice == 0 && i < width) {
      for (int w = 1; w < kSlices; ++w) s += s_col[w][col];
      float* out = i < a.channels ? z.ggamma : z.gbeta;
      if (out) out[i < a.channels ? i : i - a.channels] = s;
    }
    __syncthreads();
  }
}
// A launch of their own; sums(b, g): a thread's shares of group g's sums.
template <typename F>
__device__ __forceinline__ void between(const GroupArgs& a, const Between& z, F&& sums) {
  __shared__ float2 s_red[kWaves];
  if (blockIdx.x >= z.groups) return weight_sums(a, z);
  const int64_t sides = a.batch * a.groups;
  const float inv = 1.0f / ((float)(a.channels / a.groups) * (float)a.npts);
  for (int64_t i = blockIdx.x; i < sides; i += z.groups) {
    const int64_t b = z.by_groups.of(i);
    const float2 own = sums(b, (int)(i - b * a.groups));
    __syncthreads();
    const float2 v = block_sum<kWaves>(own.x, own.y, s_red);
    if (threadIdx.x == 0) z.means[i] = make_float2(v.x * inv, v.y * inv);
  }
}

// ---- launches ------------------------------------------------------------------------------------
constexpr int64_t kMaxGrid = 1 << 20;  // further work goes to the same work-groups
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline dim3 grid_of(int64_t total) { return dim3((unsigned)std::min<int64_t>(total, kMaxGrid)); }
inline size_t up(int64_t bytes) { return ((size_t)bytes + 255) / 256 * 256; }

template <int N>
struct Int {
  static constexpr int value = N;
};
// Calls f(elements of a vector): single ones where runs of neighbours are shorter than a vector.
template <int VEC, typename F>
auto by_vector(int64_t run, F&& f) {
  if (run < VEC) return f(Int<1>());
  return f(Int<VEC>());
}
template <typename F>
auto by_type(int dtype, F&& f) {
  if (dtype == FNO_DTYPE_F32) return f(0.f);
  return dtype == FNO_DTYPE_BF16 ? f((__bf16)0.f) : f((_Float16)0.f);
}
// Whether an output goes past the caches (nontemporal stores): where it fills half of the 256 MB cache
// behind the L2s (4 x 64 x 512^2 float32, 268 MB, with GELU forward 136 us against 140 and backward 216
// against 224; 8 x 64 x 512^2 bf16, as large, 152 against 154 and 249 against 259, with dropout as well
// 165 against 167 and the same 305; below, no difference).
template <typename T>
bool stream_out(const GroupArgs& a) {
  return a.batch * a.channels * a.npts > ((int64_t)128 << 20) / (int64_t)sizeof(T);
}

// Whether a backward's second pass should do for itself what is between the passes: small data, where a
// launch counts (4 x 20 x 64^2 float32 18 us against 22; 4 x 96^2 x 320 half, three times as large as
// the limit, loses 2 of 47).
inline bool small(const GroupArgs& a) { return a.batch * a.channels * a.npts <= 1 << 22; }

// Partial rows [2][channels] beyond `most` are folded into sums of `size` neighbours first: their number
// goes with the batch, and the weights' sums over them have few work-groups, which add up one row after
// the other in float32 (gradients of one sign came out up to 3000 units of 2^-24 off, and 300000 x 8 x 2
// float32 backward took 1150 us, now 930; 65536 x 4 x 64 bf16 channels last 1097, now 934).  Up to
// 2048 the chains are of 128 and the launch would not pay (2000 x 8 x 64 float32 channels last 28 us;
// 4000 rows 51, 54 without).  About the root of their number to a sum, more where that would leave more
// than the limit; in float64.
constexpr int64_t kMostRows = 2048;
struct Fold {
  int64_t size, rows;  // rows of a sum, and sums; 1: none
  explicit Fold(int64_t n, int64_t most = kMostRows) : size(1), rows(n) {
    if (n <= most) return;
    while (size * size < n || size * most < n) size *= 2;
    rows = ceil_div(n, size);
  }
  size_t bytes(const GroupArgs& a) const {
    return size == 1 ? 0 : up((int64_t)sizeof(float) * 2 * rows * a.channels);
  }
};
// the rows to add up in place of n at `part`; `to`: f.bytes() of workspace, f of n rows
Rows fold_rows(const GroupArgs& a, const Fold& f, int64_t n, const float* part, float* to,
               hipStream_t s);

// A backward's workspace: the partial rows, what they are folded into, the segments' sums (channels
// last), the means.
struct Space {
  int64_t rows;
  size_t part, fold, seg, means;
  Space(const GroupArgs& a, int64_t rows, int64_t segments)
      : rows(rows), part(up((int64_t)sizeof(float) * 2 * rows * a.channels)),
        fold(Fold(rows).bytes(a)), seg(up((int64_t)sizeof(float2) * segments)),
        means(up((int64_t)sizeof(float2) * a.batch * a.groups)) {}
  size_t bytes() const { return part + fold + seg + means; }
  float2* segments_at(void* ws) const {
    return reinterpret_cast<float2*>(static_cast<char*>(ws) + part + fold);
  }
  float2* means_at(void* ws) const {
    return reinterpret_cast<float2*>(static_cast<char*>(ws) + part + fold + seg);
  }
  // what is between the passes; items: of the second pass, in whose launch it is done where `own`
  Between between(const GroupArgs& a, void* ws, bool means, float* ggamma, float* gbeta, bool own,
                  int64_t items) const {
    own = own && means;
    const int64_t groups = own ? items : means ? a.batch * a.groups : 0;
    const float* part_at = static_cast<const float*>(ws);
    return {{rows, part_at}, std::min<int64_t>(groups, kMaxGrid), part_at, means_at(ws),
            ggamma, gbeta, Divider(a.groups), own};
  }
  // after the first pass: the rows for the weights folded
  void fold_in(const GroupArgs& a, Between& z, void* ws, hipStream_t s) const {
    if (fold > 0 && (z.ggamma || z.gbeta))
      z.sums = fold_rows(a, Fold(rows), rows, z.part,
                         reinterpret_cast<float*>(static_cast<char*>(ws) + part), s);
  }
  // the grid with the weights' work-groups
  static dim3 grid(const GroupArgs& a, const Between& z) {
    const int64_t cols = z.ggamma || z.gbeta ? ceil_div(2 * (int64_t)a.channels, kSumCols) : 0;
    return dim3((unsigned)(z.groups + std::min<int64_t>(cols, kMaxGrid)));
  }
};

// ---- channels last (kernels_groupnorm_last.hip) --------------------------------------------------
size_t group_norm_last_fwd_bytes(const GroupArgs& a);
size_t group_norm_last_bwd_bytes(const GroupArgs& a);
hipError_t launch_group_norm_last_fwd(const GroupArgs& a, int dtype, const void* x,
                                      const float* gamma, const float* beta, void* y, float* stats,
                                      void* ws, hipStream_t s);
hipError_t launch_group_norm_last_bwd(const GroupArgs& a, int dtype, const void* x,
                                      const float* gamma, const float* beta, const float* stats,
                                      const void* gy, void* gx, float* ggamma, float* gbeta,
                                      void* ws, hipStream_t s);

}  // namespace fno
