// Layer norm over the channels of a field [batch][channels][npts], forward and backward.
//
//   forward   mu = sum_c x / C,  r = 1 / sqrt(sum_c (x - mu)^2 / C + eps),  h = (x - mu) r,
//             y = gamma h + beta
//   backward  g = gamma grad_y,  grad_x = r (g - sum_c g / C - h sum_c(g h) / C),
//             grad_gamma = sum grad_y h,  grad_beta = sum grad_y  (over batch and points)
//
// Each pass reads its fields once and writes once; memory bounds it (8 and 14 operations an element
// against 8 and 12 bytes in float32).  A row or point is therefore held in registers from its load
// to its store, and only the sums over channels leave a lane.  All sums and statistics are float32 or
// wider.
// The variance comes from deviations about a mean, never from E[x^2] - E[x]^2; where several waves
// share a row or point, each takes its own mean and the squared deviations about it, and they join
// as M2 = sum_w (M2_w + n_w (mean_w - mean)^2), which needs one exchange where two sweeps need two.
// The reciprocal square root is the hardware's (1 ulp).  The weight gradients are sums in a fixed
// order: per work-group over its rows or points, then over the work-groups' partial rows.
//
// Measured on an MI355X whose large copies run at 4.9 TB/s, three inputs in turn.  Outputs below 256 MB
// (the rows' here) are taken by the cache behind the L2s; the float32 fields' go past it.
//   rows    8192 x 4096 bf16       forward  24 us (5.6 TB/s)   backward  40 us (5.1)
//           8192 x 4096 float32    forward  42 us (6.4)        backward  69 us (5.8)
//           16384 x 1024 bf16      forward  14 us (4.8)        backward  23 us (4.4)
//   fields  8 x 64 x 512^2 float32 forward 186 us (5.9)        backward 288 us (5.7)
//           2 x 20 x 128^3 float32 forward 135 us (5.2)        backward 200 us (5.2)
//           8 x 64 x 512^2 bf16    forward 124 us (4.4)        backward 166 us (5.0)
#include <algorithm>
#include <type_traits>

#include "train_device.h"
#include "train_ops.h"

namespace fno {
namespace {

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);  // elements of a 16-byte load

// ---- rows (npts = 1) ---------------------------------------------------------------------------
// TPR threads hold a row, NV vectors of VEC elements each: eight lanes for the shortest rows, the
// work-group for the longest.  Vector j of the row starts at element j VEC; the last one is moved
// back to end with the row, and the elements that it then shares with its neighbour (i < lo) count
// once in sums and are stored twice with the same value.  So any length takes whole 16-byte loads.
template <int VEC>
__device__ __forceinline__ void place(int j, int d, int& start, int& lo) {
  const int e = j * VEC;
  start = e < d - VEC ? e : d - VEC;
  lo = e < d ? e - start : VEC;
}

// A row's slice of gamma or beta; `none` where there is none.  In 16-byte loads: loaded element by
// element, 32 bytes apart from lane to lane, the weights cost more than the row itself (8192 x 4096
// bf16 forward 39 us instead of 24).
template <int VEC>
__device__ __forceinline__ void load_weight(const float* w, int start, float none,
                                            float (&f)[VEC]) {
  if (w) {
    constexpr int M = VEC < 4 ? VEC : 4;
#pragma unroll
    for (int i = 0; i < VEC; i += M) {
      float q[M];
      load_pack<float, M>(w + start + i, q);
#pragma unroll
      for (int e = 0; e < M; ++e) f[i + e] = q[e];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = none;
  }
}

// elements of the row that wave `w` of the row's waves holds (TPR > 64)
template <int VEC, int TPR, int NV>
__device__ __forceinline__ float wave_count(int w, int d) {
  int n = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int at = (k * TPR + w * 64) * VEC, left = d - at;
    n += left < 0 ? 0 : (left < 64 * VEC ? left : 64 * VEC);
  }
  return (float)n;
}

// Sum over the row's WAVES waves of a value that lane l has for wave l % WAVES, in every lane.
template <int WAVES>
__device__ __forceinline__ float wave_sum(float v) {
  constexpr int kLanes = WAVES < 8 ? 8 : WAVES;
  return lane_sum<kLanes>(v) * ((float)WAVES / kLanes);
}

// Calls f(masked) with a constant: whether any lane of the wave has elements that are not its own
// (asked once; most waves of most rows have none, and are spared a select per element and sum).
template <typename F>
__device__ __forceinline__ void by_mask(bool masked, F&& f) {
  if (masked) f(std::true_type());
  else f(std::false_type());
}

// A work-group goes over many rows: the weights stay in its registers, and the next row's loads go
// ahead of this row's sums (two rows ahead measured the same).  Sums go over a wave's lanes without
// LDS; a row of several waves takes one barrier, after which every lane reads one wave's part.
// Eight elements to a thread keep eight waves on a SIMD; sixteen measured 0 to 4% slower.
template <typename T, int VEC, int TPR, int NV, int BLOCK>
__global__ __launch_bounds__(BLOCK) void k_ln_fwd_rows(NormArgs a, const T* x, const float* gamma,
                                                       const float* beta, T* y, float* stats) {
  constexpr int kGroups = BLOCK / TPR, kWaves = TPR > 64 ? TPR / 64 : 1;
  constexpr int kLanes = TPR < 64 ? TPR : 64;
  __shared__ float s_stat[2][kGroups][kWaves][2];
  const int tid = threadIdx.x, t = tid % TPR, group = tid / TPR, wave = t / 64;
  const int d = a.channels;
  const float inv_d = 1.0f / (float)d;
  int start[NV], lo[NV];
  float ga[NV][VEC], be[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    place<VEC>(k * TPR + t, d, start[k], lo[k]);
    load_weight<VEC>(gamma, start[k], 1.f, ga[k]);
    load_weight<VEC>(beta, start[k], 0.f, be[k]);
  }
  bool partial = false;
#pragma unroll
  for (int k = 0; k < NV; ++k) partial |= lo[k] != 0;
  partial = __any(partial);
  const int other = t % kWaves;  // the wave whose part of a joint sum this lane reads
  const float n = wave_count<VEC, TPR, NV>(wave, d), n_other = wave_count<VEC, TPR, NV>(other, d);
  const float inv_n = TPR > 64 ? 1.0f / fmaxf(n, 1.f) : inv_d, share_other = n_other * inv_d;
  const int64_t rows = a.batch, step = (int64_t)gridDim.x * kGroups;
  int64_t base = (int64_t)blockIdx.x * kGroups;
  Raw<T, VEC> next[NV];
  const auto fetch = [&](int64_t at) {
    const int64_t row = at + group < rows ? at + group : rows - 1;
    const T* p = x + row * a.x_stride;
#pragma unroll
    for (int k = 0; k < NV; ++k) next[k] = load_raw<T, VEC, true>(p + start[k]);
  };
  if (base < rows) fetch(base);
  int flip = 0;
  for (; base < rows; base += step, flip ^= 1) {
    float f[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV; ++k) unpack<T, VEC>(next[k], f[k]);
    if (base + step < rows) fetch(base + step);
    float mean, sq;
    by_mask(partial, [&](auto masked) {
      float sum = 0.f, sum2 = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum += !masked.value || i >= lo[k] ? f[k][i] : 0.f;
      mean = lane_sum<kLanes>(sum) * inv_n;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float c = f[k][i] - mean;
          sum2 += !masked.value || i >= lo[k] ? c * c : 0.f;
        }
      sq = lane_sum<kLanes>(sum2) * inv_d;
    });
    if (TPR > 64) {
      // the waves' means and squared deviations join: var = sum (M2_w + n_w (mean_w - mean)^2) / d,
      // divided before the sum, which passes float32's range where the variance is far from it.  In
      // this order of products a wave without entries adds 0, whatever the mean.
      if (t % 64 == 0) {
        s_stat[flip][group][wave][0] = mean;
        s_stat[flip][group][wave][1] = sq;
      }
      __syncthreads();
      const float m = s_stat[flip][group][other][0], q2 = s_stat[flip][group][other][1];
      mean = wave_sum<kWaves>(n_other * m) * inv_d;
      sq = wave_sum<kWaves>(q2 + (share_other * (m - mean)) * (m - mean));
    }
    const float rstd = rsqrtf(sq + a.eps);
    const int64_t row = base + group;
    if (row < rows) {
      T* o = y + row * a.y_stride;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          f[k][i] = ga[k][i] * ((f[k][i] - mean) * rstd) + be[k][i];
        if (lo[k] < VEC) store_pack<T, VEC>(o + start[k], f[k], a.stream);
      }
      if (stats && t == 0) {
        stats[row] = mean;
        stats[rows + row] = rstd;
      }
    }
  }
}

// Work-group `block` of `blocks` of the backward.  WEIGHTS: also the sums of its rows for the weight
// gradients, into row `block` of part; they stay in registers until its last row is done.  One
// work-group of 16 waves to a compute unit: 256 partial rows, the fewest that fill the card, since
// each is 8 bytes a channel to write and read again (512 of them, half as long, cost 8192 x 4096
// bf16 52 us instead of 43).
template <typename T, int VEC, int TPR, int NV, int BLOCK, bool WEIGHTS>
__device__ __forceinline__ void bwd_rows(const NormArgs& a, const T* x, const float* gamma,
                                         const float* stats, const T* gy, T* gx, float* part,
                                         int block, int blocks) {
  constexpr int kGroups = BLOCK / TPR, kWaves = TPR > 64 ? TPR / 64 : 1;
  constexpr int kLanes = TPR < 64 ? TPR : 64;
  // the next row's loads go ahead of this one's sums where the registers allow
  constexpr bool kAhead = NV * VEC < 16;
  constexpr int kSets = BLOCK / (TPR < 64 ? 64 : TPR), kCols = TPR * VEC;
  __shared__ float s_sum[2][kGroups][kWaves][2];
  __shared__ float s_cols[WEIGHTS ? kSets : 1][WEIGHTS ? kCols : 1];
  const int tid = threadIdx.x, t = tid % TPR, group = tid / TPR, wave = t / 64;
  const int d = a.channels;
  const float inv_d = 1.0f / (float)d;
  int start[NV], lo[NV];
  float ga[NV][VEC], dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    place<VEC>(k * TPR + t, d, start[k], lo[k]);
    load_weight<VEC>(gamma, start[k], 1.f, ga[k]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) dg[k][i] = db[k][i] = 0.f;
  }
  bool partial = false;
#pragma unroll
  for (int k = 0; k < NV; ++k) partial |= lo[k] != 0;
  partial = __any(partial);
  const int64_t rows = a.batch, step = (int64_t)blocks * kGroups;
  int64_t base = (int64_t)block * kGroups;
  Raw<T, VEC> next_x[NV], next_g[NV];
  float next_mean = 0.f, next_rstd = 0.f;
  const auto fetch = [&](int64_t at) {
    const int64_t row = at + group < rows ? at + group : rows - 1;
    const T *p = x + row * a.x_stride, *r = gy + row * a.y_stride;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      next_x[k] = load_raw<T, VEC, true>(p + start[k]);
      next_g[k] = load_raw<T, VEC, true>(r + start[k]);
    }
    next_mean = stats[row];
    next_rstd = stats[rows + row];
  };
  if (kAhead && base < rows) fetch(base);
  int flip = 0;
  for (; base < rows; base += step, flip ^= 1) {
    const int64_t row = base + group;
    const bool live = row < rows;
    if (!kAhead) fetch(base);
    const float mean = next_mean, rstd = next_rstd;
    float h[NV][VEC], g[NV][VEC], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      unpack<T, VEC>(next_x[k], h[k]);
      unpack<T, VEC>(next_g[k], g[k]);
    }
    if (kAhead && base + step < rows) fetch(base + step);
    if (live) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          h[k][i] = (h[k][i] - mean) * rstd;
          if (WEIGHTS) {
            dg[k][i] += g[k][i] * h[k][i];
            db[k][i] += g[k][i];
          }
          g[k][i] *= ga[k][i];
        }
    }
    by_mask(partial, [&](auto masked) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float v = !masked.value || i >= lo[k] ? g[k][i] : 0.f;
          s1 += v;
          s2 += v * h[k][i];
        }
    });
    s1 = lane_sum<kLanes>(s1);
    s2 = lane_sum<kLanes>(s2);
    if (TPR > 64) {
      if (t % 64 == 0) {
        s_sum[flip][group][wave][0] = s1;
        s_sum[flip][group][wave][1] = s2;
      }
      __syncthreads();
      s1 = wave_sum<kWaves>(s_sum[flip][group][t % kWaves][0]);
      s2 = wave_sum<kWaves>(s_sum[flip][group][t % kWaves][1]);
    }
    s1 *= inv_d;
    s2 *= inv_d;
    if (gx && live) {
      T* o = gx + row * a.gx_stride;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) g[k][i] = rstd * (g[k][i] - s1 - h[k][i] * s2);
        if (lo[k] < VEC) store_pack<T, VEC>(o + start[k], g[k], a.stream);
      }
    }
  }
  if (!WEIGHTS) return;
  // the work-group's rows' sums of each column: lanes of a wave first, then its waves through LDS
  part += (int64_t)block * 2 * d;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float v = stride_sum<kLanes>(m == 0 ? dg[k][i] : db[k][i]);
        if (TPR >= 64 || tid % 64 < TPR)
          s_cols[tid / (TPR < 64 ? 64 : TPR)][t * VEC + i] = v;
      }
      __syncthreads();
      for (int c = tid; c < kCols; c += BLOCK) {
        int st, low;
        place<VEC>(k * TPR + c / VEC, d, st, low);
        if (c % VEC < low) continue;
        float v = 0.f;
#pragma unroll
        for (int s = 0; s < kSets; ++s) v += s_cols[s][c];
        part[(int64_t)m * d + st + c % VEC] = v;
      }
    }
}

template <typename T, int VEC, int TPR, int NV, int BLOCK, bool WEIGHTS>
__global__ __launch_bounds__(BLOCK) void k_ln_bwd_rows(NormArgs a, const T* x, const float* gamma,
                                                       const float* stats, const T* gy, T* gx,
                                                       float* part) {
  bwd_rows<T, VEC, TPR, NV, BLOCK, WEIGHTS>(a, x, gamma, stats, gy, gx, part, blockIdx.x,
                                            gridDim.x);
}

// Few rows: work-groups [0, row_blocks) take the rows, and the others 64 columns each, down all
// rows, whose weight gradients they finish: x and grad_y are read twice (out of a cache), which
// costs less than a second launch.
template <typename T, int VEC, int TPR, int NV, int BLOCK>
__global__ __launch_bounds__(BLOCK) void k_ln_bwd_few(NormArgs a, const T* x, const float* gamma,
                                                      const float* stats, const T* gy, T* gx,
                                                      float* ggamma, float* gbeta,
                                                      int row_blocks) {
  if ((int)blockIdx.x < row_blocks) {
    bwd_rows<T, VEC, TPR, NV, BLOCK, false>(a, x, gamma, stats, gy, gx, nullptr, blockIdx.x,
                                            row_blocks);
    return;
  }
  constexpr int kWaves = BLOCK / 64;
  __shared__ float s_sum[2][kWaves][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int c = (blockIdx.x - row_blocks) * 64 + lane, col = c < a.channels ? c : a.channels - 1;
  float sg = 0.f, sb = 0.f;
#pragma unroll 4
  for (int r = wave; r < (int)a.batch; r += kWaves) {
    const float g = to_float(gy[r * a.y_stride + col]);
    const float h = (to_float(x[r * a.x_stride + col]) - stats[r]) * stats[a.batch + r];
    sg += g * h;
    sb += g;
  }
  s_sum[0][wave][lane] = sg;
  s_sum[1][wave][lane] = sb;
  __syncthreads();
  if (threadIdx.x < 128 && c < a.channels) {
    float* out = wave == 0 ? ggamma : gbeta;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += s_sum[wave][w][lane];
    if (out) out[c] = v;
  }
}

// Rows longer than a work-group's registers hold (over 16384): sweeps over the row, which stays in
// the L2.
constexpr int kLong = 1024;

__device__ __forceinline__ float group_sum(float v, float* s_red) {
  v = lane_sum<64>(v);
  __syncthreads();
  if (threadIdx.x % 64 == 0) s_red[threadIdx.x / 64] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < kLong / 64; ++w) s += s_red[w];
  return s;
}

template <typename T>
__global__ __launch_bounds__(kLong) void k_ln_fwd_long(NormArgs a, const T* x, const float* gamma,
                                                       const float* beta, T* y, float* stats) {
  constexpr int VEC = kVec<T>;
  __shared__ float s_red[kLong / 64];
  const int tid = threadIdx.x, d = a.channels, nvec = (int)(((int64_t)d + VEC - 1) / VEC);
  const double inv_d = 1.0 / d;
  for (int64_t row = blockIdx.x; row < a.batch; row += gridDim.x) {
    const T* p = x + row * a.x_stride;
    T* q = y + row * a.y_stride;
    float f[VEC];
    double sum = 0.0, sq = 0.0;
    int st, lo;
    for (int j = tid; j < nvec; j += kLong) {
      place<VEC>(j, d, st, lo);
      load_pack<T, VEC>(p + st, f);
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) v += i >= lo ? f[i] : 0.f;
      sum += v;
    }
    const float mean = group_sum((float)sum, s_red) / (float)d;
    for (int j = tid; j < nvec; j += kLong) {
      place<VEC>(j, d, st, lo);
      load_pack<T, VEC>(p + st, f);
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) v += i >= lo ? (f[i] - mean) * (f[i] - mean) : 0.f;
      sq += v;
    }
    const float rstd = rsqrtf(group_sum((float)(sq * inv_d), s_red) + a.eps);
    // in place the vector that overlaps its neighbour must not read what that one wrote: the last
    // vector stores only its own elements, one by one
    for (int j = tid; j < nvec; j += kLong) {
      place<VEC>(j, d, st, lo);
      load_pack<T, VEC>(p + st, f);
      float ga[VEC], be[VEC];
      load_weight<VEC>(gamma, st, 1.f, ga);
      load_weight<VEC>(beta, st, 0.f, be);
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] = ga[i] * ((f[i] - mean) * rstd) + be[i];
      if (lo == 0) store_pack<T, VEC>(q + st, f);
      else
        for (int i = 0; i < VEC; ++i)
          if (i >= lo) q[st + i] = from_float<T>(f[i]);
    }
    if (stats && tid == 0) {
      stats[row] = mean;
      stats[a.batch + row] = rstd;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kLong) void k_ln_bwd_long(NormArgs a, const T* x, const float* gamma,
                                                       const float* stats, const T* gy, T* gx) {
  constexpr int VEC = kVec<T>;
  __shared__ float s_red[kLong / 64];
  const int tid = threadIdx.x, d = a.channels, nvec = (int)(((int64_t)d + VEC - 1) / VEC);
  for (int64_t row = blockIdx.x; row < a.batch; row += gridDim.x) {
    const T* p = x + row * a.x_stride;
    const T* r = gy + row * a.y_stride;
    T* q = gx + row * a.gx_stride;
    const float mean = stats[row], rstd = stats[a.batch + row];
    float h[VEC], g[VEC], ga[VEC];
    double sum1 = 0.0, sum2 = 0.0;
    int st, lo;
    for (int j = tid; j < nvec; j += kLong) {
      place<VEC>(j, d, st, lo);
      load_pack<T, VEC>(p + st, h);
      load_pack<T, VEC>(r + st, g);
      load_weight<VEC>(gamma, st, 1.f, ga);
      float v1 = 0.f, v2 = 0.f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float v = g[i] * ga[i];
        v1 += i >= lo ? v : 0.f;
        v2 += i >= lo ? v * ((h[i] - mean) * rstd) : 0.f;
      }
      sum1 += v1;
      sum2 += v2;
    }
    const float s1 = group_sum((float)sum1, s_red) / (float)d;
    const float s2 = group_sum((float)sum2, s_red) / (float)d;
    for (int j = tid; j < nvec; j += kLong) {
      place<VEC>(j, d, st, lo);
      load_pack<T, VEC>(p + st, h);
      load_pack<T, VEC>(r + st, g);
      load_weight<VEC>(gamma, st, 1.f, ga);
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        g[i] = rstd * (g[i] * ga[i] - s1 - (h[i] - mean) * rstd * s2);
      if (lo == 0) store_pack<T, VEC>(q + st, g);
      else
        for (int i = 0; i < VEC; ++i)
          if (i >= lo) q[st + i] = from_float<T>(g[i]);
    }
  }
}

// Column sums of long rows: work-group (slab, part) goes down the part's rows of its 256 vectors.
template <typename T>
__global__ __launch_bounds__(256) void k_ln_cols_long(NormArgs a, const T* x, const float* stats,
                                                      const T* gy, float* part) {
  constexpr int VEC = kVec<T>;
  const int d = a.channels;
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j * VEC >= d) return;
  int st, lo;
  place<VEC>((int)j, d, st, lo);
  float h[VEC], g[VEC], dg[VEC] = {}, db[VEC] = {};
  for (int64_t row = blockIdx.y; row < a.batch; row += gridDim.y) {
    load_pack<T, VEC>(x + row * a.x_stride + st, h);
    load_pack<T, VEC>(gy + row * a.y_stride + st, g);
    const float mean = stats[row], rstd = stats[a.batch + row];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      dg[i] += g[i] * ((h[i] - mean) * rstd);
      db[i] += g[i];
    }
  }
  part += (int64_t)blockIdx.y * 2 * d + st;
  for (int i = 0; i < VEC; ++i)
    if (i >= lo) {
      part[i] = dg[i];
      part[(int64_t)d + i] = db[i];
    }
}

// ---- fields (npts > 1) -------------------------------------------------------------------------
// A channel's points are next to one another, so lanes go along the points, VEC to a lane, and the
// sums over channels stay inside a lane.  A work-group takes a tile of points, and its waves share
// the channels, N each, in registers; what a point's channels sum to joins through LDS, one thread
// to a point, between two barriers (every wave adding up for itself needs only one, but reads LDS
// for as many values as the fields have: 4 x 100 x 100003 forward 79 us instead of 66, 8 x 64 x
// 512^2 bf16 141 instead of 124).  FLAT: one point to a lane, counted through all batch entries;
// else tiles of 64 VEC points of one entry.
struct Tile {
  int64_t b, p;   // batch entry and point where the tile starts (FLAT: of the lane's own point)
  uint32_t off;   // the lane's first element from there (below 64 VEC)
  int lo;         // the lane's own points are i >= lo
};

// The tiles of a work-group, a grid apart, without a division for each.
template <int VEC, bool FLAT>
struct Tiles {
  int64_t left, entry, at, step_entries, step_at;
  int blocks;
  __device__ __forceinline__ Tiles(int64_t tiles, int64_t per_entry, int block, int blocks_)
      : blocks(blocks_) {
    left = tiles - block;
    if (FLAT) {
      entry = step_entries = step_at = 0;
      at = block;
    } else {
      entry = uniform((int64_t)block / per_entry);
      at = (int64_t)block - entry * per_entry;
      step_entries = uniform((int64_t)blocks / per_entry);
      step_at = (int64_t)blocks - step_entries * per_entry;
    }
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next(int64_t per_entry) {
    left -= blocks;
    if (FLAT) {
      at += blocks;
      return;
    }
    entry += step_entries;
    at += step_at;
    if (at >= per_entry) {
      at -= per_entry;
      ++entry;
    }
  }
  __device__ __forceinline__ Tile tile(const NormArgs& a) const {
    Tile t;
    const int lane = threadIdx.x & 63;
    if (FLAT) {
      const int64_t rows = a.batch * a.npts;
      int64_t r = at * 64 + lane;
      t.lo = r < rows ? 0 : 1;
      r = r < rows ? r : rows - 1;
      t.off = 0;
      if (rows <= 0x7fffffff) {
        const uint32_t b = (uint32_t)r / (uint32_t)a.npts;
        t.b = b;
        t.p = (uint32_t)r - b * (uint32_t)a.npts;
      } else {
        t.b = r / a.npts;
        t.p = r - t.b * a.npts;
      }
    } else {
      t.b = entry;
      const int64_t first = at * (64 * VEC), last = a.npts - VEC;
      t.p = first < last ? first : last;
      const int most = last - t.p < 64 * VEC ? (int)(last - t.p) : 64 * VEC;
      const int e = (int)(first - t.p) + lane * VEC, own = e < most ? e : most;
      t.off = (uint32_t)own;
      t.lo = e - own < VEC ? e - own : VEC;
    }
    return t;
  }
};

template <typename T, int VEC>
__device__ __forceinline__ void store_own(T* p, const float (&f)[VEC], int lo, bool stream) {
  if (lo == 0) {
    store_pack<T, VEC>(p, f, stream);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i >= lo) p[i] = from_float<T>(f[i]);
  }
}

template <typename T, int N, int VEC, bool FLAT>
__global__ __launch_bounds__(N <= 8 ? 512 : 1024) void k_ln_fwd_field(
    NormArgs a, int64_t tiles, int64_t per_entry, const T* x, const float* gamma,
    const float* beta, T* y, float* stats) {
  extern __shared__ float s_mem[];  // a tile's means and deviations, then each wave's
  constexpr int kTile = 64 * VEC;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), waves = blockDim.x / 64;
  const int c0 = wave * N, nc = a.channels - c0 < N ? a.channels - c0 : N;
  const float inv_c = 1.0f / (float)a.channels, inv_n = 1.0f / (float)nc;
  const auto count = [&](int w) { return (float)(a.channels - w * N < N ? a.channels - w * N : N); };
  for (Tiles<VEC, FLAT> at(tiles, per_entry, blockIdx.x, gridDim.x); at.more();
       at.next(per_entry)) {
    const Tile t = at.tile(a);
    const T* p = x + t.b * a.x_stride + t.p;
    float f[N][VEC], mean[VEC] = {}, sq[VEC] = {};
#pragma unroll
    for (int c = 0; c < N; ++c)
      unpack<T, VEC>(
          load_raw<T, VEC, true>(p + (c < nc ? c0 + c : a.channels - 1) * a.npts + t.off), f[c]);
    by_mask(nc < N, [&](auto masked) {
#pragma unroll
      for (int c = 0; c < N; ++c)
#pragma unroll
        for (int i = 0; i < VEC; ++i) mean[i] += !masked.value || c < nc ? f[c][i] : 0.f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) mean[i] *= inv_n;
#pragma unroll
      for (int c = 0; c < N; ++c)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float e = f[c][i] - mean[i];
          sq[i] += !masked.value || c < nc ? e * e : 0.f;
        }
    });
    float rstd[VEC];
    if (waves > 1) {
      // the waves' means and squared deviations join, one point to a thread
      float *s_part = s_mem + 2 * kTile, *mine = s_part + wave * 2 * kTile + lane * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        mine[i] = mean[i];
        mine[kTile + i] = sq[i];
      }
      __syncthreads();
      for (int q = threadIdx.x; q < kTile; q += blockDim.x) {
        float all = 0.f, m2 = 0.f;
        for (int w = 0; w < waves; ++w) all += count(w) * s_part[w * 2 * kTile + q];
        all *= inv_c;
        for (int w = 0; w < waves; ++w) {
          const float e = s_part[w * 2 * kTile + q] - all;
          m2 += s_part[(w * 2 + 1) * kTile + q] + count(w) * e * e;
        }
        s_mem[q] = all;
        s_mem[kTile + q] = rsqrtf(m2 * inv_c + a.eps);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        mean[i] = s_mem[lane * VEC + i];
        rstd[i] = s_mem[kTile + lane * VEC + i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) rstd[i] = rsqrtf(sq[i] * inv_c + a.eps);
    }
    if (t.lo < VEC) {
      T* o = y + t.b * a.y_stride + t.p;
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (c < nc) {
          const float ga = gamma ? gamma[c0 + c] : 1.f, be = beta ? beta[c0 + c] : 0.f;
#pragma unroll
          for (int i = 0; i < VEC; ++i) f[c][i] = ga * ((f[c][i] - mean[i]) * rstd[i]) + be;
          store_own<T, VEC>(o + (c0 + c) * a.npts + t.off, f[c], t.lo, a.stream);
        }
      if (stats && wave == 0) {
        float* st = stats + t.b * a.npts + t.p;
        store_own<float, VEC>(st + t.off, mean, t.lo, false);
        store_own<float, VEC>(st + a.batch * a.npts + t.off, rstd, t.lo, false);
      }
    }
  }
}

// Work-group `block` of `blocks` of the backward.  WEIGHTS: also the sums of its points for the
// weight gradients, into row `block` of part.
template <typename T, int N, int VEC, bool FLAT, bool WEIGHTS>
__device__ __forceinline__ void bwd_field(const NormArgs& a, int64_t tiles, int64_t per_entry,
                                          const T* x, const float* gamma, const float* stats,
                                          const T* gy, T* gx, float* part, int block,
                                          int blocks) {
  extern __shared__ float s_mem[];  // a tile's two sums, then each wave's
  constexpr int kTile = 64 * VEC;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), waves = blockDim.x / 64;
  const int c0 = wave * N, nc = a.channels - c0 < N ? a.channels - c0 : N;
  const float inv_c = 1.0f / (float)a.channels;
  float dg[N] = {}, db[N] = {};
  for (Tiles<VEC, FLAT> at(tiles, per_entry, block, blocks); at.more(); at.next(per_entry)) {
    const Tile t = at.tile(a);
    const T* p = x + t.b * a.x_stride + t.p;
    const T* r = gy + t.b * a.y_stride + t.p;
    float h[N][VEC], g[N][VEC], mean[VEC], rstd[VEC], s1[VEC] = {}, s2[VEC] = {};
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const int64_t ch = (c < nc ? c0 + c : a.channels - 1) * a.npts;
      unpack<T, VEC>(load_raw<T, VEC, true>(p + ch + t.off), h[c]);
      unpack<T, VEC>(load_raw<T, VEC, true>(r + ch + t.off), g[c]);
    }
    const float* st = stats + t.b * a.npts + t.p;
    load_pack<float, VEC>(st + t.off, mean);
    load_pack<float, VEC>(st + a.batch * a.npts + t.off, rstd);
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const float ga = c < nc ? (gamma ? gamma[c0 + c] : 1.f) : 0.f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        h[c][i] = (h[c][i] - mean[i]) * rstd[i];
        if (WEIGHTS && i >= t.lo) {
          dg[c] += g[c][i] * h[c][i];
          db[c] += g[c][i];
        }
        g[c][i] *= ga;
        if (c < nc) {
          s1[i] += g[c][i];
          s2[i] += g[c][i] * h[c][i];
        }
      }
    }
    if (waves > 1) {
      float *s_part = s_mem + 2 * kTile, *mine = s_part + wave * 2 * kTile + lane * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        mine[i] = s1[i];
        mine[kTile + i] = s2[i];
      }
      __syncthreads();
      for (int q = threadIdx.x; q < 2 * kTile; q += blockDim.x) {
        float v = 0.f;
        for (int w = 0; w < waves; ++w) v += s_part[w * 2 * kTile + q];
        s_mem[q] = v;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        s1[i] = s_mem[lane * VEC + i];
        s2[i] = s_mem[kTile + lane * VEC + i];
      }
    }
    if (gx && t.lo < VEC) {
      T* o = gx + t.b * a.gx_stride + t.p;
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (c < nc) {
          float f[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            f[i] = rstd[i] * (g[c][i] - s1[i] * inv_c - h[c][i] * (s2[i] * inv_c));
          store_own<T, VEC>(o + (c0 + c) * a.npts + t.off, f, t.lo, a.stream);
        }
    }
  }
  if (!WEIGHTS) return;
  part += (int64_t)block * 2 * a.channels + c0;
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const float sg = lane_sum<64>(dg[c]), sb = lane_sum<64>(db[c]);
    if (lane == 0 && c < nc) {
      part[c] = sg;
      part[a.channels + c] = sb;
    }
  }
}

template <typename T, int N, int VEC, bool FLAT, bool WEIGHTS>
__global__ __launch_bounds__(1024) void k_ln_bwd_field(NormArgs a, int64_t tiles,
                                                       int64_t per_entry, const T* x,
                                                       const float* gamma, const float* stats,
                                                       const T* gy, T* gx, float* part) {
  bwd_field<T, N, VEC, FLAT, WEIGHTS>(a, tiles, per_entry, x, gamma, stats, gy, gx, part,
                                      blockIdx.x, gridDim.x);
}

// Few points: as k_ln_bwd_few, with a channel to each of the work-groups from tile_blocks on.
template <typename T, int N, int VEC, bool FLAT>
__global__ __launch_bounds__(1024) void k_ln_bwd_field_few(NormArgs a, int64_t tiles,
                                                           int64_t per_entry, const T* x,
                                                           const float* gamma, const float* stats,
                                                           const T* gy, T* gx, float* ggamma,
                                                           float* gbeta, int tile_blocks) {
  if ((int)blockIdx.x < tile_blocks) {
    bwd_field<T, N, VEC, FLAT, false>(a, tiles, per_entry, x, gamma, stats, gy, gx, nullptr,
                                      blockIdx.x, tile_blocks);
    return;
  }
  __shared__ float s_sum[2][16];
  constexpr int V = FLAT ? 1 : 4;
  const int c = blockIdx.x - tile_blocks, npts = (int)a.npts, rows = (int)a.batch * npts;
  const int per = (npts + V - 1) / V, vectors = (int)a.batch * per;
  const T *p = x + c * a.npts, *r = gy + c * a.npts;
  float sg = 0.f, sb = 0.f;
#pragma unroll 4
  for (int q = threadIdx.x; q < vectors; q += blockDim.x) {
    const int b = (uint32_t)q / (uint32_t)per;
    int at, lo;
    place<V>(q - b * per, npts, at, lo);
    float g[V], h[V], mean[V], rstd[V];
    load_pack<T, V>(r + b * a.y_stride + at, g);
    load_pack<T, V>(p + b * a.x_stride + at, h);
    load_pack<float, V>(stats + b * npts + at, mean);
    load_pack<float, V>(stats + rows + b * npts + at, rstd);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i >= lo) {
        sg += g[i] * ((h[i] - mean[i]) * rstd[i]);
        sb += g[i];
      }
  }
  sg = lane_sum<64>(sg);
  sb = lane_sum<64>(sb);
  if (threadIdx.x % 64 == 0) {
    s_sum[0][threadIdx.x / 64] = sg;
    s_sum[1][threadIdx.x / 64] = sb;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    float v = 0.f;
    for (int w = 0; w < (int)blockDim.x / 64; ++w) v += s_sum[threadIdx.x][w];
    float* out = threadIdx.x == 0 ? ggamma : gbeta;
    if (out) out[c] = v;
  }
}

// Fields of more channels than a work-group holds: one thread to a point, sweeps over the channels.
// What a thread adds up in one chain, here and in the long rows (there vector by vector), is float64:
// a float32 chain of 9000 channels is off by more than the rest of the arithmetic together, and its
// squares overflow where the variance does not.
template <typename T>
__global__ __launch_bounds__(256) void k_ln_fwd_points(NormArgs a, const T* x, const float* gamma,
                                                       const float* beta, T* y, float* stats) {
  const int64_t rows = a.batch * a.npts;
  for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < rows;
       r += (int64_t)gridDim.x * 256) {
    const int64_t b = r / a.npts, p = r - b * a.npts;
    const T* xr = x + b * a.x_stride + p;
    T* yr = y + b * a.y_stride + p;
    double sum = 0.0, sq = 0.0;
    for (int c = 0; c < a.channels; ++c) sum += to_float(xr[c * a.npts]);
    const float mean = (float)(sum / a.channels);
    for (int c = 0; c < a.channels; ++c) {
      const double d = to_float(xr[c * a.npts]) - mean;
      sq += d * d;
    }
    const float rstd = rsqrtf((float)(sq / a.channels) + a.eps);
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
__global__ __launch_bounds__(256) void k_ln_bwd_points(NormArgs a, const T* x, const float* gamma,
                                                       const float* stats, const T* gy, T* gx) {
  const int64_t rows = a.batch * a.npts;
  for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < rows;
       r += (int64_t)gridDim.x * 256) {
    const int64_t b = r / a.npts, p = r - b * a.npts;
    const T* xr = x + b * a.x_stride + p;
    const T* gr = gy + b * a.y_stride + p;
    T* o = gx + b * a.gx_stride + p;
    const float mean = stats[r], rstd = stats[rows + r];
    double sum1 = 0.0, sum2 = 0.0;
    for (int c = 0; c < a.channels; ++c) {
      const float g = to_float(gr[c * a.npts]) * (gamma ? gamma[c] : 1.f);
      sum1 += g;
      sum2 += (double)g * ((to_float(xr[c * a.npts]) - mean) * rstd);
    }
    const float s1 = (float)(sum1 / a.channels), s2 = (float)(sum2 / a.channels);
    for (int c = 0; c < a.channels; ++c) {
      const float g = to_float(gr[c * a.npts]) * (gamma ? gamma[c] : 1.f);
      const float h = (to_float(xr[c * a.npts]) - mean) * rstd;
      o[c * a.npts] = from_float<T>(rstd * (g - s1 - h * s2));
    }
  }
}

// Work-group (part, c): the sums of grad_y h and grad_y over the part's points of channel c.
template <typename T>
__global__ __launch_bounds__(256) void k_ln_cols_points(NormArgs a, const T* x, const float* stats,
                                                        const T* gy, float* part) {
  __shared__ float s_red[2][4];
  const int64_t rows = a.batch * a.npts;
  const int tid = threadIdx.x;
  for (int64_t c = blockIdx.y; c < a.channels; c += gridDim.y) {
    float sg = 0.f, sb = 0.f;
    for (int64_t r = (int64_t)blockIdx.x * 256 + tid; r < rows; r += (int64_t)gridDim.x * 256) {
      const int64_t b = r / a.npts, at = (r - b * a.npts) + c * a.npts;
      const float g = to_float(gy[b * a.y_stride + at]);
      const float h = (to_float(x[b * a.x_stride + at]) - stats[r]) * stats[rows + r];
      sg += g * h;
      sb += g;
    }
    sg = lane_sum<64>(sg);
    sb = lane_sum<64>(sb);
    __syncthreads();
    if (tid % 64 == 0) {
      s_red[0][tid / 64] = sg;
      s_red[1][tid / 64] = sb;
    }
    __syncthreads();
    if (tid < 2)
      part[((int64_t)blockIdx.x * 2 + tid) * a.channels + c] =
          (s_red[tid][0] + s_red[tid][1]) + (s_red[tid][2] + s_red[tid][3]);
  }
}

// ---- the weight gradients: sums of the parts' rows [nparts][2][channels] -------------------------
// COLS columns to a work-group at a time, 256 / COLS threads down each.
template <int COLS>
__global__ __launch_bounds__(256) void k_ln_finish(int channels, int nparts, const float* part,
                                                   float* ggamma, float* gbeta) {
  constexpr int kSlices = 256 / COLS;
  __shared__ float s_red[kSlices][COLS];
  const int col = threadIdx.x % COLS, slice = threadIdx.x / COLS;
  const int64_t width = 2 * (int64_t)channels, step = (int64_t)gridDim.x * COLS;
  for (int64_t base = (int64_t)blockIdx.x * COLS; base < width; base += step) {
    const int64_t i = base + col;
    float s = 0.f;
    if (i < width)
#pragma unroll 8
      for (int k = slice; k < nparts; k += kSlices) s += part[k * width + i];
    s_red[slice][col] = s;
    __syncthreads();
    if (slice == 0 && i < width) {
      for (int w = 1; w < kSlices; ++w) s += s_red[w][col];
      float* out = i < channels ? ggamma : gbeta;
      if (out) out[i < channels ? i : i - channels] = s;
    }
    __syncthreads();
  }
}

// ---- launches ----------------------------------------------------------------------------------
constexpr int kMaxField = 256;   // channels that a field's work-group holds
constexpr int kPointParts = 64;  // parts of the kernels that sweep

enum Form { kRows, kLongRows, kField, kPoints };
template <typename T>
Form form_of(const NormArgs& a) {
  if (a.npts == 1) return a.channels <= 16384 ? kRows : kLongRows;
  return a.channels <= kMaxField ? kField : kPoints;
}

int64_t cut(int64_t v, int64_t most) { return v < most ? v : most; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Work-groups of a kernel that the 256 compute units hold at a time (asked for once).
template <auto Kernel>
int64_t resident(int block) {
  static const int64_t n = [block]() {
    int per_cu = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, Kernel, block, 0) != hipSuccess)
      per_cu = 1;
    return (int64_t)256 * (per_cu > 0 ? per_cu : 1);
  }();
  return n;
}

// Calls f(elements of a vector, threads to a row, vectors to a thread) as constants.
template <int N>
struct Int {
  static constexpr int value = N;
};
template <typename T, typename F>
void pick_rows(int channels, F&& f) {
  constexpr int VEC = kVec<T>, NV = 8 / VEC;  // 8 elements to a thread, 16 in the longest rows
  if (channels < VEC) return f(Int<1>(), Int<8>(), Int<1>());
  const int nvec = (channels + VEC - 1) / VEC;
  const Int<VEC> v;
  if (nvec <= 8) return f(v, Int<8>(), Int<1>());
  if (nvec <= 16) return f(v, Int<16>(), Int<1>());
  if (nvec <= 32) return f(v, Int<32>(), Int<1>());
  if (nvec <= 64) return f(v, Int<64>(), Int<1>());
  if constexpr (NV > 1)
    if (nvec <= 64 * NV) return f(v, Int<64>(), Int<NV>());
  if (nvec <= 128 * NV) return f(v, Int<128>(), Int<NV>());
  if (nvec <= 256 * NV) return f(v, Int<256>(), Int<NV>());
  if (nvec <= 512 * NV) return f(v, Int<512>(), Int<NV>());
  if (nvec <= 1024 * NV) return f(v, Int<1024>(), Int<NV>());
  return f(v, Int<1024>(), Int<2 * NV>());
}

constexpr int kBwdBlock = 1024;
template <int TPR>
int bwd_rows_groups(int64_t rows) {
  return (int)cut(ceil_div(rows, kBwdBlock / TPR), 256);
}

// Fields: channels to a wave, at most 8 for up to 64 channels (and so at most 8 waves).  Float32
// forward with up to 12 from 49 channels on: 4 x 64 x 300000 126 us against 123, 2 x 64 x 1024^2 200
// against 193, 8 x 50 x 512^2 149 against 148.
int field_n(int c) {
  if (c <= 64) return (int)ceil_div(c, ceil_div(c, 8));
  return c <= 100 ? 10 : c <= 120 ? 12 : 16;
}
template <typename F>
void pick_field(int c, F&& f) {
  switch (field_n(c)) {
    case 1: return f(Int<1>());
    case 2: return f(Int<2>());
    case 3: return f(Int<3>());
    case 4: return f(Int<4>());
    case 5: return f(Int<5>());
    case 6: return f(Int<6>());
    case 7: return f(Int<7>());
    case 8: return f(Int<8>());
    case 10: return f(Int<10>());
    case 12: return f(Int<12>());
    default: return f(Int<16>());
  }
}

// Points to a lane.  Forward: 4 (8 of a half type, whole 16-byte loads, spill: 8 x 64 x 512^2 bf16
// 202 us against 141).  Backward, with twice the registers: 2 (4: 496 us against 322 on
// 8 x 64 x 512^2 float32, before streaming stores), 1 beyond 10 channels a wave.
template <typename T>
constexpr int kFwdVec = 4;
template <typename T, int N>
constexpr int kBwdVec = N <= 10 ? 2 : 1;
struct FieldShape {
  bool flat;
  int waves;
  int64_t per_entry, tiles;
  size_t lds;
};
// Entries below 256 points go FLAT.  Forward, flat and not: 400 x 32 x 200 9.0 and 9.4 us,
// 400 x 32 x 300 12.6 and 12.1, 400 x 32 x 600 18.9 and 14.4.
FieldShape field_shape(const NormArgs& a, int n, int wide) {
  FieldShape s;
  s.flat = a.npts < 256;
  const int vec = s.flat ? 1 : wide;
  s.waves = (int)ceil_div(a.channels, n);
  s.per_entry = ceil_div(a.npts, 64 * vec);
  s.tiles = s.flat ? ceil_div(a.batch * a.npts, 64) : a.batch * s.per_entry;
  s.lds = s.waves > 1 ? sizeof(float) * (1 + s.waves) * 2 * 64 * vec : 0;
  return s;
}
int field_bwd_groups(const FieldShape& s) { return (int)cut(s.tiles, ceil_div(8192, s.waves)); }

// Whether an output goes past the caches (nontemporal stores): where it is larger than the 256 MB
// cache behind the L2s, and its rows or planes are whole 128-byte lines.  Forward, with and without:
// 8 x 64 x 512^2 (537 MB) 196 against 208 us, 2 x 20 x 128^3 (336 MB) 140 against 149; backward 291
// against 319 and 201 against 217.  Below it the cache takes the writes: 8 x 20 x 512^2 (168 MB) 65
// against 60, backward 111 against 102.  Lines that two work-groups share suffer: 8 x 20 x 300001
// 92 against 72, backward 171 against 130.
template <typename T>
bool stream_out(const NormArgs& a, const T* out, int64_t stride) {
  const int64_t pitch = (a.npts == 1 ? stride : a.npts) * (int64_t)sizeof(T);
  return a.batch * a.npts * a.channels * (int64_t)sizeof(T) > ((int64_t)256 << 20) && pitch % 128 == 0 &&
         (a.batch <= 1 || stride * (int64_t)sizeof(T) % 128 == 0) &&
         reinterpret_cast<uintptr_t>(out) % 128 == 0;
}

// Dynamic LDS with which a compute unit (160 KB) holds at most as many of the float32 forward's
// work-groups as make up 16 waves, rounded up to whole ones, where its output streams; 0: no limit.
// Time with the limit over time without, 4 to 256 channels, 64 to 200 million entries:
//   planes of 2^16 to 500000 points, up to 8 waves     0.92 to 1.02, 0.986 in the mean
//   planes a multiple of 2 MB apart (2^19 points)
//     2 to 4 waves (9 to 32 channels), 2^21 and more   0.85 to 1.02, 0.956
//     the same, fewer points                           0.96 to 1.15, 1.012
//     1 and 5 to 8 waves                               0.91 to 1.06, 0.999
//   9 to 16 waves                                      0.99 to 1.01, 1.000
// The first two kinds take it: 5 x 64 x 512^2 119 us against 130, 2 x 20 x 128^3 135 against 140, but
// 5 x 32 x 2^19 165 against 147.  12 and 8 waves gain nothing more and cost narrow fields up to 15%.
// The backward's registers limit its waves already.  Outputs that the cache takes, and half ones, want
// all the waves: 16 x 32 x 256^2 49.2 against 48.5, 8 x 20 x 300001 75 against 72, 8 x 64 x 512^2 bf16
// 134 against 123.
size_t lds_for_16_waves(int waves, int64_t npts) {
  const bool apart = npts * 4 % (2 << 20) == 0;
  if (waves > 8 || (apart && (waves == 1 || waves > 4 || npts < 1 << 21))) return 0;
  const int groups = (int)ceil_div(16, waves), total = 160 << 10;
  return total / (groups + 1) / 512 * 512 + 512;
}

template <typename T>
hipError_t fwd_t(NormArgs a, const T* x, const float* gamma, const float* beta, T* y,
                 float* stats, hipStream_t s) {
  a.stream = stream_out(a, y, a.y_stride);
  switch (form_of<T>(a)) {
    case kRows:
      pick_rows<T>(a.channels, [&](auto vec, auto tpr, auto nv) {
        constexpr int kBlock = tpr.value < 256 ? 256 : tpr.value;
        constexpr auto kernel = k_ln_fwd_rows<T, vec.value, tpr.value, nv.value, kBlock>;
        // As many rounds as the resident work-groups take, shared out evenly; half of them where the
        // output streams to memory: 65536 x 4096 bf16 177 us against 191, 262144 x 1024 176 against
        // 197, 16384 x 8192 float32 183 against 189, 131072 x 1024 196 against 195.
        const int64_t need = ceil_div(a.batch, kBlock / tpr.value);
        const int64_t most = resident<kernel>(kBlock) / (a.stream ? 2 : 1);
        const int64_t groups = ceil_div(need, ceil_div(need, most));
        hipLaunchKernelGGL(kernel, dim3(groups), dim3(kBlock), 0, s, a, x, gamma, beta, y, stats);
      });
      break;
    case kLongRows:
      hipLaunchKernelGGL(k_ln_fwd_long<T>, dim3(cut(a.batch, 1024)), dim3(kLong), 0, s, a, x, gamma,
                         beta, y, stats);
      break;
    case kField:
      pick_field(a.channels, [&](auto n) {
        FieldShape f = field_shape(a, n.value, kFwdVec<T>);
        if (sizeof(T) == 4 && a.stream) f.lds = std::max(f.lds, lds_for_16_waves(f.waves, a.npts));
        const dim3 grid(cut(f.tiles, 1 << 20)), block(64 * f.waves);
        if (f.flat)
          hipLaunchKernelGGL((k_ln_fwd_field<T, n.value, 1, true>), grid, block, f.lds, s, a,
                             f.tiles, f.per_entry, x, gamma, beta, y, stats);
        else
          hipLaunchKernelGGL((k_ln_fwd_field<T, n.value, kFwdVec<T>, false>), grid, block, f.lds,
                             s, a, f.tiles, f.per_entry, x, gamma, beta, y, stats);
      });
      break;
    case kPoints:
      hipLaunchKernelGGL(k_ln_fwd_points<T>, dim3(cut(ceil_div(a.batch * a.npts, 256), 4096)),
                         dim3(256), 0, s, a, x, gamma, beta, y, stats);
  }
  return hipGetLastError();
}

// work-groups of the backward's pass over rows, and rows of its partial sums
template <typename T>
int groups_t(const NormArgs& a) {
  if (a.batch == 0 || a.npts == 0) return 0;
  switch (form_of<T>(a)) {
    case kRows: {
      int n = 0;
      pick_rows<T>(a.channels,
                   [&](auto, auto tpr, auto) { n = bwd_rows_groups<tpr.value>(a.batch); });
      return n;
    }
    case kField: {
      int n = 0;
      pick_field(a.channels, [&](auto c) {
        n = field_bwd_groups(field_shape(a, c.value, kBwdVec<T, c.value>));
      });
      return n;
    }
    default: return (int)cut(a.npts == 1 ? a.batch : kPointParts, kPointParts);
  }
}

hipError_t finish(const NormArgs& a, int parts, const float* part, float* ggamma, float* gbeta,
                  hipStream_t s) {
  const int64_t width = 2 * (int64_t)a.channels;
  // a launch has fewer than 2^32 threads: 2^22 work-groups go over more columns in turn (with more
  // the runtime starts only a part of them, and says nothing)
  const auto go = [&](auto cols) {
    hipLaunchKernelGGL(k_ln_finish<cols.value>, dim3(cut(ceil_div(width, cols.value), 1 << 22)),
                       dim3(256), 0, s, a.channels, parts, part, ggamma, gbeta);
    return hipGetLastError();
  };
  return width >= 8192 ? go(Int<64>()) : width >= 1024 ? go(Int<16>()) : go(Int<4>());
}

// Whether the weight gradients come from the columns' own reading of x and grad_y and not from
// partial sums of the rows' pass: few enough rows that this is short, which saves a launch (4 us for
// the host) and the workspace.  On the GPU, one launch against two and their gap: 48 x 640 float32
// 3.7 us against 8; 512 x 1024 6.7 against 10; 5 x 20 x 4095 (27 vectors to a thread) 10 against 10,
// 20 x 26000 (34) 12 against 10; 16 x 32 x 250 (16 points to a thread) 6.4 against 9, 32 x 16 x 250
// (62) 16 against 9.  By the shape alone, so that what else is asked for does not change their bits.
template <typename T>
bool few(const NormArgs& a) {
  const int64_t rows = a.batch * a.npts;
  if (rows * a.channels > 1 << 19) return false;
  if (form_of<T>(a) == kRows) return rows <= 512;
  if (form_of<T>(a) != kField) return false;
  // a channel's work-group has 64 threads for each wave of the tiles'
  const int threads = 64 * (int)ceil_div(a.channels, field_n(a.channels));
  return rows <= threads * (a.npts < 256 ? 16 : 4 * 28);
}

template <typename T>
hipError_t bwd_t(NormArgs a, const T* x, const float* gamma, const float* stats, const T* gy,
                 T* gx, float* ggamma, float* gbeta, float* part, hipStream_t s) {
  const bool weights = ggamma || gbeta, by_columns = few<T>(a);
  const int groups = groups_t<T>(a);
  // one launch takes the rows and the columns, except in place, where the columns go first
  if (by_columns && weights && gx && (gx == x || gx == gy)) {
    const hipError_t e = bwd_t<T>(a, x, gamma, stats, gy, nullptr, ggamma, gbeta, part, s);
    return e != hipSuccess ? e : bwd_t<T>(a, x, gamma, stats, gy, gx, nullptr, nullptr, part, s);
  }
  const bool columns = by_columns && weights, sums = weights && !by_columns;
  const int with_rows = gx ? groups : 0;  // work-groups before the columns'
  a.stream = stream_out(a, gx, a.gx_stride);
  switch (form_of<T>(a)) {
    case kRows:
      pick_rows<T>(a.channels, [&](auto vec, auto tpr, auto nv) {
        constexpr int V = vec.value, TPR = tpr.value, NV = nv.value;
        if (columns)
          hipLaunchKernelGGL((k_ln_bwd_few<T, V, TPR, NV, kBwdBlock>),
                             dim3(with_rows + ceil_div(a.channels, 64)), dim3(kBwdBlock), 0, s, a, x,
                             gamma, stats, gy, gx, ggamma, gbeta, with_rows);
        else if (sums)
          hipLaunchKernelGGL((k_ln_bwd_rows<T, V, TPR, NV, kBwdBlock, true>), dim3(groups),
                             dim3(kBwdBlock), 0, s, a, x, gamma, stats, gy, gx, part);
        else
          hipLaunchKernelGGL((k_ln_bwd_rows<T, V, TPR, NV, kBwdBlock, false>), dim3(groups),
                             dim3(kBwdBlock), 0, s, a, x, gamma, stats, gy, gx, part);
      });
      break;
    case kField:
      pick_field(a.channels, [&](auto n) {
        constexpr int N = n.value, kWide = kBwdVec<T, N>;
        const FieldShape f = field_shape(a, N, kWide);
        const auto go = [&](auto vec, auto flat) {
          constexpr int V = vec.value;
          constexpr bool F = flat.value;
          const dim3 grid(groups), block(64 * f.waves);
          if (columns)
            hipLaunchKernelGGL((k_ln_bwd_field_few<T, N, V, F>), dim3(with_rows + a.channels), block,
                               f.lds, s, a, f.tiles, f.per_entry, x, gamma, stats, gy, gx, ggamma,
                               gbeta, with_rows);
          else if (sums)
            hipLaunchKernelGGL((k_ln_bwd_field<T, N, V, F, true>), grid, block, f.lds, s, a,
                               f.tiles, f.per_entry, x, gamma, stats, gy, gx, part);
          else
            hipLaunchKernelGGL((k_ln_bwd_field<T, N, V, F, false>), grid, block, f.lds, s, a,
                               f.tiles, f.per_entry, x, gamma, stats, gy, gx, part);
        };
        if (f.flat) go(Int<1>(), std::true_type());
        else go(Int<kWide>(), std::false_type());
      });
      break;
    // the column sums first: grad_x may overwrite x or grad_y
    case kLongRows:
      if (weights)
        hipLaunchKernelGGL(k_ln_cols_long<T>, dim3(ceil_div(a.channels, 256 * kVec<T>), groups),
                           dim3(256), 0, s, a, x, stats, gy, part);
      if (gx)
        hipLaunchKernelGGL(k_ln_bwd_long<T>, dim3(cut(a.batch, 1024)), dim3(kLong), 0, s, a, x,
                           gamma, stats, gy, gx);
      break;
    case kPoints:
      if (weights)
        hipLaunchKernelGGL(k_ln_cols_points<T>, dim3(groups, cut(a.channels, 32768)), dim3(256), 0,
                           s, a, x, stats, gy, part);
      if (gx)
        hipLaunchKernelGGL(k_ln_bwd_points<T>, dim3(cut(ceil_div(a.batch * a.npts, 256), 4096)),
                           dim3(256), 0, s, a, x, gamma, stats, gy, gx);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !sums) return e;
  return finish(a, groups, part, ggamma, gbeta, s);
}

}  // namespace

hipError_t launch_layer_norm_fwd(const NormArgs& a, int dtype, const void* x, const float* gamma,
                                 const float* beta, void* y, float* stats, hipStream_t s) {
  const auto go = [&](auto t) {
    typedef decltype(t) T;
    return fwd_t<T>(a, static_cast<const T*>(x), gamma, beta, static_cast<T*>(y), stats, s);
  };
  if (dtype == FNO_DTYPE_F32) return go(0.f);
  return dtype == FNO_DTYPE_BF16 ? go((__bf16)0.f) : go((_Float16)0.f);
}

int layer_norm_parts(const NormArgs& a, int dtype) {
  const auto parts = [&](auto t) {
    typedef decltype(t) T;
    return few<T>(a) ? 0 : groups_t<T>(a);
  };
  return dtype == FNO_DTYPE_F32 ? parts(0.f) : parts((__bf16)0.f);
}

hipError_t launch_layer_norm_bwd(const NormArgs& a, int dtype, const void* x, const float* gamma,
                                 const float* stats, const void* gy, void* gx, float* ggamma,
                                 float* gbeta, float* part, hipStream_t s) {
  if (a.batch == 0 || a.npts == 0) return finish(a, 0, part, ggamma, gbeta, s);
  const auto go = [&](auto t) {
    typedef decltype(t) T;
    return bwd_t<T>(a, static_cast<const T*>(x), gamma, stats, static_cast<const T*>(gy),
                    static_cast<T*>(gx), ggamma, gbeta, part, s);
  };
  if (dtype == FNO_DTYPE_F32) return go(0.f);
  return dtype == FNO_DTYPE_BF16 ? go((__bf16)0.f) : go((_Float16)0.f);
}

}  // namespace fno
