// Layer norm over the channels of a field [batch][channels][npts], forward and backward.
#include "train_device.h"
#include "train_ops.h"

namespace fno {
namespace {

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);  // elements of a 16-byte load

// ---- rows (npts = 1) ---------------------------------------------------------------------------
// Threads(TPR) hold a row, NV vectors of VEC elements each.  Vector j of the row starts at element
// j VEC; the last one is moved back to end with the row, and the elements that it then shares with
// its neighbour (i < lo) count once in sums and are stored twice with the same value.
template <int VEC>
__device__ __forceinline__ void place(int j, int d, int& start, int& lo) {
  const int e = j * VEC;
  start = e < d - VEC ? e : d - VEC;
  lo = e < d ? e - start : VEC;
}

// elements of the row that wave `w` of the row's waves holds (TPR >= 64)
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

template <typename T, int VEC, int TPR, int NV, int BLOCK>
__global__ __launch_bounds__(BLOCK) void k_ln_fwd_rows(NormArgs a, const T* x, const float* gamma,
                                                       const float* beta, T* y, float* stats) {
  constexpr int kGroups = BLOCK / TPR, kWaves = TPR > 64 ? TPR / 64 : 1;
  __shared__ float s_stat[2][kGroups][kWaves][2];
  const int tid = threadIdx.x, t = tid % TPR, group = tid / TPR, wave = t / 64;
  const int d = a.channels;
  const float inv_d = 1.0f / (float)d;
  int start[NV], lo[NV];
  float ga[NV][VEC], be[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    place<VEC>(k * TPR + t, d, start[k], lo[k]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      ga[k][i] = gamma ? gamma[start[k] + i] : 1.f;
      be[k][i] = beta ? beta[start[k] + i] : 0.f;
    }
  }
  const int64_t rows = a.batch, step = (int64_t)gridDim.x * kGroups;
  int64_t base = (int64_t)blockIdx.x * kGroups;
  Pack<T, VEC> next[NV];
  const auto fetch = [&](int64_t at) {
    const int64_t row = at + group < rows ? at + group : rows - 1;
    const T* p = x + row * a.x_stride;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      next[k] = *reinterpret_cast<const Pack<T, VEC>*>(p + start[k]);
  };
  if (base < rows) fetch(base);
  int flip = 0;
  for (; base < rows; base += step, flip ^= 1) {
    float f[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV; ++k) unpack<T, VEC>(next[k], f[k]);
    if (base + step < rows) fetch(base + step);
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum += i >= lo[k] ? f[k][i] : 0.f;
    sum = lane_sum<(TPR < 64 ? TPR : 64)>(sum);
    const float n = TPR > 64 ? wave_count<VEC, TPR, NV>(wave, d) : (float)d;
    float mean = TPR > 64 ? sum / fmaxf(n, 1.f) : sum * inv_d;
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float c = f[k][i] - mean;
        sq += i >= lo[k] ? c * c : 0.f;
      }
    sq = lane_sum<(TPR < 64 ? TPR : 64)>(sq);
    if (TPR > 64) {
      // the waves' means and squared deviations join: M2 = sum M2_w + n_w (mean_w - mean)^2
      if (t % 64 == 0) {
        s_stat[flip][group][wave][0] = mean;
        s_stat[flip][group][wave][1] = sq;
      }
      __syncthreads();
      float mw[kWaves], nw[kWaves], all = 0.f;
      sq = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        mw[w] = s_stat[flip][group][w][0];
        sq += s_stat[flip][group][w][1];
        nw[w] = wave_count<VEC, TPR, NV>(w, d);
        all += nw[w] * mw[w];
      }
      mean = all * inv_d;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) sq += nw[w] * (mw[w] - mean) * (mw[w] - mean);
    }
    const float rstd = 1.0f / sqrtf(sq * inv_d + a.eps);
    const int64_t row = base + group;
    if (row < rows) {
      T* q = y + row * a.y_stride;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = ga[k][i] * ((f[k][i] - mean) * rstd) + be[k][i];
        if (lo[k] < VEC) store_pack<T, VEC>(q + start[k], o);
      }
      if (stats && t == 0) {
        stats[row] = mean;
        stats[rows + row] = rstd;
      }
    }
  }
}

template <typename T, int VEC, int TPR, int NV, int BLOCK>
__global__ __launch_bounds__(BLOCK) void k_ln_bwd_rows(NormArgs a, const T* x, const float* gamma,
                                                       const float* stats, const T* gy, T* gx,
                                                       float* part) {
  constexpr int kGroups = BLOCK / TPR, kWaves = TPR > 64 ? TPR / 64 : 1;
  constexpr bool kAhead = NV * VEC < 16;  // the next row's loads ahead, where registers allow
  constexpr int kSets = BLOCK / (TPR < 64 ? 64 : TPR), kCols = TPR * VEC;
  __shared__ float s_sum[2][kGroups][kWaves][2];
  __shared__ float s_cols[kSets][kCols];
  const int tid = threadIdx.x, t = tid % TPR, group = tid / TPR, wave = t / 64;
  const int d = a.channels;
  const float inv_d = 1.0f / (float)d;
  int start[NV], lo[NV];
  float ga[NV][VEC], dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    place<VEC>(k * TPR + t, d, start[k], lo[k]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      ga[k][i] = gamma ? gamma[start[k] + i] : 1.f;
      dg[k][i] = db[k][i] = 0.f;
    }
  }
  const int64_t rows = a.batch, step = (int64_t)gridDim.x * kGroups;
  int64_t base = (int64_t)blockIdx.x * kGroups;
  Pack<T, VEC> nx[NV], ng[NV];
  float nmean = 0.f, nrstd = 0.f;
  const auto fetch = [&](int64_t at) {
    const int64_t row = at + group < rows ? at + group : rows - 1;
    const T* p = x + row * a.x_stride;
    const T* q = gy + row * a.y_stride;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      nx[k] = *reinterpret_cast<const Pack<T, VEC>*>(p + start[k]);
      ng[k] = *reinterpret_cast<const Pack<T, VEC>*>(q + start[k]);
    }
    nmean = stats[row];
    nrstd = stats[rows + row];
  };
  if (kAhead && base < rows) fetch(base);
  int flip = 0;
  for (; base < rows; base += step, flip ^= 1) {
    const int64_t row = base + group;
    const bool live = row < rows;
    if (!kAhead) fetch(base);
    const float mean = nmean, rstd = nrstd;
    float h[NV][VEC], g[NV][VEC], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      unpack<T, VEC>(nx[k], h[k]);
      unpack<T, VEC>(ng[k], g[k]);
    }
    if (kAhead && base + step < rows) fetch(base + step);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const bool mine = i >= lo[k];
        h[k][i] = (h[k][i] - mean) * rstd;
        if (live) {
          dg[k][i] += g[k][i] * h[k][i];
          db[k][i] += g[k][i];
        }
        g[k][i] *= ga[k][i];
        s1 += mine ? g[k][i] : 0.f;
        s2 += mine ? g[k][i] * h[k][i] : 0.f;
      }
    s1 = lane_sum<(TPR < 64 ? TPR : 64)>(s1);
    s2 = lane_sum<(TPR < 64 ? TPR : 64)>(s2);
    if (TPR > 64) {
      if (t % 64 == 0) {
        s_sum[flip][group][wave][0] = s1;
        s_sum[flip][group][wave][1] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        s1 += s_sum[flip][group][w][0];
        s2 += s_sum[flip][group][w][1];
      }
    }
    s1 *= inv_d;
    s2 *= inv_d;
    if (gx && live) {
      T* q = gx + row * a.gx_stride;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = rstd * (g[k][i] - s1 - h[k][i] * s2);
        if (lo[k] < VEC) store_pack<T, VEC>(q + start[k], o);
      }
    }
  }
  if (!part) return;
  // the work-group's rows' sums of each column: lanes of a wave first, then its waves through LDS
  part += (int64_t)blockIdx.x * 2 * d;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float v = stride_sum<(TPR < 64 ? TPR : 64)>(m == 0 ? dg[k][i] : db[k][i]);
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

// Rows longer than a work-group's registers hold: sweeps over the row, which stays in the L2.
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
  for (int64_t row = blockIdx.x; row < a.batch; row += gridDim.x) {
    const T* p = x + row * a.x_stride;
    T* q = y + row * a.y_stride;
    float f[VEC], sum = 0.f, sq = 0.f;
    int st, lo;
    for (int j = tid; j < nvec; j += kLong) {
      place<VEC>(j, d, st, lo);
      load_pack<T, VEC>(p + st, f);
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum += i >= lo ? f[i] : 0.f;
    }
    const float mean = group_sum(sum, s_red) / (float)d;
    for (int j = tid; j < nvec; j += kLong) {
      place<VEC>(j, d, st, lo);
      load_pack<T, VEC>(p + st, f);
#pragma unroll
      for (int i = 0; i < VEC; ++i) sq += i >= lo ? (f[i] - mean) * (f[i] - mean) : 0.f;
    }
    const float rstd = 1.0f / sqrtf(group_sum(sq, s_red) / (float)d + a.eps);
    // in place the vector that overlaps its neighbour must not read what that one wrote: the last
    // vector stores only its own elements, one by one
    for (int j = tid; j < nvec; j += kLong) {
      place<VEC>(j, d, st, lo);
      load_pack<T, VEC>(p + st, f);
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        f[i] = (gamma ? gamma[st + i] : 1.f) * ((f[i] - mean) * rstd) + (beta ? beta[st + i] : 0.f);
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
    float h[VEC], g[VEC], s1 = 0.f, s2 = 0.f;
    int st, lo;
    for (int j = tid; j < nvec; j += kLong) {
      place<VEC>(j, d, st, lo);
      load_pack<T, VEC>(p + st, h);
      load_pack<T, VEC>(r + st, g);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float v = g[i] * (gamma ? gamma[st + i] : 1.f);
        s1 += i >= lo ? v : 0.f;
        s2 += i >= lo ? v * ((h[i] - mean) * rstd) : 0.f;
      }
    }
    s1 = group_sum(s1, s_red) / (float)d;
    s2 = group_sum(s2, s_red) / (float)d;
    for (int j = tid; j < nvec; j += kLong) {
      place<VEC>(j, d, st, lo);
      load_pack<T, VEC>(p + st, h);
      load_pack<T, VEC>(r + st, g);
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        g[i] = rstd * (g[i] * (gamma ? gamma[st + i] : 1.f) - s1 - (h[i] - mean) * rstd * s2);
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
      part[d + i] = db[i];
    }
}

// ---- fields (npts > 1) -------------------------------------------------------------------------
// A work-group takes a tile of points, VEC to a lane, and its waves share the channels, N each, in
// registers; what a point's channels sum to joins through LDS.  FLAT: one point to a lane, counted
// through all batch entries (short entries); else tiles of 64 VEC points of one entry.
struct Tile {
  int64_t at;    // (batch, point) of the lane's first element, in rows
  int64_t b, p;
  int lo;        // the lane's own points are i >= lo
};

template <int VEC, bool FLAT>
__device__ __forceinline__ Tile tile_of(const NormArgs& a, int64_t tile, int64_t per_entry) {
  Tile t;
  const int lane = threadIdx.x & 63;
  if (FLAT) {
    const int64_t rows = a.batch * a.npts, r = tile * 64 + lane;
    t.at = r < rows ? r : rows - 1;
    t.lo = r < rows ? 0 : 1;
    if (rows <= 0x7fffffff) {
      const uint32_t b = (uint32_t)t.at / (uint32_t)a.npts;
      t.b = b;
      t.p = (uint32_t)t.at - b * (uint32_t)a.npts;
    } else {
      t.b = t.at / a.npts;
      t.p = t.at - t.b * a.npts;
    }
  } else {
    t.b = tile / per_entry;
    const int64_t e = (tile - t.b * per_entry) * (64 * VEC) + lane * VEC;
    t.p = e < a.npts - VEC ? e : a.npts - VEC;
    t.lo = e < a.npts ? (int)(e - t.p) : VEC;
    t.at = t.b * a.npts + t.p;
  }
  return t;
}

template <typename T, int VEC>
__device__ __forceinline__ void store_own(T* p, const float (&f)[VEC], int lo) {
  if (lo == 0) {
    store_pack<T, VEC>(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i >= lo) p[i] = from_float<T>(f[i]);
  }
}

template <typename T, int N, int VEC, bool FLAT>
__global__ __launch_bounds__(1024) void k_ln_fwd_field(NormArgs a, int64_t tiles,
                                                       int64_t per_entry, const T* x,
                                                       const float* gamma, const float* beta,
                                                       T* y, float* stats) {
  extern __shared__ float s_mem[];  // [2][waves][2][64 VEC]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), waves = blockDim.x / 64;
  const int c0 = wave * N, nc = a.channels - c0 < N ? a.channels - c0 : N;
  const float inv_c = 1.0f / (float)a.channels, inv_n = 1.0f / (float)nc;
  int flip = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, flip ^= 1) {
    const Tile t = tile_of<VEC, FLAT>(a, tile, per_entry);
    const T* p = x + t.b * a.x_stride + t.p;
    float f[N][VEC], mean[VEC], sq[VEC];
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const int ch = c < nc ? c0 + c : a.channels - 1;
      load_pack<T, VEC>(p + ch * a.npts, f[c]);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float s = 0.f, q = 0.f;
#pragma unroll
      for (int c = 0; c < N; ++c) s += c < nc ? f[c][i] : 0.f;
      mean[i] = s * inv_n;
#pragma unroll
      for (int c = 0; c < N; ++c) {
        const float e = f[c][i] - mean[i];
        q += c < nc ? e * e : 0.f;
      }
      sq[i] = q;
    }
    if (waves > 1) {
      float* s_t = s_mem + flip * waves * 2 * 64 * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        s_t[(wave * 2) * 64 * VEC + lane * VEC + i] = mean[i];
        s_t[(wave * 2 + 1) * 64 * VEC + lane * VEC + i] = sq[i];
      }
      __syncthreads();
      float all[VEC] = {};
      for (int w = 0; w < waves; ++w) {
        const float n = (float)(a.channels - w * N < N ? a.channels - w * N : N);
#pragma unroll
        for (int i = 0; i < VEC; ++i) all[i] += n * s_t[(w * 2) * 64 * VEC + lane * VEC + i];
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        mean[i] = all[i] * inv_c;
        sq[i] = 0.f;
      }
      for (int w = 0; w < waves; ++w) {
        const float n = (float)(a.channels - w * N < N ? a.channels - w * N : N);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float e = s_t[(w * 2) * 64 * VEC + lane * VEC + i] - mean[i];
          sq[i] += s_t[(w * 2 + 1) * 64 * VEC + lane * VEC + i] + n * e * e;
        }
      }
    }
    float rstd[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) rstd[i] = 1.0f / sqrtf(sq[i] * inv_c + a.eps);
    if (t.lo < VEC) {
      T* q = y + t.b * a.y_stride + t.p;
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (c < nc) {
          const float ga = gamma ? gamma[c0 + c] : 1.f, be = beta ? beta[c0 + c] : 0.f;
          float o[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) o[i] = ga * ((f[c][i] - mean[i]) * rstd[i]) + be;
          store_own<T, VEC>(q + (c0 + c) * a.npts, o, t.lo);
        }
      if (stats && wave == 0) {
        store_own<float, VEC>(stats + t.at, mean, t.lo);
        store_own<float, VEC>(stats + a.batch * a.npts + t.at, rstd, t.lo);
      }
    }
  }
}

template <typename T, int N, int VEC, bool FLAT>
__global__ __launch_bounds__(1024) void k_ln_bwd_field(NormArgs a, int64_t tiles,
                                                       int64_t per_entry, const T* x,
                                                       const float* gamma, const float* stats,
                                                       const T* gy, T* gx, float* part) {
  extern __shared__ float s_mem[];  // [2][waves][2][64 VEC]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), waves = blockDim.x / 64;
  const int c0 = wave * N, nc = a.channels - c0 < N ? a.channels - c0 : N;
  const float inv_c = 1.0f / (float)a.channels;
  float dg[N] = {}, db[N] = {};
  int flip = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, flip ^= 1) {
    const Tile t = tile_of<VEC, FLAT>(a, tile, per_entry);
    const T* p = x + t.b * a.x_stride + t.p;
    const T* r = gy + t.b * a.y_stride + t.p;
    float h[N][VEC], g[N][VEC], mean[VEC], rstd[VEC], s1[VEC] = {}, s2[VEC] = {};
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const int ch = c < nc ? c0 + c : a.channels - 1;
      load_pack<T, VEC>(p + ch * a.npts, h[c]);
      load_pack<T, VEC>(r + ch * a.npts, g[c]);
    }
    load_pack<float, VEC>(stats + t.at, mean);
    load_pack<float, VEC>(stats + a.batch * a.npts + t.at, rstd);
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const float ga = c < nc ? (gamma ? gamma[c0 + c] : 1.f) : 0.f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        h[c][i] = (h[c][i] - mean[i]) * rstd[i];
        if (i >= t.lo) {
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
      float* s_t = s_mem + flip * waves * 2 * 64 * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        s_t[(wave * 2) * 64 * VEC + lane * VEC + i] = s1[i];
        s_t[(wave * 2 + 1) * 64 * VEC + lane * VEC + i] = s2[i];
        s1[i] = s2[i] = 0.f;
      }
      __syncthreads();
      for (int w = 0; w < waves; ++w)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          s1[i] += s_t[(w * 2) * 64 * VEC + lane * VEC + i];
          s2[i] += s_t[(w * 2 + 1) * 64 * VEC + lane * VEC + i];
        }
    }
    if (gx && t.lo < VEC) {
      T* q = gx + t.b * a.gx_stride + t.p;
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (c < nc) {
          float o[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            o[i] = rstd[i] * (g[c][i] - s1[i] * inv_c - h[c][i] * (s2[i] * inv_c));
          store_own<T, VEC>(q + (c0 + c) * a.npts, o, t.lo);
        }
    }
  }
  if (!part) return;
  part += (int64_t)blockIdx.x * 2 * a.channels + c0;
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const float sg = lane_sum<64>(dg[c]), sb = lane_sum<64>(db[c]);
    if (lane == 0 && c < nc) {
      part[c] = sg;
      part[a.channels + c] = sb;
    }
  }
}

// Fields of more channels than a work-group holds: one thread to a point, sweeps over the channels.
template <typename T>
__global__ __launch_bounds__(256) void k_ln_fwd_points(NormArgs a, const T* x, const float* gamma,
                                                       const float* beta, T* y, float* stats) {
  const int64_t rows = a.batch * a.npts;
  for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < rows;
       r += (int64_t)gridDim.x * 256) {
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
__global__ __launch_bounds__(256) void k_ln_cols_points(NormArgs a, const T* x, const float* stats,
                                                        const T* gy, float* part) {
  __shared__ float s_red[2][4];
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
// COLS columns to a work-group, 256 / COLS threads down each.
template <int COLS>
__global__ __launch_bounds__(256) void k_ln_finish(int channels, int nparts, const float* part,
                                                   float* ggamma, float* gbeta) {
  constexpr int kSlices = 256 / COLS;
  __shared__ float s_red[kSlices][COLS];
  const int col = threadIdx.x % COLS, slice = threadIdx.x / COLS;
  const int64_t width = 2 * (int64_t)channels, i = (int64_t)blockIdx.x * COLS + col;
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

// Calls f(threads to a row, vectors to a thread) as constants, for rows of `nvec` vectors.
template <int N>
struct Int {
  static constexpr int value = N;
};
template <typename T, typename F>
void pick_rows(int channels, F&& f) {
  constexpr int VEC = kVec<T>;
  if (channels < VEC) return f(Int<1>(), Int<8>(), Int<1>());
  const int nvec = (channels + VEC - 1) / VEC;
  const Int<VEC> v;
  if (nvec <= 8) return f(v, Int<8>(), Int<1>());
  if (nvec <= 16) return f(v, Int<16>(), Int<1>());
  if (nvec <= 32) return f(v, Int<32>(), Int<1>());
  if (nvec <= 64) return f(v, Int<64>(), Int<1>());
  if (nvec <= 128) return f(v, Int<128>(), Int<1>());
  if (nvec <= 256) return f(v, Int<256>(), Int<1>());
  if (nvec <= 512) return f(v, Int<512>(), Int<1>());
  if (nvec <= 1024) return f(v, Int<1024>(), Int<1>());
  if (nvec <= 2048) return f(v, Int<1024>(), Int<2>());
  if constexpr (VEC == 4) return f(v, Int<1024>(), Int<4>());
}

constexpr int kBwdBlock = 1024;
template <int TPR>
int bwd_rows_groups(int64_t rows) {
  return (int)cut(ceil_div(rows, kBwdBlock / TPR), 256);
}

// fields: channels to a wave, and waves
#ifndef FN
#define FN 8
#endif
#ifndef BN
#define BN 8
#endif
#ifndef FV
#define FV 4
#endif
#ifndef BV
#define BV 2
#endif
#ifndef FG
#define FG (1<<20)
#endif
#ifndef BG
#define BG 4096
#endif
int field_n(int c, int most) {
  const int waves = (int)cut(ceil_div(c, most), 16), n = (int)ceil_div(c, waves);
  return n <= 8 ? n : n <= 12 ? 12 : 16;
}
template <typename F>
void pick_field(int n, F&& f) {
  switch (n) {
    case 1: return f(Int<1>());
    case 2: return f(Int<2>());
    case 3: return f(Int<3>());
    case 4: return f(Int<4>());
    case 5: return f(Int<5>());
    case 6: return f(Int<6>());
    case 7: return f(Int<7>());
    case 8: return f(Int<8>());
    case 12: return f(Int<12>());
    default: return f(Int<16>());
  }
}
struct FieldShape {
  bool flat;
  int n, waves;
  int64_t per_entry, tiles;
  size_t lds;
};
FieldShape field_shape(const NormArgs& a, int most, int wide) {
  FieldShape s;
  s.flat = a.npts < 512;
  const int vec = s.flat ? 1 : wide;
  s.n = field_n(a.channels, most);
  s.waves = (int)ceil_div(a.channels, s.n);
  s.per_entry = ceil_div(a.npts, 64 * vec);
  s.tiles = s.flat ? ceil_div(a.batch * a.npts, 64) : a.batch * s.per_entry;
  s.lds = s.waves > 1 ? sizeof(float) * 2 * s.waves * 2 * 64 * vec : 0;
  return s;
}
int field_bwd_groups(const FieldShape& s) { return (int)cut(s.tiles, ceil_div(BG, s.waves)); }

template <typename T>
hipError_t fwd_t(const NormArgs& a, const T* x, const float* gamma, const float* beta, T* y,
                 float* stats, hipStream_t s) {
  switch (form_of<T>(a)) {
    case kRows:
      pick_rows<T>(a.channels, [&](auto vec, auto tpr, auto nv) {
        constexpr int kBlock = tpr.value < 256 ? 256 : tpr.value;
        const int64_t groups = cut(ceil_div(a.batch, kBlock / tpr.value), 256 * 2048 / kBlock);
        hipLaunchKernelGGL((k_ln_fwd_rows<T, vec.value, tpr.value, nv.value, kBlock>),
                           dim3(groups), dim3(kBlock), 0, s, a, x, gamma, beta, y, stats);
      });
      break;
    case kLongRows:
      hipLaunchKernelGGL(k_ln_fwd_long<T>, dim3(cut(a.batch, 1024)), dim3(kLong), 0, s, a, x, gamma,
                         beta, y, stats);
      break;
    case kField: {
      const FieldShape f = field_shape(a, FN, FV);
      const dim3 grid(cut(f.tiles, FG)), block(64 * f.waves);
      pick_field(f.n, [&](auto n) {
        if (f.flat)
          hipLaunchKernelGGL((k_ln_fwd_field<T, n.value, 1, true>), grid, block, f.lds, s, a,
                             f.tiles, f.per_entry, x, gamma, beta, y, stats);
        else
          hipLaunchKernelGGL((k_ln_fwd_field<T, n.value, FV, false>), grid, block, f.lds, s,
                             a, f.tiles, f.per_entry, x, gamma, beta, y, stats);
      });
      break;
    }
    case kPoints:
      hipLaunchKernelGGL(k_ln_fwd_points<T>, dim3(cut(ceil_div(a.batch * a.npts, 256), 4096)),
                         dim3(256), 0, s, a, x, gamma, beta, y, stats);
  }
  return hipGetLastError();
}

template <typename T>
int parts_t(const NormArgs& a) {
  if (a.batch == 0 || a.npts == 0) return 0;
  switch (form_of<T>(a)) {
    case kRows: {
      int n = 0;
      pick_rows<T>(a.channels,
                   [&](auto, auto tpr, auto) { n = bwd_rows_groups<tpr.value>(a.batch); });
      return n;
    }
    case kField: return field_bwd_groups(field_shape(a, BN, BV));
    default: return (int)cut(a.npts == 1 ? a.batch : kPointParts, kPointParts);
  }
}

template <typename T>
hipError_t bwd_t(const NormArgs& a, const T* x, const float* gamma, const float* stats,
                 const T* gy, T* gx, float* part, hipStream_t s) {
  const int parts = parts_t<T>(a);
  switch (form_of<T>(a)) {
    case kRows:
      pick_rows<T>(a.channels, [&](auto vec, auto tpr, auto nv) {
        hipLaunchKernelGGL((k_ln_bwd_rows<T, vec.value, tpr.value, nv.value, kBwdBlock>),
                           dim3(parts), dim3(kBwdBlock), 0, s, a, x, gamma, stats, gy, gx, part);
      });
      break;
    case kField: {
      const FieldShape f = field_shape(a, BN, BV);
      const dim3 grid(parts), block(64 * f.waves);
      pick_field(f.n, [&](auto n) {
        if (f.flat)
          hipLaunchKernelGGL((k_ln_bwd_field<T, n.value, 1, true>), grid, block, f.lds, s, a,
                             f.tiles, f.per_entry, x, gamma, stats, gy, gx, part);
        else
          hipLaunchKernelGGL((k_ln_bwd_field<T, n.value, BV, false>), grid, block, f.lds, s,
                             a, f.tiles, f.per_entry, x, gamma, stats, gy, gx, part);
      });
      break;
    }
    // the column sums first: grad_x may overwrite x or grad_y
    case kLongRows:
      if (part)
        hipLaunchKernelGGL(k_ln_cols_long<T>, dim3(ceil_div(a.channels, 256 * kVec<T>), parts),
                           dim3(256), 0, s, a, x, stats, gy, part);
      if (gx)
        hipLaunchKernelGGL(k_ln_bwd_long<T>, dim3(cut(a.batch, 1024)), dim3(kLong), 0, s, a, x,
                           gamma, stats, gy, gx);
      break;
    case kPoints:
      if (part)
        hipLaunchKernelGGL(k_ln_cols_points<T>, dim3(parts, cut(a.channels, 32768)), dim3(256), 0,
                           s, a, x, stats, gy, part);
      if (gx)
        hipLaunchKernelGGL(k_ln_bwd_points<T>, dim3(cut(ceil_div(a.batch * a.npts, 256), 4096)),
                           dim3(256), 0, s, a, x, gamma, stats, gy, gx);
  }
  return hipGetLastError();
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
  return dtype == FNO_DTYPE_F32 ? parts_t<float>(a) : parts_t<__bf16>(a);
}

hipError_t launch_layer_norm_bwd(const NormArgs& a, int dtype, const void* x, const float* gamma,
                                 const float* stats, const void* gy, void* gx, float* part,
                                 hipStream_t s) {
  const auto go = [&](auto t) {
    typedef decltype(t) T;
    return bwd_t<T>(a, static_cast<const T*>(x), gamma, stats, static_cast<const T*>(gy),
                    static_cast<T*>(gx), part, s);
  };
  if (dtype == FNO_DTYPE_F32) return go(0.f);
  return dtype == FNO_DTYPE_BF16 ? go((__bf16)0.f) : go((_Float16)0.f);
}

hipError_t launch_layer_norm_finish(const NormArgs& a, int nparts, const float* part,
                                    float* ggamma, float* gbeta, hipStream_t s) {
  const int64_t width = 2 * (int64_t)a.channels;
  const auto go = [&](auto cols) {
    hipLaunchKernelGGL(k_ln_finish<cols.value>, dim3(ceil_div(width, cols.value)), dim3(256), 0, s,
                       a.channels, nparts, part, ggamma, gbeta);
    return hipGetLastError();
  };
  return width >= 8192 ? go(Int<64>()) : width >= 1024 ? go(Int<16>()) : go(Int<4>());
}

}  // namespace fno
