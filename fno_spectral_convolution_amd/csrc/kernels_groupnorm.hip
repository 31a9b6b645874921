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
// float32 in a fixed order.
#include <algorithm>

#include "dropout_device.h"
#include "pointwise.h"
#include "train_device.h"
#include "train_ops.h"

namespace fno {
namespace {

constexpr int kBlock = 256, kWaves = kBlock / 64;

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);  // elements of a 16-byte load

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

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
__device__ __forceinline__ float2 block_sum(float a, float b, float2* s) {
  a = lane_sum<64>(a);
  b = lane_sum<64>(b);
  if (threadIdx.x % 64 == 0) s[threadIdx.x / 64] = make_float2(a, b);
  __syncthreads();
  float2 t = s[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) {
    t.x += s[w].x;
    t.y += s[w].y;
  }
  return t;
}

// Count, mean, and the sum of squared deviations over the m entries of the whole group: a share of
// its variance, which stays in range where the sum by itself would pass float32's.
struct Moments {
  float n, mean, var;
};
__device__ __forceinline__ void join(Moments& a, float n, float mean, float var, float inv_m) {
  const float all = a.n + n, share = n > 0.f ? n * __builtin_amdgcn_rcpf(all) : 0.f;
  const float d = mean - a.mean;
  a.mean += d * share;
  a.var += var + (d * (share * (a.n * inv_m))) * d;
  a.n = all;
}
// All threads' moments, the same bits in every one.
__device__ __forceinline__ Moments block_moments(const Moments& m, float inv_m,
                                                 float2 (&s)[2][kWaves]) {
  const float2 t = block_sum(m.n, m.n * m.mean, s[0]);
  Moments r;
  r.n = t.x;
  r.mean = t.y / t.x;
  const float d = m.mean - r.mean;
  r.var = block_sum(m.n > 0.f ? m.var + (d * (m.n * inv_m)) * d : 0.f, 0.f, s[1]).x;
  return r;
}

// uniform 64-bit division, short where both fit 32 bits
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// ---- channels first --------------------------------------------------------------------------------
// A strip is what a work-group holds in registers at a time: K vectors a thread out of one group of an
// entry.  A plane (one channel's points) has nvec vectors, the last one moved back to end with it.
// Short planes: 2^tpp threads to a plane, kv vectors each, several planes to a strip.  Planes longer
// than a strip: the whole work-group on one plane, `strips` of them to the plane.
struct Strip {
  int64_t nvec, strips;   // vectors, strips of a plane (1: whole planes in a strip)
  int tpp, kv, planes;    // log2 of the threads to a plane, vectors of a thread in it, planes
  int cg, runs, parts;    // channels of a group, strips along them, partial sums of a plane
};
template <int VEC, int K>
Strip strip_of(const GroupArgs& a) {
  Strip p;
  p.cg = a.channels / a.groups;
  p.nvec = ceil_div(a.npts, VEC);
  p.tpp = 0;
  while (p.tpp < 8 && ((int64_t)1 << p.tpp) < p.nvec) ++p.tpp;
  const int64_t own = ceil_div(p.nvec, (int64_t)1 << p.tpp);
  if (own <= K) {
    p.kv = (int)own;
    p.planes = K / p.kv * (kBlock >> p.tpp);
    p.strips = p.parts = 1;
  } else {
    p.kv = K;
    p.planes = 1;
    p.strips = ceil_div(p.nvec, (int64_t)kBlock * K);
    // partial sums: enough work-groups for the card, and few enough for the next pass to join
    const int64_t want = ceil_div(4096, std::max<int64_t>(1, a.batch * a.channels));
    const int64_t most = std::max<int64_t>(1, 1024 / p.cg);
    p.parts = (int)std::min(p.strips, std::min(want, most));
  }
  p.runs = (int)ceil_div(p.cg, p.planes);
  return p;
}

// A thread's vectors of strip `s` of run `run`.
template <int VEC, int K>
struct Items {
  int channel[K];   // in its group
  int64_t start[K]; // element of the plane
  int lo[K];        // elements from here on are its own; VEC: none
  __device__ __forceinline__ void place(const Strip& p, int64_t npts, int run, int64_t s) {
    const int t = threadIdx.x & ((1 << p.tpp) - 1), slot = threadIdx.x >> p.tpp;
    const int slots = kBlock >> p.tpp;
    int pass = 0, j = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int row = pass * slots + slot;
      const int64_t v = s * kBlock * K + t + ((int64_t)j << p.tpp), at = v * VEC;
      channel[k] = run * p.planes + row;
      const bool there = row < p.planes && channel[k] < p.cg && v < p.nvec;
      start[k] = at < npts - VEC ? at : npts - VEC;
      lo[k] = there ? (int)(at - start[k]) : VEC;
      if (!there) channel[k] = 0, start[k] = 0;
      if (++j == p.kv) j = 0, ++pass;
    }
  }
};

// work item w of a launch -> entry, group, run, part
struct Place {
  int64_t b, bg, rest;
  int g, run;
};
__device__ __forceinline__ Place place_of(int64_t w, const Strip& p, int64_t per_run, int groups) {
  Place q;
  const int64_t lines = quotient(w, per_run);
  q.rest = w - lines * per_run;
  q.bg = quotient(lines, p.runs);
  q.run = (int)(lines - q.bg * p.runs);
  q.b = quotient(q.bg, groups);
  q.g = (int)(q.bg - q.b * groups);
  return q;
}

template <typename T, int VEC, int K>
__device__ __forceinline__ void load_items(const Items<VEC, K>& it, const T* x, int64_t npts,
                                           Raw<T, VEC> (&raw)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (it.lo[k] < VEC) raw[k] = load_raw<T, VEC>(x + it.channel[k] * npts + it.start[k]);
}

template <typename T, int VEC>
__device__ __forceinline__ void store_own(T* o, const float (&f)[VEC], int lo) {
  if (lo == 0) {
    store_pack<T, VEC>(o, f);
  } else {
#pragma unroll
    for (int e = 1; e < VEC; ++e)
      if (e >= lo) o[e] = from_float<T>(f[e]);
  }
}

// moments of a thread's vectors, one join for all
template <typename T, int VEC, int K>
__device__ __forceinline__ void add_moments(Moments& m, const Raw<T, VEC> (&raw)[K],
                                            const int (&lo)[K], float inv_m) {
  float n = 0.f, sum = 0.f, sq = 0.f, f[K][VEC];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    n += (float)(VEC - lo[k]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      f[k][e] = element<T, VEC>(raw[k], e);
      sum += e >= lo[k] ? f[k][e] : 0.f;
    }
  }
  if (n == 0.f) return;
  const float mean = sum * __builtin_amdgcn_rcpf(n);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float d = f[k][e] - mean;
      sq += e >= lo[k] ? d * d : 0.f;
    }
  join(m, n, mean, sq * inv_m, inv_m);
}

// parts of a group: float4 (its Moments, -), [batch * groups][runs * parts]
template <typename T, int VEC, int K>
__global__ __launch_bounds__(kBlock) void k_gn_stats(GroupArgs a, Strip p, int64_t total,
                                                     const T* x, float4* part) {
  __shared__ float2 s_red[2][kWaves];
  const float inv_m = 1.0f / ((float)p.cg * (float)a.npts);
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const Place q = place_of(w, p, p.parts, a.groups);
    const T* slab = x + q.b * a.x_stride + (int64_t)q.g * p.cg * a.npts;
    Moments m = {0.f, 0.f, 0.f};
    for (int64_t s = q.rest; s < p.strips; s += p.parts) {
      Items<VEC, K> it;
      it.place(p, a.npts, q.run, s);
      Raw<T, VEC> raw[K] = {};
      load_items<T, VEC, K>(it, slab, a.npts, raw);
      add_moments<T, VEC, K>(m, raw, it.lo, inv_m);
    }
    __syncthreads();
    m = block_moments(m, inv_m, s_red);
    if (threadIdx.x == 0) part[w] = make_float4(m.n, m.mean, m.var, 0.f);
  }
}

// A group's statistics from its `n` parts, in every thread.
__device__ __forceinline__ float2 group_stats(const float4* part, int n, float eps, float inv_m,
                                              float2 (&s)[2][kWaves]) {
  Moments m = {0.f, 0.f, 0.f};
  for (int i = threadIdx.x; i < n; i += kBlock) {
    const float4 v = part[i];
    join(m, v.x, v.y, v.z, inv_m);
  }
  __syncthreads();
  m = block_moments(m, inv_m, s);
  return make_float2(m.mean, rsqrtf(m.var + eps));
}

template <typename T, int VEC, int K>
__global__ __launch_bounds__(kBlock) void k_gn_apply(GroupArgs a, Strip p, int64_t total,
                                                     const T* x, const float* gamma,
                                                     const float* beta, const float4* part, T* y,
                                                     float* stats) {
  __shared__ float2 s_red[2][kWaves];
  const Dropper drop(a.drop);
  const bool aligned = a.npts % VEC == 0;
  const float inv_m = 1.0f / ((float)p.cg * (float)a.npts);
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const Place q = place_of(w, p, p.strips, a.groups);
    Items<VEC, K> it;
    it.place(p, a.npts, q.run, q.rest);
    Raw<T, VEC> raw[K] = {};
    const int64_t first = (int64_t)q.g * p.cg;  // channel
    load_items<T, VEC, K>(it, x + q.b * a.x_stride + first * a.npts, a.npts, raw);
    const int n = p.runs * p.parts;
    const float2 st = group_stats(part + q.bg * n, n, a.eps, inv_m, s_red);
    if (stats && threadIdx.x == 0 && q.run == 0 && q.rest == 0) {
      stats[q.bg] = st.x;
      stats[a.batch * a.groups + q.bg] = st.y;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (it.lo[k] >= VEC) continue;
      const int64_t c = first + it.channel[k];
      const float by = (gamma ? gamma[c] : 1.f) * st.y, at = beta ? beta[c] : 0.f;
      float f[VEC];
      unpack<T, VEC>(raw[k], f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = fmaf(f[e] - st.x, by, at);
      activate(f, a.act);
      if (a.drop.threshold)
        drop.apply<VEC>(f, (uint64_t)((q.b * a.channels + c) * a.npts + it.start[k]), aligned);
      store_own<T, VEC>(y + q.b * a.y_stride + c * a.npts + it.start[k], f, it.lo[k]);
    }
  }
}

// What both backward passes need of an element: h = (x - mu) r, g = act'(u) drop(grad_y).
template <typename T, int VEC>
__device__ __forceinline__ void backward_terms(const GroupArgs& a, const Dropper& drop,
                                               const Raw<T, VEC>& rx, const Raw<T, VEC>& rg,
                                               const float (&mu)[VEC], const float (&rs)[VEC],
                                               const float (&ga)[VEC], const float (&be)[VEC],
                                               uint64_t i, bool aligned, float (&h)[VEC],
                                               float (&g)[VEC]) {
  unpack<T, VEC>(rx, h);
  unpack<T, VEC>(rg, g);
#pragma unroll
  for (int e = 0; e < VEC; ++e) h[e] = (h[e] - mu[e]) * rs[e];
  if (a.drop.threshold) drop.apply<VEC>(g, i, aligned);
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

// sums of a plane's g h and g: rows [batch * parts] of [2][channels]
template <typename T, int VEC, int K>
__global__ __launch_bounds__(kBlock) void k_gn_sums(GroupArgs a, Strip p, int64_t total, const T* x,
                                                    const float* gamma, const float* beta,
                                                    const float* stats, const T* gy, float* part) {
  __shared__ float2 s_sum[K][kWaves];
  const Dropper drop(a.drop);
  const bool aligned = a.npts % VEC == 0;
  const int64_t sides = a.batch * a.groups;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const Place q = place_of(w, p, p.parts, a.groups);
    const int64_t first = (int64_t)q.g * p.cg;
    const float mean = stats[q.bg], rstd = stats[sides + q.bg];
    const T* xs = x + q.b * a.x_stride + first * a.npts;
    const T* gs = gy + q.b * a.y_stride + first * a.npts;
    float* row = part + (q.b * p.parts + q.rest) * 2 * a.channels;
    const int t = threadIdx.x & ((1 << p.tpp) - 1), slot = threadIdx.x >> p.tpp;
    const int lanes = 1 << (p.tpp < 6 ? p.tpp : 6);
    float mu[VEC], rs[VEC], ga[VEC], be[VEC];
    fill(mu, mean);
    fill(rs, rstd);
    float sg = 0.f, sb = 0.f;  // of the present plane
    // the lanes' sums of pass `i` over the planes
    const auto flush = [&](int i) {
      for (int m = 1; m < lanes; m <<= 1) {
        sg += __shfl_xor(sg, m);
        sb += __shfl_xor(sb, m);
      }
      const int c = q.run * p.planes + i * (kBlock >> p.tpp) + slot;
      if (p.tpp > 6) {
        if (threadIdx.x % 64 == 0) s_sum[i][threadIdx.x / 64] = make_float2(sg, sb);
      } else if (t == 0 && i * (kBlock >> p.tpp) + slot < p.planes && c < p.cg) {
        row[first + c] = sg;
        row[a.channels + first + c] = sb;
      }
      sg = sb = 0.f;
    };
    if (p.tpp > 6) __syncthreads();
    for (int64_t s = q.rest; s < p.strips; s += p.parts) {
      Items<VEC, K> it;
      it.place(p, a.npts, q.run, s);
      Raw<T, VEC> rx[K] = {}, rg[K] = {};
      load_items<T, VEC, K>(it, xs, a.npts, rx);
      load_items<T, VEC, K>(it, gs, a.npts, rg);
      int pass = 0, j = 0;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (it.lo[k] < VEC) {
          const int64_t c = first + it.channel[k];
          fill(ga, gamma ? gamma[c] : 1.f);
          fill(be, beta ? beta[c] : 0.f);
          float h[VEC], g[VEC];
          backward_terms<T, VEC>(a, drop, rx[k], rg[k], mu, rs, ga, be,
                                 (uint64_t)((q.b * a.channels + c) * a.npts + it.start[k]), aligned,
                                 h, g);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            sg += e >= it.lo[k] ? g[e] * h[e] : 0.f;
            sb += e >= it.lo[k] ? g[e] : 0.f;
          }
        }
        if (p.strips == 1 && ++j == p.kv) {
          flush(pass);
          j = 0;
          ++pass;
        }
      }
    }
    if (p.strips > 1) flush(0);
    if (p.tpp > 6) {  // 2 or 4 waves to a plane
      __syncthreads();
      const int waves = 1 << (p.tpp - 6), slots = kBlock >> p.tpp;
      if ((int)threadIdx.x < p.planes) {
        const int i = threadIdx.x / slots, sl = threadIdx.x % slots;
        const int c = q.run * p.planes + threadIdx.x;
        if (c < p.cg) {
          float2 v = s_sum[i][sl * waves];
          for (int u = 1; u < waves; ++u) {
            v.x += s_sum[i][sl * waves + u].x;
            v.y += s_sum[i][sl * waves + u].y;
          }
          row[first + c] = v.x;
          row[a.channels + first + c] = v.y;
        }
      }
    }
  }
}

template <typename T, int VEC, int K>
__global__ __launch_bounds__(kBlock) void k_gn_grad(GroupArgs a, Strip p, int64_t total, const T* x,
                                                    const float* gamma, const float* beta,
                                                    const float* stats, const T* gy,
                                                    const float* part, T* gx) {
  __shared__ float2 s_red[kWaves];
  const Dropper drop(a.drop);
  const bool aligned = a.npts % VEC == 0;
  const int64_t sides = a.batch * a.groups;
  const float inv_m = 1.0f / ((float)p.cg * (float)a.npts);
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const Place q = place_of(w, p, p.strips, a.groups);
    const int64_t first = (int64_t)q.g * p.cg;
    Items<VEC, K> it;
    it.place(p, a.npts, q.run, q.rest);
    Raw<T, VEC> rx[K] = {}, rg[K] = {};
    load_items<T, VEC, K>(it, x + q.b * a.x_stride + first * a.npts, a.npts, rx);
    load_items<T, VEC, K>(it, gy + q.b * a.y_stride + first * a.npts, a.npts, rg);
    const float mean = stats[q.bg], rstd = stats[sides + q.bg];
    float s1 = 0.f, s2 = 0.f;  // sums of gamma g, gamma g h
    const float* rows = part + q.b * p.parts * 2 * a.channels + first;
    for (int i = threadIdx.x; i < p.cg * p.parts; i += kBlock) {
      const int j = i / p.cg, c = i - j * p.cg;
      const float ga = gamma ? gamma[first + c] : 1.f;
      s2 += ga * rows[(int64_t)j * 2 * a.channels + c];
      s1 += ga * rows[((int64_t)j * 2 + 1) * a.channels + c];
    }
    __syncthreads();
    const float2 sum = block_sum(s1, s2, s_red);
    const float m1 = sum.x * inv_m, m2 = sum.y * inv_m;
    float mu[VEC], rs[VEC], ga[VEC], be[VEC];
    fill(mu, mean);
    fill(rs, rstd);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (it.lo[k] >= VEC) continue;
      const int64_t c = first + it.channel[k];
      fill(ga, gamma ? gamma[c] : 1.f);
      fill(be, beta ? beta[c] : 0.f);
      float h[VEC], g[VEC];
      backward_terms<T, VEC>(a, drop, rx[k], rg[k], mu, rs, ga, be,
                             (uint64_t)((q.b * a.channels + c) * a.npts + it.start[k]), aligned, h,
                             g);
#pragma unroll
      for (int e = 0; e < VEC; ++e) g[e] = rstd * fmaf(ga[e], g[e], -fmaf(h[e], m2, m1));
      store_own<T, VEC>(gx + q.b * a.gx_stride + c * a.npts + it.start[k], g, it.lo[k]);
    }
  }
}

// ---- channels last -------------------------------------------------------------------------------
// A row is one point's channels.  A work-group takes a block of `cols` channels (tc vectors) and a
// tile of rows, tr of them at a time: a thread keeps to its vector's channels.  The part of a group
// that lies in a block is a segment; group g and block k make segment g + k, so that a group's
// segments are neighbours (numbers that no pair has stay unused).
struct Tiles {
  int cols, blocks, tc, tr;  // channels of a block, blocks, vectors of a block, rows at a time
  int cg, tiles;             // channels of a group, tiles
  int64_t rows, segments;    // rows of a tile, segments
};
template <int VEC>
Tiles tiles_of(const GroupArgs& a, int least) {
  Tiles p;
  p.cg = a.channels / a.groups;
  const int64_t nvec = ceil_div(a.channels, VEC);
  p.blocks = (int)ceil_div(nvec, 32);
  p.tc = (int)ceil_div(nvec, p.blocks);
  p.cols = p.tc * VEC;
  p.blocks = (int)ceil_div(a.channels, p.cols);
  p.tr = kBlock / p.tc;
  p.segments = (int64_t)a.groups + p.blocks;
  // enough work-groups for the card, a tile of `least` rows for each thread at least, and few enough
  // tiles for the next pass to join
  const int64_t want = ceil_div(4096, std::max<int64_t>(1, a.batch * p.blocks));
  const int64_t in_block = std::min<int64_t>(p.cols, (p.cols + p.cg - 1) / p.cg + 1);
  const int64_t most = std::max<int64_t>(32, 8192 / in_block);
  const int64_t tiles =  // (rows of a tile fit 31 bits)
      std::max(ceil_div(a.npts, (int64_t)1 << 30),
               std::min(ceil_div(a.npts, (int64_t)p.tr * least), std::min(want, most)));
  p.rows = std::max<int64_t>(1, ceil_div(a.npts, tiles));
  p.tiles = (int)std::max<int64_t>(1, ceil_div(a.npts, p.rows));
  return p;
}

struct Block {
  int64_t b, row0;     // entry, first row
  int k, tile, rows;   // column block, tile, rows of it
  int c0, c1, g0, segs;  // channels, first group, groups that it touches
};
__device__ __forceinline__ Block block_of(int64_t w, const GroupArgs& a, const Tiles& p) {
  Block q;
  const int64_t rest = quotient(w, p.blocks);
  q.k = (int)(w - rest * p.blocks);
  q.b = quotient(rest, p.tiles);
  q.tile = (int)(rest - q.b * p.tiles);
  q.row0 = q.tile * p.rows;
  q.rows = (int)(p.rows < a.npts - q.row0 ? p.rows : a.npts - q.row0);
  q.c0 = q.k * p.cols;
  q.c1 = q.c0 + p.cols < a.channels ? q.c0 + p.cols : a.channels;
  q.g0 = q.c0 / p.cg;
  q.segs = (q.c1 - 1) / p.cg - q.g0 + 1;
  return q;
}
// A thread's vector in a block: its first channel, and its own elements (as Items).
template <int VEC>
__device__ __forceinline__ void vector_of(const Block& q, const Tiles& p, int channels, int& r,
                                          int& c, int& lo) {
  r = threadIdx.x / p.tc;
  const int at = q.c0 + (threadIdx.x - r * p.tc) * VEC;
  c = at < channels - VEC ? at : channels - VEC;
  lo = r < p.tr && at < channels ? at - c : VEC;
}

// Lanes to a segment: a power of two, so that the segments take the work-group between them.
__device__ __forceinline__ int lanes_of(int segs) {
  int l = 64;
  while (l > 1 && l * segs > kBlock) l >>= 1;
  return l;
}
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int m = 1; m < lanes; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// part [batch][segments][tiles]: mean, squared deviations over m
template <typename T, int VEC, int K>
__global__ __launch_bounds__(kBlock) void k_gn_stats_last(GroupArgs a, Tiles p, int64_t total,
                                                          const T* x, float2* part) {
  __shared__ float2 s_mom[kBlock * VEC];  // [tr][cols]
  const float inv_m = 1.0f / ((float)p.cg * (float)a.npts);
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const Block q = block_of(w, a, p);
    int r, c, lo;
    vector_of<VEC>(q, p, a.channels, r, c, lo);
    float n = 0.f, mean[VEC], sq[VEC];
    fill(mean, 0.f);
    fill(sq, 0.f);
    if (lo < VEC) {
      const T* base = x + q.b * a.x_stride + (q.row0 + r) * a.channels + c;
      const int64_t step = (int64_t)p.tr * a.channels;
      for (int i = r; i < q.rows; i += K * p.tr) {
        Raw<T, VEC> raw[K] = {};
        float count = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (i + k * p.tr < q.rows) {
            raw[k] = load_raw<T, VEC>(base + k * step);
            count += 1.f;
          }
        base += K * step;
        const float inv = __builtin_amdgcn_rcpf(count), all = n + count;
        const float share = count * __builtin_amdgcn_rcpf(all);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float s = 0.f, s2 = 0.f;
#pragma unroll
          for (int k = 0; k < K; ++k) s += element<T, VEC>(raw[k], e);  // 0 where there is no row
          const float m = s * inv;
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const float d = element<T, VEC>(raw[k], e) - m;
            s2 += i + k * p.tr < q.rows ? d * d : 0.f;
          }
          const float d = m - mean[e];
          mean[e] += d * share;
          sq[e] += s2 * inv_m + (d * (share * (n * inv_m))) * d;
        }
        n = all;
      }
    }
    __syncthreads();
    if (lo < VEC)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e >= lo) s_mom[r * p.cols + c + e - q.c0] = make_float2(mean[e], sq[e]);
    __syncthreads();
    const int lanes = lanes_of(q.segs), lane = threadIdx.x & (lanes - 1);
    for (int s = threadIdx.x / lanes; s < q.segs; s += kBlock / lanes) {
      const int g = q.g0 + s;
      const int from = max(q.c0, g * p.cg), width = min(q.c1, (g + 1) * p.cg) - from;
      const float2* mom = s_mom + from - q.c0;
      const float inv = 1.0f / ((float)q.rows * (float)width);
      // rows that slot r has seen
      const auto seen = [&](int r) { return (float)((q.rows - r + p.tr - 1) / p.tr); };
      const int slots = min(p.tr, q.rows);
      float sum = 0.f, sq2 = 0.f;
      for (int i = lane; i < slots * width; i += lanes) {
        const int r = i / width;
        sum += seen(r) * mom[r * p.cols + i - r * width].x;
      }
      const float m = lanes_sum(sum, lanes) * inv;
      for (int i = lane; i < slots * width; i += lanes) {
        const int r = i / width;
        const float2 v = mom[r * p.cols + i - r * width];
        sq2 += v.y + ((v.x - m) * (seen(r) * inv_m)) * (v.x - m);
      }
      sq2 = lanes_sum(sq2, lanes);
      if (lane == 0)
        part[(q.b * p.segments + g + q.k) * p.tiles + q.tile] = make_float2(m, sq2);
    }
  }
}

// The segments of group g: their number, and that of the first.
struct Segments {
  int blocks, first;
};
__device__ __forceinline__ Segments segments_of(const Tiles& p, int g) {
  const int k0 = g * p.cg / p.cols, k1 = (int)(((int64_t)(g + 1) * p.cg - 1) / p.cols);
  return {k1 - k0 + 1, k0};
}

// statistics of the groups that a block touches, into LDS
__device__ __forceinline__ void block_stats(const GroupArgs& a, const Tiles& p, const Block& q,
                                            const float2* part, float2* s_st) {
  const int lanes = lanes_of(q.segs), lane = threadIdx.x & (lanes - 1);
  const float inv = 1.0f / ((float)p.cg * (float)a.npts);
  for (int s = threadIdx.x / lanes; s < q.segs; s += kBlock / lanes) {
    const int g = q.g0 + s;
    const Segments sg = segments_of(p, g);
    const float2* from = part + (q.b * p.segments + g + sg.first) * p.tiles;
    const auto count = [&](int i, int k) {
      const int kk = sg.first + k;
      const int width = (int)(min((int64_t)(kk + 1) * p.cols, (int64_t)(g + 1) * p.cg) -
                              max((int64_t)kk * p.cols, (int64_t)g * p.cg));
      const int64_t row0 = (i - k * p.tiles) * p.rows;
      const int64_t rows = p.rows < a.npts - row0 ? p.rows : a.npts - row0;
      return (float)rows * (float)width;
    };
    float sum = 0.f, sq = 0.f;
    for (int i = lane; i < sg.blocks * p.tiles; i += lanes)
      sum += count(i, i / p.tiles) * from[i].x;
    const float m = lanes_sum(sum, lanes) * inv;
    for (int i = lane; i < sg.blocks * p.tiles; i += lanes) {
      const float2 v = from[i];
      sq += v.y + ((v.x - m) * (count(i, i / p.tiles) * inv)) * (v.x - m);
    }
    sq = lanes_sum(sq, lanes);
    if (lane == 0) s_st[s] = make_float2(m, rsqrtf(sq + a.eps));
  }
}

// a thread's channels' mean, r, gamma and beta
template <int VEC>
__device__ __forceinline__ void channel_terms(const Tiles& p, const Block& q, int c,
                                              const float* gamma, const float* beta,
                                              const float2* s_st, int lo, float (&mu)[VEC],
                                              float (&rs)[VEC], float (&ga)[VEC],
                                              float (&be)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    if (e < lo) {
      mu[e] = rs[e] = ga[e] = be[e] = 0.f;
      continue;
    }
    const float2 st = s_st[(c + e) / p.cg - q.g0];
    mu[e] = st.x;
    rs[e] = st.y;
    ga[e] = gamma ? gamma[c + e] : 1.f;
    be[e] = beta ? beta[c + e] : 0.f;
  }
}

template <typename T, int VEC, int K>
__global__ __launch_bounds__(kBlock) void k_gn_apply_last(GroupArgs a, Tiles p, int64_t total,
                                                          const T* x, const float* gamma,
                                                          const float* beta, const float2* part,
                                                          T* y, float* stats) {
  __shared__ float2 s_st[32 * VEC];
  const Dropper drop(a.drop);
  const bool aligned = a.channels % VEC == 0;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const Block q = block_of(w, a, p);
    int r, c, lo;
    vector_of<VEC>(q, p, a.channels, r, c, lo);
    __syncthreads();
    block_stats(a, p, q, part, s_st);
    __syncthreads();
    if (stats && q.tile == 0)
      for (int s = threadIdx.x; s < q.segs; s += kBlock)
        if ((q.g0 + s) * (int64_t)p.cg >= q.c0) {  // the block that has the group's first channel
          stats[q.b * a.groups + q.g0 + s] = s_st[s].x;
          stats[(a.batch + q.b) * a.groups + q.g0 + s] = s_st[s].y;
        }
    if (lo >= VEC) continue;
    float mu[VEC], by[VEC], ga[VEC], at[VEC];
    channel_terms<VEC>(p, q, c, gamma, beta, s_st, lo, mu, by, ga, at);
#pragma unroll
    for (int e = 0; e < VEC; ++e) by[e] *= ga[e];
    const T* from = x + q.b * a.x_stride + c;
    T* to = y + q.b * a.y_stride + c;
    for (int i = r; i < q.rows; i += K * p.tr) {
      Raw<T, VEC> raw[K];
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (i + k * p.tr < q.rows)
          raw[k] = load_raw<T, VEC>(from + (q.row0 + i + k * p.tr) * a.channels);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (i + k * p.tr >= q.rows) continue;
        const int64_t off = (q.row0 + i + k * p.tr) * a.channels;
        float f[VEC];
        unpack<T, VEC>(raw[k], f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = fmaf(f[e] - mu[e], by[e], at[e]);
        activate(f, a.act);
        if (a.drop.threshold)
          drop.apply<VEC>(f, (uint64_t)(q.b * a.npts * a.channels + off + c), aligned);
        store_own<T, VEC>(to + off, f, lo);
      }
    }
  }
}

// the statistics of the groups that a block touches, as the forward left them, into LDS
__device__ __forceinline__ void given_stats(const GroupArgs& a, const Block& q, const float* stats,
                                            float2* s_st) {
  for (int s = threadIdx.x; s < q.segs; s += kBlock)
    s_st[s] = make_float2(stats[q.b * a.groups + q.g0 + s],
                          stats[(a.batch + q.b) * a.groups + q.g0 + s]);
}

// part: rows [batch * tiles] of [2][channels], sums of g h and g; seg [batch][segments][tiles]: sums
// of gamma g h and gamma g
template <typename T, int VEC, int K>
__global__ __launch_bounds__(kBlock) void k_gn_sums_last(GroupArgs a, Tiles p, int64_t total,
                                                         const T* x, const float* gamma,
                                                         const float* beta, const float* stats,
                                                         const T* gy, float* part, float2* seg) {
  __shared__ float2 s_st[32 * VEC], s_sum[kBlock * VEC];
  const Dropper drop(a.drop);
  const bool aligned = a.channels % VEC == 0;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const Block q = block_of(w, a, p);
    int r, c, lo;
    vector_of<VEC>(q, p, a.channels, r, c, lo);
    __syncthreads();
    given_stats(a, q, stats, s_st);
    __syncthreads();
    float mu[VEC], rs[VEC], ga[VEC], be[VEC], sg[VEC], sb[VEC];
    fill(sg, 0.f);
    fill(sb, 0.f);
    if (lo < VEC) {
      channel_terms<VEC>(p, q, c, gamma, beta, s_st, lo, mu, rs, ga, be);
      const T* xs = x + q.b * a.x_stride + c;
      const T* gs = gy + q.b * a.y_stride + c;
      for (int i = r; i < q.rows; i += K * p.tr) {
        Raw<T, VEC> rx[K], rg[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (i + k * p.tr < q.rows) {
            const int64_t off = (q.row0 + i + k * p.tr) * a.channels;
            rx[k] = load_raw<T, VEC>(xs + off);
            rg[k] = load_raw<T, VEC>(gs + off);
          }
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (i + k * p.tr >= q.rows) continue;
          const int64_t off = (q.row0 + i + k * p.tr) * a.channels;
          float h[VEC], g[VEC];
          backward_terms<T, VEC>(a, drop, rx[k], rg[k], mu, rs, ga, be,
                                 (uint64_t)(q.b * a.npts * a.channels + off + c), aligned, h, g);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            sg[e] += g[e] * h[e];
            sb[e] += g[e];
          }
        }
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e >= lo) s_sum[r * p.cols + c + e - q.c0] = make_float2(sg[e], sb[e]);
    }
    __syncthreads();
    const int width = q.c1 - q.c0, slots = min(p.tr, q.rows);
    float* row = part + (q.b * p.tiles + q.tile) * 2 * a.channels + q.c0;
    for (int i = threadIdx.x; i < width; i += kBlock) {
      float2 v = s_sum[i];
      for (int k = 1; k < slots; ++k) {
        v.x += s_sum[k * p.cols + i].x;
        v.y += s_sum[k * p.cols + i].y;
      }
      row[i] = v.x;
      row[a.channels + i] = v.y;
      const float ga = gamma ? gamma[q.c0 + i] : 1.f;
      s_sum[i] = make_float2(ga * v.x, ga * v.y);
    }
    __syncthreads();
    const int lanes = lanes_of(q.segs), lane = threadIdx.x & (lanes - 1);
    for (int s = threadIdx.x / lanes; s < q.segs; s += kBlock / lanes) {
      const int g = q.g0 + s, to = min(q.c1, (g + 1) * p.cg);
      float u = 0.f, v = 0.f;
      for (int ch = max(q.c0, g * p.cg) + lane; ch < to; ch += lanes) {
        u += s_sum[ch - q.c0].x;
        v += s_sum[ch - q.c0].y;
      }
      u = lanes_sum(u, lanes);
      v = lanes_sum(v, lanes);
      if (lane == 0) seg[(q.b * p.segments + g + q.k) * p.tiles + q.tile] = make_float2(u, v);
    }
  }
}

template <typename T, int VEC, int K>
__global__ __launch_bounds__(kBlock) void k_gn_grad_last(GroupArgs a, Tiles p, int64_t total,
                                                         const T* x, const float* gamma,
                                                         const float* beta, const float* stats,
                                                         const T* gy, const float2* seg, T* gx) {
  __shared__ float2 s_st[32 * VEC], s_k[32 * VEC];
  const Dropper drop(a.drop);
  const bool aligned = a.channels % VEC == 0;
  const float inv = 1.0f / ((float)p.cg * (float)a.npts);
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const Block q = block_of(w, a, p);
    int r, c, lo;
    vector_of<VEC>(q, p, a.channels, r, c, lo);
    __syncthreads();
    given_stats(a, q, stats, s_st);
    const int lanes = lanes_of(q.segs), lane = threadIdx.x & (lanes - 1);
    for (int s = threadIdx.x / lanes; s < q.segs; s += kBlock / lanes) {
      const int g = q.g0 + s;
      const Segments sg = segments_of(p, g);
      const float2* from = seg + (q.b * p.segments + g + sg.first) * p.tiles;
      float u = 0.f, v = 0.f;
      for (int i = lane; i < sg.blocks * p.tiles; i += lanes) {
        u += from[i].x;
        v += from[i].y;
      }
      u = lanes_sum(u, lanes);
      v = lanes_sum(v, lanes);
      if (lane == 0) s_k[s] = make_float2(v * inv, u * inv);
    }
    __syncthreads();
    if (lo >= VEC) continue;
    float mu[VEC], rs[VEC], ga[VEC], be[VEC], m1[VEC], m2[VEC];
    channel_terms<VEC>(p, q, c, gamma, beta, s_st, lo, mu, rs, ga, be);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float2 v = s_k[e >= lo ? (c + e) / p.cg - q.g0 : 0];
      m1[e] = v.x;
      m2[e] = v.y;
    }
    const T* xs = x + q.b * a.x_stride + c;
    const T* gs = gy + q.b * a.y_stride + c;
    T* to = gx + q.b * a.gx_stride + c;
    for (int i = r; i < q.rows; i += K * p.tr) {
      Raw<T, VEC> rx[K], rg[K];
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (i + k * p.tr < q.rows) {
          const int64_t off = (q.row0 + i + k * p.tr) * a.channels;
          rx[k] = load_raw<T, VEC>(xs + off);
          rg[k] = load_raw<T, VEC>(gs + off);
        }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (i + k * p.tr >= q.rows) continue;
        const int64_t off = (q.row0 + i + k * p.tr) * a.channels;
        float h[VEC], g[VEC];
        backward_terms<T, VEC>(a, drop, rx[k], rg[k], mu, rs, ga, be,
                               (uint64_t)(q.b * a.npts * a.channels + off + c), aligned, h, g);
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[e] = rs[e] * fmaf(ga[e], g[e], -fmaf(h[e], m2[e], m1[e]));
        store_own<T, VEC>(to + off, g, lo);
      }
    }
  }
}

// ---- launches ------------------------------------------------------------------------------------
constexpr int kMaxGrid = 1 << 20;  // further work goes to the same work-groups
dim3 grid_of(int64_t total) { return dim3((unsigned)std::min<int64_t>(total, kMaxGrid)); }

template <int N>
struct Int {
  static constexpr int value = N;
};

// vectors of a thread at a time
template <typename T>
constexpr int kFwd = sizeof(T) == 4 ? 8 : 4;
constexpr int kBwd = 4;

// Rows as channels-last data of one point: a "field" of one point is the same memory.
bool by_rows(const GroupArgs& a) { return a.last || a.npts == 1; }
// elements that are neighbours in memory
int64_t run_of(const GroupArgs& a) { return by_rows(a) ? a.channels : a.npts; }
// Calls f(elements of a vector): single ones where runs are shorter than a 16-byte load.
template <typename T, typename F>
auto pick(const GroupArgs& a, F&& f) {
  if (run_of(a) < kVec<T>) return f(Int<1>());
  return f(Int<kVec<T>>());
}

size_t up(int64_t bytes) { return ((size_t)bytes + 255) / 256 * 256; }

template <typename T>
size_t fwd_bytes(const GroupArgs& a) {
  return pick<T>(a, [&](auto vec) {
    if (by_rows(a)) {
      const Tiles p = tiles_of<vec.value>(a, kFwd<T>);
      return up((int64_t)sizeof(float2) * a.batch * p.segments * p.tiles);
    }
    const Strip p = strip_of<vec.value, kFwd<T>>(a);
    return up((int64_t)sizeof(float4) * a.batch * a.groups * p.runs * p.parts);
  });
}

template <typename T>
hipError_t fwd(const GroupArgs& a, const T* x, const float* gamma, const float* beta, T* y,
               float* stats, void* ws, hipStream_t s) {
  constexpr int K = kFwd<T>;
  pick<T>(a, [&](auto vec) {
    constexpr int V = vec.value;
    if (by_rows(a)) {
      const Tiles p = tiles_of<V>(a, K);
      const int64_t total = a.batch * p.tiles * p.blocks;
      hipLaunchKernelGGL((k_gn_stats_last<T, V, K>), grid_of(total), dim3(kBlock), 0, s, a, p,
                         total, x, static_cast<float2*>(ws));
      hipLaunchKernelGGL((k_gn_apply_last<T, V, K>), grid_of(total), dim3(kBlock), 0, s, a, p,
                         total, x, gamma, beta, static_cast<const float2*>(ws), y, stats);
    } else {
      const Strip p = strip_of<V, K>(a);
      const int64_t lines = a.batch * a.groups * p.runs;
      hipLaunchKernelGGL((k_gn_stats<T, V, K>), grid_of(lines * p.parts), dim3(kBlock), 0, s, a, p,
                         lines * p.parts, x, static_cast<float4*>(ws));
      hipLaunchKernelGGL((k_gn_apply<T, V, K>), grid_of(lines * p.strips), dim3(kBlock), 0, s, a, p,
                         lines * p.strips, x, gamma, beta, static_cast<const float4*>(ws), y,
                         stats);
    }
  });
  return hipGetLastError();
}

constexpr int kLeastBwd = 16;  // rows of a tile to a thread: a tile's sums are written and read again

template <typename T>
size_t bwd_bytes(const GroupArgs& a) {
  return pick<T>(a, [&](auto vec) {
    if (by_rows(a)) {
      const Tiles p = tiles_of<vec.value>(a, kLeastBwd);
      return up((int64_t)sizeof(float) * 2 * a.batch * p.tiles * a.channels) +
             up((int64_t)sizeof(float2) * a.batch * p.segments * p.tiles);
    }
    const Strip p = strip_of<vec.value, kBwd>(a);
    return up((int64_t)sizeof(float) * 2 * a.batch * p.parts * a.channels);
  });
}

template <typename T>
hipError_t bwd(const GroupArgs& a, const T* x, const float* gamma, const float* beta,
               const float* stats, const T* gy, T* gx, float* ggamma, float* gbeta, void* ws,
               hipStream_t s) {
  constexpr int K = kBwd;
  float* part = static_cast<float*>(ws);
  int parts = 0;
  pick<T>(a, [&](auto vec) {
    constexpr int V = vec.value;
    if (by_rows(a)) {
      const Tiles p = tiles_of<V>(a, kLeastBwd);
      const int64_t total = a.batch * p.tiles * p.blocks;
      parts = (int)(a.batch * p.tiles);
      float2* seg = reinterpret_cast<float2*>(
          static_cast<char*>(ws) + up((int64_t)sizeof(float) * 2 * a.batch * p.tiles * a.channels));
      hipLaunchKernelGGL((k_gn_sums_last<T, V, K>), grid_of(total), dim3(kBlock), 0, s, a, p, total,
                         x, gamma, beta, stats, gy, part, seg);
      if (gx)
        hipLaunchKernelGGL((k_gn_grad_last<T, V, K>), grid_of(total), dim3(kBlock), 0, s, a, p,
                           total, x, gamma, beta, stats, gy, seg, gx);
    } else {
      const Strip p = strip_of<V, K>(a);
      const int64_t lines = a.batch * a.groups * p.runs;
      parts = (int)(a.batch * p.parts);
      hipLaunchKernelGGL((k_gn_sums<T, V, K>), grid_of(lines * p.parts), dim3(kBlock), 0, s, a, p,
                         lines * p.parts, x, gamma, beta, stats, gy, part);
      if (gx)
        hipLaunchKernelGGL((k_gn_grad<T, V, K>), grid_of(lines * p.strips), dim3(kBlock), 0, s, a,
                           p, lines * p.strips, x, gamma, beta, stats, gy, part, gx);
    }
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !(ggamma || gbeta)) return e;
  return launch_weight_sums(a.channels, parts, part, ggamma, gbeta, s);
}

template <typename F>
auto by_type(int dtype, F&& f) {
  if (dtype == FNO_DTYPE_F32) return f(0.f);
  return dtype == FNO_DTYPE_BF16 ? f((__bf16)0.f) : f((_Float16)0.f);
}
bool none(const GroupArgs& a) { return a.batch == 0 || a.npts == 0; }

}  // namespace

size_t group_norm_fwd_bytes(const GroupArgs& a, int dtype) {
  if (none(a)) return 0;
  return by_type(dtype, [&](auto t) { return fwd_bytes<decltype(t)>(a); });
}

hipError_t launch_group_norm_fwd(const GroupArgs& a, int dtype, const void* x, const float* gamma,
                                 const float* beta, void* y, float* stats, void* ws,
                                 hipStream_t s) {
  return by_type(dtype, [&](auto t) {
    typedef decltype(t) T;
    return fwd<T>(a, static_cast<const T*>(x), gamma, beta, static_cast<T*>(y), stats, ws, s);
  });
}

size_t group_norm_bwd_bytes(const GroupArgs& a, int dtype) {
  if (none(a)) return 0;
  return by_type(dtype, [&](auto t) { return bwd_bytes<decltype(t)>(a); });
}

hipError_t launch_group_norm_bwd(const GroupArgs& a, int dtype, const void* x, const float* gamma,
                                 const float* beta, const float* stats, const void* gy, void* gx,
                                 float* ggamma, float* gbeta, void* ws, hipStream_t s) {
  if (none(a)) return launch_weight_sums(a.channels, 0, nullptr, ggamma, gbeta, s);
  return by_type(dtype, [&](auto t) {
    typedef decltype(t) T;
    return bwd<T>(a, static_cast<const T*>(x), gamma, beta, stats, static_cast<const T*>(gy),
                  static_cast<T*>(gx), ggamma, gbeta, ws, s);
  });
}

}  // namespace fno
