// Group norm of fields [batch][channels][npts] and of rows of one point, and the choice between these
// and channels last.  groupnorm_device.h has the mathematics.
//
// Groups that a work-group's registers hold are read once and take one launch (k_gn_whole, k_gn_rows):
// 4 x 20 x 64^2 float32 with GELU 9.3 us, in which 16 groups keep 16 compute units busy; 8192 tokens of
// 4096 in 32 heads forward 45 us float32 (6.0 TB/s) and 31 bfloat16, backward bfloat16 43 and 5 for the
// weights' sums.  Larger groups are read twice, statistics first: work-groups that wait for each other
// within a launch could not share the card with a second call that does the same.  Both passes run at
// the memory's rate, which reads out of the 256 MB cache do not exceed: 8 x 64 x 512^2 float32 267 us
// forward (moments 91, output 195 traced one by one; 6.0 TB/s with the second reading), with GELU and
// dropout the same, although these keep the vector units over 80% busy in the output pass;
// 2 x 20 x 128^3 float32 with GELU backward 265 (102 and 161; 6.3 TB/s).  Half data with GELU and dropout
// are at the vector units' rate: 8 x 64 x 512^2 bfloat16 forward 165, without either 148; backward 305
// (some 41 instructions an element in each pass), with GELU alone 249, without either 212.
#include "groupnorm_device.h"

namespace fno {
namespace {

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);  // elements of a 16-byte load

// ---- channels first --------------------------------------------------------------------------------
// A strip is what a work-group holds in registers at a time: K vectors a thread out of one group of an
// entry.  A plane (one channel's points) has nvec vectors, the last one moved back to end with it.
// Short planes: 2^tpp threads to a plane, kv vectors each, several planes to a strip.  Planes longer
// than a strip: the whole work-group on one plane, `strips` of them to the plane.
struct Strip {
  int64_t strips;         // of a plane (1: whole planes in a strip)
  int tpp, kv, planes;    // log2 of the threads to a plane, vectors of a thread in it, planes
  int cg, runs, parts;    // channels of a group, strips along them, partial sums of a plane
  Divider by_parts, by_runs, by_groups;
  Scale scale;
};
template <int VEC, int K, int BLOCK>
Strip strip_of(const GroupArgs& a) {
  Strip p;
  p.cg = a.channels / a.groups;
  const int64_t nvec = ceil_div(a.npts, VEC);
  p.tpp = 0;
  while ((1 << p.tpp) < BLOCK && ((int64_t)1 << p.tpp) < nvec) ++p.tpp;
  const int64_t own = ceil_div(nvec, (int64_t)1 << p.tpp);
  if (own <= K) {
    p.kv = (int)own;
    p.planes = K / p.kv * (BLOCK >> p.tpp);
    p.strips = p.parts = 1;
  } else {
    p.kv = K;
    p.planes = 1;
    p.strips = ceil_div(nvec, (int64_t)BLOCK * K);
    // partial sums: enough work-groups for the card, and few enough for the next pass to join
    const int64_t want = ceil_div(8192, std::max<int64_t>(1, a.batch * a.channels));
    const int64_t most = std::max<int64_t>(1, 1024 / p.cg);
    p.parts = (int)std::min(p.strips, std::min(want, most));
  }
  p.runs = (int)ceil_div(p.cg, p.planes);
  p.by_parts = Divider(p.parts);
  p.by_runs = Divider(p.runs);
  p.by_groups = Divider(a.groups);
  p.scale = Scale(a);
  return p;
}

// Where a work item's strip begins: its entry, group and channels.
struct Place {
  int64_t b, bg, s;  // entry, entry and group, strip (or part) of the plane
  int run;
  int64_t channel;   // of its first plane, in the field
};
__device__ __forceinline__ Place place_of(int64_t w, const Strip& p, int groups) {
  Place q;
  const int64_t lines = p.by_parts.of(w);
  q.s = w - lines * p.parts;
  q.bg = p.by_runs.of(lines);
  q.run = (int)(lines - q.bg * p.runs);
  q.b = p.by_groups.of(q.bg);
  q.channel = (q.bg - q.b * groups) * p.cg + (int64_t)q.run * p.planes;
  return q;
}

// A thread's vectors of a strip of whole planes (p.strips = 1: a plane has no more points than a
// work-group holds).
template <int VEC, int K, int BLOCK>
struct Items {
  int row[K];  // plane, from the strip's first
  int off[K];  // element, from the strip's first
  int lo[K];   // elements from here on are its own; VEC: none
  __device__ __forceinline__ Items(const Strip& p, const Place& q, int64_t npts) {
    const int t = threadIdx.x & ((1 << p.tpp) - 1), slot = threadIdx.x >> p.tpp;
    const int slots = BLOCK >> p.tpp;
    const int planes = min(p.planes, p.cg - q.run * p.planes);
    const int points = (int)npts;
    int pass = 0, j = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int e = (t + (j << p.tpp)) * VEC, start = min(e, points - VEC);
      row[k] = pass * slots + slot;
      const bool there = row[k] < planes && e < points;
      lo[k] = there ? e - start : VEC;
      if (!there) row[k] = 0;
      off[k] = there ? row[k] * points + start : 0;
      if (++j == p.kv) j = 0, ++pass;
    }
  }
  // f(k, masked) for the vectors that are there; masked, a constant: whether a wave has vectors some
  // of whose elements are not its own (most have none, and are spared a select an element)
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
    bool partial = false;
#pragma unroll
    for (int k = 0; k < K; ++k) partial |= lo[k] > 0 && lo[k] < VEC;
    by_mask(__any(partial), [&](auto masked) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (lo[k] < VEC) f(k, masked);
    });
  }
  template <typename T>
  __device__ __forceinline__ void load(const T* strip, Raw<T, VEC> (&raw)[K]) const {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (lo[k] < VEC) raw[k] = load_raw<T, VEC>(strip + off[k]);
  }
};

// moments of a thread's vectors, one join for all
template <typename T, int VEC, int K>
__device__ __forceinline__ void add_moments(Moments& m, const Raw<T, VEC> (&raw)[K],
                                            const int (&lo)[K], float inv_m, const Scale& scale) {
  float n = 0.f, sum = 0.f, sq = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    n += (float)(VEC - lo[k]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum += e >= lo[k] ? element<T, VEC>(raw[k], e) : 0.f;
  }
  if (n == 0.f) return;
  const float mean = sum * __builtin_amdgcn_rcpf(n);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float d = scale.deviation(element<T, VEC>(raw[k], e), mean);
      sq += e >= lo[k] ? d * d : 0.f;
    }
  join(m, n, mean, sq * scale.up, inv_m);
}

// y of one vector: x from its group's mean and by = gamma r, at = beta; element i of the field
template <typename T, int VEC>
__device__ __forceinline__ void apply_vector(const GroupArgs& a, const Dropper& drop,
                                             const Raw<T, VEC>& raw, int lo, float mean, float by,
                                             float at, uint64_t i, T* o, bool stream) {
  const uint32_t mask = a.drop.threshold ? drop.mask<VEC>(i) : 0;
  float f[VEC];
  unpack<T, VEC>(raw, f);
#pragma unroll
  for (int e = 0; e < VEC; ++e) f[e] = fmaf(f[e] - mean, by, at);
  activate(f, a.act);
  if (a.drop.threshold) drop.apply<VEC>(f, mask);
  store_own<T, VEC>(o, f, lo, stream);
}

// Groups that one work-group holds whole: read once, written once, one launch.
template <typename T, int VEC, int K, int BLOCK>
__global__ __launch_bounds__(BLOCK) void k_gn_whole(GroupArgs a, Strip p, int64_t total, const T* x,
                                                    const float* gamma, const float* beta, T* y,
                                                    float* stats) {
  __shared__ float2 s_red[2][BLOCK / 64];
  const Dropper drop(a.drop);
  const Scale scale = p.scale;
  const float inv_m = scale.inv_m;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const Place q = place_of(w, p, a.groups);
    const Items<VEC, K, BLOCK> it(p, q, a.npts);
    Raw<T, VEC> raw[K] = {};
    it.load(x + q.b * a.x_stride + q.channel * a.npts, raw);
    float sum = 0.f;
    it.each([&](int k, auto masked) {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        sum += !masked.value || e >= it.lo[k] ? element<T, VEC>(raw[k], e) : 0.f;
    });
    if (BLOCK > 64) __syncthreads();
    const float mean = block_sum<BLOCK / 64>(sum, 0.f, s_red[0]).x * inv_m;
    float sq = 0.f;
    it.each([&](int k, auto masked) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = scale.deviation(element<T, VEC>(raw[k], e), mean);
        sq += !masked.value || e >= it.lo[k] ? d * d : 0.f;
      }
    });
    const float rstd = rsqrtf(block_sum<BLOCK / 64>(sq * scale.up, 0.f, s_red[1]).x + a.eps);
    if (stats && threadIdx.x == 0) {
      stats[q.bg] = mean;
      stats[a.batch * a.groups + q.bg] = rstd;
    }
    const uint64_t index = (uint64_t)((q.b * a.channels + q.channel) * a.npts);
    T* o = y + q.b * a.y_stride + q.channel * a.npts;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (it.lo[k] >= VEC) continue;
      const int64_t c = q.channel + it.row[k];
      apply_vector<T, VEC>(a, drop, raw[k], it.lo[k], mean, (gamma ? gamma[c] : 1.f) * rstd,
                           beta ? beta[c] : 0.f, index + it.off[k], o + it.off[k], false);
    }
  }
}

// Larger groups take two passes, a launch each.
struct Pass {
  Strip p;
  int64_t items;  // work items
  int joined;     // the first pass's parts of a group
  bool stream;    // the output goes past the caches
};

// Goes over the strips s, s + parts, ... of a plane of several: all(element of the thread's first
// vector) where a strip is whole, and one(element, lo) for each vector of the last one.
template <int VEC, int K, typename All, typename One>
__device__ __forceinline__ void long_strips(const Strip& p, int64_t s, int64_t npts, All&& all,
                                            One&& one) {
  constexpr int kStrip = kBlock * K * VEC;
  for (; s < p.strips; s += p.parts) {
    const int64_t at = s * kStrip + threadIdx.x * VEC;
    if ((s + 1) * kStrip <= npts) {
      all(at);
    } else {
#pragma unroll 1
      for (int k = 0; k < K; ++k) {
        const int64_t e = at + k * (kBlock * VEC), start = min(e, npts - VEC);
        if (e < npts) one(start, (int)(e - start));
      }
    }
  }
}

// K vectors of a strip, a work-group's width apart
template <typename T, int VEC, int K>
__device__ __forceinline__ void load_strip(const T* p, Raw<T, VEC> (&raw)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) raw[k] = load_raw<T, VEC, true>(p + k * (kBlock * VEC));
}

// parts of a group: float4 (its Moments, -), [batch * groups][runs * parts]
template <typename T, int VEC, int K, bool LONG>
__global__ __launch_bounds__(kBlock) void k_gn_stats(GroupArgs a, Pass ps, const T* x,
                                                     float4* part) {
  __shared__ float2 s_red[2][kWaves];
  const Strip& p = ps.p;
  const Scale scale = p.scale;
  const float inv_m = scale.inv_m;
  for (int64_t w = blockIdx.x; w < ps.items; w += gridDim.x) {
    const Place q = place_of(w, p, a.groups);
    const T* from = x + q.b * a.x_stride + q.channel * a.npts;
    Moments m = {0.f, 0.f, 0.f};
    if (LONG) {
      long_strips<VEC, K>(
          p, q.s, a.npts,
          [&](int64_t at) {
            constexpr int none[K] = {};
            Raw<T, VEC> raw[K];
            load_strip<T, VEC, K>(from + at, raw);
            add_moments<T, VEC, K>(m, raw, none, inv_m, scale);
          },
          [&](int64_t at, int lo) {
            const Raw<T, VEC> v[1] = {load_raw<T, VEC>(from + at)};
            const int own[1] = {lo};
            add_moments<T, VEC, 1>(m, v, own, inv_m, scale);
          });
    } else {
      const Items<VEC, K, kBlock> it(p, q, a.npts);
      Raw<T, VEC> raw[K] = {};
      it.load(from, raw);
      add_moments<T, VEC, K>(m, raw, it.lo, inv_m, scale);
    }
    m = block_moments<kWaves>(m, inv_m, s_red);
    if (threadIdx.x == 0) part[w] = make_float4(m.n, m.mean, m.var, 0.f);
  }
}

template <typename T, int VEC, int K, bool LONG>
__global__ __launch_bounds__(kBlock) void k_gn_apply(GroupArgs a, Pass ps, const T* x,
                                                     const float* gamma, const float* beta,
                                                     const float4* part, T* y, float* stats) {
  __shared__ float2 s_red[2][kWaves];
  const Strip& p = ps.p;
  const Dropper drop(a.drop);
  const float inv_m = p.scale.inv_m;
  const int n = ps.joined;
  for (int64_t w = blockIdx.x; w < ps.items; w += gridDim.x) {
    const Place q = place_of(w, p, a.groups);
    Moments m = {0.f, 0.f, 0.f};
    for (int i = threadIdx.x; i < n; i += kBlock) {
      const float4 v = part[q.bg * n + i];
      join(m, v.x, v.y, v.z, inv_m);
    }
    m = block_moments<kWaves>(m, inv_m, s_red);
    const float rstd = rsqrtf(m.var + a.eps);
    if (stats && threadIdx.x == 0 && q.run == 0 && q.s == 0) {
      stats[q.bg] = m.mean;
      stats[a.batch * a.groups + q.bg] = rstd;
    }
    const T* from = x + q.b * a.x_stride + q.channel * a.npts;
    T* to = y + q.b * a.y_stride + q.channel * a.npts;
    const uint64_t index = (uint64_t)((q.b * a.channels + q.channel) * a.npts);
    if (LONG) {
      const float by = (gamma ? gamma[q.channel] : 1.f) * rstd;
      const float be = beta ? beta[q.channel] : 0.f;
      long_strips<VEC, K>(
          p, q.s, a.npts,
          [&](int64_t at) {
            Raw<T, VEC> raw[K];
            load_strip<T, VEC, K>(from + at, raw);
#pragma unroll
            for (int k = 0; k < K; ++k) {
              const int64_t i = at + k * (kBlock * VEC);
              apply_vector<T, VEC>(a, drop, raw[k], 0, m.mean, by, be, index + i, to + i,
                                   ps.stream);
            }
          },
          [&](int64_t at, int lo) {
            apply_vector<T, VEC>(a, drop, load_raw<T, VEC>(from + at), lo, m.mean, by, be,
                                 index + at, to + at, false);
          });
    } else {
      const Items<VEC, K, kBlock> it(p, q, a.npts);
      Raw<T, VEC> raw[K] = {};
      it.load(from, raw);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (it.lo[k] >= VEC) continue;
        const int64_t c = q.channel + it.row[k];
        apply_vector<T, VEC>(a, drop, raw[k], it.lo[k], m.mean, (gamma ? gamma[c] : 1.f) * rstd,
                             beta ? beta[c] : 0.f, index + it.off[k], to + it.off[k], false);
      }
    }
  }
}

// h and g of one vector of a plane with the weights `weight` and `bias`; element i of the field
template <typename T, int VEC>
__device__ __forceinline__ void plane_terms(const GroupArgs& a, const Dropper& drop,
                                            const Raw<T, VEC>& rx, const Raw<T, VEC>& rg,
                                            float mean, float rstd, float weight, float bias,
                                            uint64_t i, float (&h)[VEC], float (&g)[VEC]) {
  float mu[VEC], rs[VEC], ga[VEC], be[VEC];
  fill(mu, mean);
  fill(rs, rstd);
  fill(ga, weight);
  fill(be, bias);
  const uint32_t mask = a.drop.threshold ? drop.mask<VEC>(i) : 0;
  backward_terms<T, VEC>(a, drop, rx, rg, mu, rs, ga, be, mask, h, g);
}
// grad_x of it, m1 and m2 the means of gamma g and gamma g h
template <typename T, int VEC>
__device__ __forceinline__ void plane_grad(float rstd, float weight, const float (&h)[VEC],
                                           float (&g)[VEC], float m1, float m2, T* o, int lo,
                                           bool stream) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) g[e] = rstd * fmaf(weight, g[e], -fmaf(h[e], m2, m1));
  store_own<T, VEC>(o, g, lo, stream);
}

// Sums of g h and g along planes: lanes that share a plane first, then its waves.
template <int K, int BLOCK>
struct PlaneSums {
  const Strip& p;
  const Place& q;
  float2 (&s)[K][BLOCK / 64];
  float *to_g, *to_b;        // [channels], nullable
  float sg = 0.f, sb = 0.f;  // of the present plane

  __device__ __forceinline__ void put(int c, float g, float b) const {
    if (to_g) to_g[q.channel + c] = g;
    if (to_b) to_b[q.channel + c] = b;
  }
  // the sums of pass `i` over the planes are complete in their threads
  __device__ __forceinline__ void flush(int i) {
    const int lanes = 1 << min(p.tpp, 6);
    sg = lanes_sum(sg, lanes);
    sb = lanes_sum(sb, lanes);
    const int c = i * (BLOCK >> p.tpp) + (threadIdx.x >> p.tpp);
    if (p.tpp > 6) {
      if (threadIdx.x % 64 == 0) s[i][threadIdx.x / 64] = make_float2(sg, sb);
    } else if ((threadIdx.x & (lanes - 1)) == 0 && c < p.planes && q.run * p.planes + c < p.cg) {
      put(c, sg, sb);
    }
    sg = sb = 0.f;
  }
  // the waves' parts of planes that several share; all threads, after the last flush
  __device__ __forceinline__ void finish() const {
    if (p.tpp <= 6) return;
    __syncthreads();
    const int waves = 1 << (p.tpp - 6), slots = BLOCK >> p.tpp, c = threadIdx.x;
    if (c < p.planes && q.run * p.planes + c < p.cg) {
      const int i = c / slots, first = (c - i * slots) * waves;
      float2 v = s[i][first];
      for (int u = 1; u < waves; ++u) {
        v.x += s[i][first + u].x;
        v.y += s[i][first + u].y;
      }
      put(c, v.x, v.y);
    }
    __syncthreads();
  }
};

// As k_gn_whole; to_g and to_b (nullable): sums of g h and g, an entry's `pitch` after the last one's.
template <typename T, int VEC, int K, int BLOCK>
__global__ __launch_bounds__(BLOCK) void k_gn_whole_bwd(GroupArgs a, Strip p, int64_t total,
                                                        const T* x, const float* gamma,
                                                        const float* beta, const float* stats,
                                                        const T* gy, T* gx, float* to_g,
                                                        float* to_b, int64_t pitch) {
  __shared__ float2 s_red[BLOCK / 64], s_sum[K][BLOCK / 64];
  const bool weights = to_g || to_b;
  const Dropper drop(a.drop);
  const int64_t sides = a.batch * a.groups;
  const float inv_m = p.scale.inv_m;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const Place q = place_of(w, p, a.groups);
    const Items<VEC, K, BLOCK> it(p, q, a.npts);
    Raw<T, VEC> rx[K] = {}, rg[K] = {};
    it.load(x + q.b * a.x_stride + q.channel * a.npts, rx);
    it.load(gy + q.b * a.y_stride + q.channel * a.npts, rg);
    const float mean = stats[q.bg], rstd = stats[sides + q.bg];
    const uint64_t index = (uint64_t)((q.b * a.channels + q.channel) * a.npts);
    PlaneSums<K, BLOCK> sums = {p, q, s_sum, to_g ? to_g + q.b * pitch : nullptr,
                                to_b ? to_b + q.b * pitch : nullptr};
    float h[K][VEC], g[K][VEC], weight[K], s1 = 0.f, s2 = 0.f;
    int pass = 0, j = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      weight[k] = 0.f;
      float pg = 0.f, pb = 0.f;
      if (it.lo[k] < VEC) {
        const int64_t c = q.channel + it.row[k];
        weight[k] = gamma ? gamma[c] : 1.f;
        plane_terms<T, VEC>(a, drop, rx[k], rg[k], mean, rstd, weight[k], beta ? beta[c] : 0.f,
                            index + it.off[k], h[k], g[k]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          pg += e >= it.lo[k] ? g[k][e] * h[k][e] : 0.f;
          pb += e >= it.lo[k] ? g[k][e] : 0.f;
        }
      }
      s1 += weight[k] * pb;
      s2 += weight[k] * pg;
      sums.sg += pg;
      sums.sb += pb;
      if (++j == p.kv) {
        if (weights) sums.flush(pass);
        j = 0;
        ++pass;
      }
    }
    if (weights) sums.finish();
    if (!gx) continue;
    if (BLOCK > 64) __syncthreads();
    const float2 sum = block_sum<BLOCK / 64>(s1, s2, s_red);
    T* to = gx + q.b * a.gx_stride + q.channel * a.npts;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (it.lo[k] < VEC)
        plane_grad<T, VEC>(rstd, weight[k], h[k], g[k], sum.x * inv_m, sum.y * inv_m,
                           to + it.off[k], it.lo[k], false);
  }
}

// A thread's shares of a group's sums of gamma g and gamma g h, from the partial rows.
struct Sums {
  int cg, parts;  // channels of a group, partial sums of a plane
  Divider by_cg;
  __device__ __forceinline__ float2 of(const GroupArgs& a, const float* part, const float* gamma,
                                       int64_t b, int64_t g) const {
    const int64_t first = g * cg;
    const float* rows = part + b * parts * 2 * a.channels + first;
    double u = 0.0, v = 0.0;  // (a wide group has many)
    for (int64_t k = threadIdx.x; k < (int64_t)cg * parts; k += kBlock) {
      const int64_t j = by_cg.of(k), c = k - j * cg;
      const float weight = gamma ? gamma[first + c] : 1.f;
      u += weight * rows[(j * 2 + 1) * a.channels + c];
      v += weight * rows[j * 2 * a.channels + c];
    }
    return make_float2((float)u, (float)v);
  }
};

// to [ceil(n / size)][2][channels]: sums of `size` neighbouring rows, kSumCols columns to a work-group
__global__ __launch_bounds__(kBlock) void k_gn_fold(int64_t width, int64_t n, int64_t size,
                                                    int64_t columns, int64_t total,
                                                    const float* part, float* to) {
  constexpr int kSlices = kBlock / kSumCols;
  __shared__ double s_col[kSlices][kSumCols];
  const int col = threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int64_t row = w / columns, i = (w - row * columns) * kSumCols + col;
    const int64_t end = (row + 1) * size < n ? (row + 1) * size : n;
    double s = 0.0;
    if (i < width)
#pragma unroll 8
      for (int64_t k = row * size + slice; k < end; k += kSlices) s += part[k * width + i];
    s_col[slice][col] = s;
    __syncthreads();
    if (slice == 0 && i < width) {
      for (int u = 1; u < kSlices; ++u) s += s_col[u][col];
      to[row * width + i] = (float)s;
    }
    __syncthreads();
  }
}
__global__ __launch_bounds__(kBlock) void k_gn_between(GroupArgs a, Between z, Sums sums,
                                                       const float* gamma) {
  between(a, z, [&](int64_t b, int g) { return sums.of(a, z.part, gamma, b, g); });
}

// part: rows [batch * parts] of [2][channels], sums of g h and g
template <typename T, int VEC, int K, bool LONG>
__global__ __launch_bounds__(kBlock) void k_gn_sums(GroupArgs a, Pass ps, const T* x,
                                                    const float* gamma, const float* beta,
                                                    const float* stats, const T* gy, float* part) {
  __shared__ float2 s_sum[K][kWaves];
  const Strip& p = ps.p;
  const Dropper drop(a.drop);
  for (int64_t w = blockIdx.x; w < ps.items; w += gridDim.x) {
    const Place q = place_of(w, p, a.groups);
    const float mean = stats[q.bg], rstd = stats[a.batch * a.groups + q.bg];
    const T* px = x + q.b * a.x_stride + q.channel * a.npts;
    const T* pg = gy + q.b * a.y_stride + q.channel * a.npts;
    const uint64_t index = (uint64_t)((q.b * a.channels + q.channel) * a.npts);
    float* row = part + (q.b * p.parts + q.s) * 2 * a.channels;
    PlaneSums<K, kBlock> sums = {p, q, s_sum, row, row + a.channels};
    if (LONG) {
      const float weight = gamma ? gamma[q.channel] : 1.f, bias = beta ? beta[q.channel] : 0.f;
      long_strips<VEC, K>(
          p, q.s, a.npts,
          [&](int64_t at) {
            Raw<T, VEC> rx[K], rg[K];
            load_strip<T, VEC, K>(px + at, rx);
            load_strip<T, VEC, K>(pg + at, rg);
            float sg = 0.f, sb = 0.f;  // of the strip: short chains
#pragma unroll
            for (int k = 0; k < K; ++k) {
              float h[VEC], g[VEC];
              plane_terms<T, VEC>(a, drop, rx[k], rg[k], mean, rstd, weight, bias,
                                  index + at + k * (kBlock * VEC), h, g);
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                sg += g[e] * h[e];
                sb += g[e];
              }
            }
            sums.sg += sg;
            sums.sb += sb;
          },
          [&](int64_t at, int lo) {
            float h[VEC], g[VEC];
            plane_terms<T, VEC>(a, drop, load_raw<T, VEC>(px + at), load_raw<T, VEC>(pg + at),
                                mean, rstd, weight, bias, index + at, h, g);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              sums.sg += e >= lo ? g[e] * h[e] : 0.f;
              sums.sb += e >= lo ? g[e] : 0.f;
            }
          });
      sums.flush(0);
    } else {
      const Items<VEC, K, kBlock> it(p, q, a.npts);
      Raw<T, VEC> rx[K] = {}, rg[K] = {};
      it.load(px, rx);
      it.load(pg, rg);
      int pass = 0, j = 0;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (it.lo[k] < VEC) {
          float h[VEC], g[VEC];
          const int64_t c = q.channel + it.row[k];
          plane_terms<T, VEC>(a, drop, rx[k], rg[k], mean, rstd, gamma ? gamma[c] : 1.f,
                              beta ? beta[c] : 0.f, index + it.off[k], h, g);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            sums.sg += e >= it.lo[k] ? g[e] * h[e] : 0.f;
            sums.sb += e >= it.lo[k] ? g[e] : 0.f;
          }
        }
        if (++j == p.kv) {
          sums.flush(pass);
          j = 0;
          ++pass;
        }
      }
    }
    sums.finish();
  }
}

template <typename T, int VEC, int K, bool LONG>
__global__ __launch_bounds__(kBlock) void k_gn_grad(GroupArgs a, Pass ps, const T* x,
                                                    const float* gamma, const float* beta,
                                                    const float* stats, const T* gy, Between z,
                                                    Sums sums, T* gx) {
  __shared__ float2 s_red[kWaves];
  const Strip& p = ps.p;
  const Dropper drop(a.drop);
  if (z.own && blockIdx.x >= z.groups) return weight_sums(a, z);
  const int64_t stride = z.own ? z.groups : gridDim.x;
  for (int64_t w = blockIdx.x; w < ps.items; w += stride) {
    const Place q = place_of(w, p, a.groups);
    const float mean = stats[q.bg], rstd = stats[a.batch * a.groups + q.bg];
    float2 m;
    if (z.own) {
      const float2 v = sums.of(a, z.part, gamma, q.b, q.bg - q.b * a.groups);
      __syncthreads();
      m = block_sum<kWaves>(v.x, v.y, s_red);
      const float inv = p.scale.inv_m;
      m = make_float2(m.x * inv, m.y * inv);
    } else {
      m = z.means[q.bg];
    }
    const float m1 = m.x, m2 = m.y;
    const T* px = x + q.b * a.x_stride + q.channel * a.npts;
    const T* pg = gy + q.b * a.y_stride + q.channel * a.npts;
    T* to = gx + q.b * a.gx_stride + q.channel * a.npts;
    const uint64_t index = (uint64_t)((q.b * a.channels + q.channel) * a.npts);
    if (LONG) {
      const float weight = gamma ? gamma[q.channel] : 1.f, bias = beta ? beta[q.channel] : 0.f;
      long_strips<VEC, K>(
          p, q.s, a.npts,
          [&](int64_t at) {
            Raw<T, VEC> rx[K], rg[K];
            load_strip<T, VEC, K>(px + at, rx);
            load_strip<T, VEC, K>(pg + at, rg);
#pragma unroll
            for (int k = 0; k < K; ++k) {
              float h[VEC], g[VEC];
              const int64_t i = at + k * (kBlock * VEC);
              plane_terms<T, VEC>(a, drop, rx[k], rg[k], mean, rstd, weight, bias, index + i, h, g);
              plane_grad<T, VEC>(rstd, weight, h, g, m1, m2, to + i, 0, ps.stream);
            }
          },
          [&](int64_t at, int lo) {
            float h[VEC], g[VEC];
            plane_terms<T, VEC>(a, drop, load_raw<T, VEC>(px + at), load_raw<T, VEC>(pg + at), mean,
                                rstd, weight, bias, index + at, h, g);
            plane_grad<T, VEC>(rstd, weight, h, g, m1, m2, to + at, lo, false);
          });
    } else {
      const Items<VEC, K, kBlock> it(p, q, a.npts);
      Raw<T, VEC> rx[K] = {}, rg[K] = {};
      it.load(px, rx);
      it.load(pg, rg);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (it.lo[k] >= VEC) continue;
        float h[VEC], g[VEC];
        const int64_t c = q.channel + it.row[k];
        const float weight = gamma ? gamma[c] : 1.f;
        plane_terms<T, VEC>(a, drop, rx[k], rg[k], mean, rstd, weight, beta ? beta[c] : 0.f,
                            index + it.off[k], h, g);
        plane_grad<T, VEC>(rstd, weight, h, g, m1, m2, to + it.off[k], it.lo[k], false);
      }
    }
  }
}

// ---- rows: one point ------------------------------------------------------------------------------
// A group is `cg` neighbours: TPR threads hold it, NV vectors each, the last one moved back to end
// with the group; the elements that it then shares with its neighbour (i < lo) count once, and are
// stored twice with the same value.  A slot (TPR threads) keeps to one group of the channels, so that
// its weights stay in registers, and goes down the batch.
template <int VEC>
__device__ __forceinline__ void place(int j, int d, int& start, int& lo) {
  const int e = j * VEC;
  start = e < d - VEC ? e : d - VEC;
  lo = e < d ? e - start : VEC;
}

// Whether any lane of the wave has elements that are not its own.
template <int NV>
__device__ __forceinline__ bool any_partial(const int (&lo)[NV]) {
  bool partial = false;
#pragma unroll
  for (int k = 0; k < NV; ++k) partial |= lo[k] != 0;
  return __any(partial);
}

// Sum over a slot's threads, in all of them.  Slots of several waves go through `s`, whose two halves
// are taken in turn: one barrier a sum.
template <int TPR, int BLOCK>
__device__ __forceinline__ float slot_sum(float v, float (&s)[2][BLOCK / 64], int& flip) {
  if (TPR <= 64) return lane_sum<TPR>(v);
  v = lane_sum<64>(v);
  if (threadIdx.x % 64 == 0) s[flip][threadIdx.x / 64] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < TPR / 64; ++w) v += s[flip][threadIdx.x / TPR * (TPR / 64) + w];
  flip ^= 1;
  return v;
}

// `stride` slots in the launch: a multiple of the groups, `rows` times as many
template <typename T, int VEC, int TPR, int NV, int BLOCK>
__global__ __launch_bounds__(BLOCK) void k_gn_rows(GroupArgs a, int cg, Divider by_groups,
                                                   Scale scale, int64_t stride, int64_t rows, bool stream,
                                                   const T* x,
                                                   const float* gamma, const float* beta, T* y,
                                                   float* stats) {
  constexpr int kSlots = BLOCK / TPR;
  __shared__ float s_sum[2][BLOCK / 64];
  const Dropper drop(a.drop);
  const int t = threadIdx.x % TPR;
  const float inv = scale.inv_m;
  const int64_t total = a.batch * a.groups, slot = (int64_t)blockIdx.x * kSlots + threadIdx.x / TPR;
  const int64_t row0 = by_groups.of(slot);
  const int group = (int)(slot - row0 * a.groups), first = group * cg;
  int start[NV], lo[NV];
  float ga[NV][VEC], be[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    place<VEC>(k * TPR + t, cg, start[k], lo[k]);
    start[k] += first;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      ga[k][e] = gamma ? gamma[start[k] + e] : 1.f;
      be[k][e] = beta ? beta[start[k] + e] : 0.f;
    }
  }
  const bool partial = any_partial(lo);
  int flip = 0;
  // every thread of the work-group goes round as often as the first slot, for the barriers; the next
  // row's loads go ahead of this one's sums
  int64_t b = row0;
  Raw<T, VEC> next[NV];
  const auto fetch = [&](int64_t row) {
    const T* p = x + (row < a.batch ? row : a.batch - 1) * a.x_stride;
#pragma unroll
    for (int k = 0; k < NV; ++k) next[k] = load_raw<T, VEC, true>(p + start[k]);
  };
  fetch(b);
  for (int64_t at = (int64_t)blockIdx.x * kSlots; at < total; at += stride, b += rows) {
    const bool live = b < a.batch;
    float f[NV][VEC], sum = 0.f, sq = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) unpack<T, VEC>(next[k], f[k]);
    if (at + stride < total) fetch(b + rows);
    by_mask(partial, [&](auto masked) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum += !masked.value || e >= lo[k] ? f[k][e] : 0.f;
    });
    const float mean = slot_sum<TPR, BLOCK>(sum, s_sum, flip) * inv;
    by_mask(partial, [&](auto masked) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          f[k][e] = scale.deviation(f[k][e], mean);
          sq += !masked.value || e >= lo[k] ? f[k][e] * f[k][e] : 0.f;
        }
    });
    const float rstd = rsqrtf(slot_sum<TPR, BLOCK>(sq * scale.up, s_sum, flip) + a.eps);
    if (!live) continue;
    const float by = rstd * scale.back;
    T* o = y + b * a.y_stride;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (lo[k] >= VEC) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[k][e] = fmaf(f[k][e] * by, ga[k][e], be[k][e]);
      activate(f[k], a.act);
      if (a.drop.threshold)
        drop.apply<VEC>(f[k], drop.mask<VEC>((uint64_t)(b * a.channels + start[k])));
      store_pack<T, VEC>(o + start[k], f[k], stream);
    }
    if (stats && t == 0) {
      const int64_t i = b * a.groups + group;
      stats[i] = mean;
      stats[total + i] = rstd;
    }
  }
}

// A work-group takes `wide` groups (chunk blockIdx.x % chunks of them) of `deep` rows at a time.
// Their weights' sums stay in registers until its last row and go out to to_g and to_b (nullable),
// those of work-group blockIdx.x / chunks `pitch` after the last one's.
template <typename T, int VEC, int TPR, int NV, int BLOCK, bool WEIGHTS>
__global__ __launch_bounds__(BLOCK) void k_gn_rows_bwd(GroupArgs a, int cg, Divider by_wide,
                                                       int wide, int deep, int chunks, bool stream,
                                                       const T* x, const float* gamma,
                                                       const float* beta, const float* stats,
                                                       const T* gy, T* gx, float* to_g,
                                                       float* to_b, int64_t pitch) {
  constexpr int kCols = TPR * VEC;
  __shared__ float s_sum[2][BLOCK / 64];
  __shared__ float s_cols[WEIGHTS ? BLOCK * VEC : 1];
  const Dropper drop(a.drop);
  const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const float inv = 1.0f / (float)cg;
  const int64_t total = a.batch * a.groups;
  const int chunk = blockIdx.x % chunks, g0 = chunk * wide;
  const int here = min(wide, a.groups - g0), down = by_wide.of((uint32_t)slot), across = slot - down * wide;
  const bool mine = down < deep && across < here;
  const int g = mine ? g0 + across : g0;
  int start[NV], lo[NV];
  float ga[NV][VEC], be[NV][VEC], dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    place<VEC>(k * TPR + t, cg, start[k], lo[k]);
    start[k] += g * cg;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      ga[k][e] = gamma ? gamma[start[k] + e] : 1.f;
      be[k][e] = beta ? beta[start[k] + e] : 0.f;
      dg[k][e] = db[k][e] = 0.f;
    }
  }
  const bool partial = any_partial(lo);
  int flip = 0;
  const int64_t step = (int64_t)(gridDim.x / chunks) * deep;
  // the next row's loads go ahead of this one's sums
  Raw<T, VEC> next_x[NV], next_g[NV];
  float next_mean, next_rstd;
  const auto fetch = [&](int64_t row) {
    const int64_t b = mine && row < a.batch ? row : a.batch - 1;
    next_mean = stats[b * a.groups + g];
    next_rstd = stats[total + b * a.groups + g];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      next_x[k] = load_raw<T, VEC, true>(x + b * a.x_stride + start[k]);
      next_g[k] = load_raw<T, VEC, true>(gy + b * a.y_stride + start[k]);
    }
  };
  int64_t base = (int64_t)(blockIdx.x / chunks) * deep;
  if (base < a.batch) fetch(base + down);
  for (; base < a.batch; base += step) {
    const bool live = mine && base + down < a.batch;
    const int64_t b = live ? base + down : a.batch - 1;
    const float mean = next_mean, rstd = next_rstd;
    float h[NV][VEC], v[NV][VEC], s1 = 0.f, s2 = 0.f;
    Raw<T, VEC> rx[NV], rg[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      rx[k] = next_x[k];
      rg[k] = next_g[k];
    }
    if (base + step < a.batch) fetch(base + step + down);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float mu[VEC], rs[VEC];
      fill(mu, mean);
      fill(rs, rstd);
      const uint32_t mask =
          a.drop.threshold ? drop.mask<VEC>((uint64_t)(b * a.channels + start[k])) : 0;
      backward_terms<T, VEC>(a, drop, rx[k], rg[k], mu, rs, ga[k], be[k], mask, h[k], v[k]);
      if (WEIGHTS && live) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          dg[k][e] += v[k][e] * h[k][e];
          db[k][e] += v[k][e];
        }
      }
    }
    by_mask(partial, [&](auto masked) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          v[k][e] *= ga[k][e];
          s1 += !masked.value || e >= lo[k] ? v[k][e] : 0.f;
          s2 += !masked.value || e >= lo[k] ? v[k][e] * h[k][e] : 0.f;
        }
    });
    s1 = slot_sum<TPR, BLOCK>(s1, s_sum, flip) * inv;
    s2 = slot_sum<TPR, BLOCK>(s2, s_sum, flip) * inv;
    if (!gx || !live) continue;
    T* o = gx + b * a.gx_stride;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (lo[k] >= VEC) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[k][e] = rstd * (v[k][e] - fmaf(h[k][e], s2, s1));
      store_pack<T, VEC>(o + start[k], v[k], stream);
    }
  }
  if (!WEIGHTS) return;
  // the slots' sums of each column, down their rows
  const int64_t first = (int64_t)(blockIdx.x / chunks) * pitch + (int64_t)g0 * cg;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float* to = m == 0 ? to_g : to_b;
      if (!to) continue;
      __syncthreads();
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        s_cols[threadIdx.x * VEC + e] = m == 0 ? dg[k][e] : db[k][e];
      __syncthreads();
      for (int c = threadIdx.x; c < here * kCols; c += BLOCK) {
        const int i = c / kCols, r = c - i * kCols;
        int st, low;
        place<VEC>(k * TPR + r / VEC, cg, st, low);
        if (r % VEC < low) continue;
        float sum = 0.f;
        for (int d = 0; d < deep; ++d) sum += s_cols[d * wide * kCols + c];
        to[first + i * cg + st + r % VEC] = sum;
      }
    }
}

// ---- launches ------------------------------------------------------------------------------------
// vectors of a thread at a time
constexpr int kAhead = 4;
template <int VEC>
constexpr int kWhole = VEC == 1 ? 4 : 32 / VEC;     // 32 elements (single ones: planes of few points)
template <int VEC>
constexpr int kWholeBwd = VEC == 1 ? 4 : 16 / VEC;  // 16, whose h and g stay in registers

// Which kernels: rows of one point whose groups a work-group's registers hold, channels last (and
// longer rows, the same memory), channels first.
constexpr int kMostRow = 8192;  // 1024 threads with 8 elements each
enum Form { kRows, kLast, kFirst };
Form form_of(const GroupArgs& a) {
  if (a.npts == 1 && a.channels / a.groups <= kMostRow && a.groups <= 1 << 20) return kRows;
  return a.last || a.npts == 1 ? kLast : kFirst;
}

// Calls f(threads to a group, vectors to a thread) for rows.
template <int VEC, typename F>
auto pick_rows(int cg, F&& f) {
  constexpr int N = 8 / VEC;
  const int nvec = (cg + VEC - 1) / VEC;
  if (VEC == 1 || nvec <= 8) return f(Int<8>(), Int<1>());
  if constexpr (VEC > 1) {
    if (nvec <= 16) return f(Int<16>(), Int<1>());
    if (nvec <= 32) return f(Int<32>(), Int<1>());
    if (nvec <= 64) return f(Int<64>(), Int<1>());
    if (nvec <= 64 * N) return f(Int<64>(), Int<N>());
    if (nvec <= 256 * N) return f(Int<256>(), Int<N>());
    return f(Int<1024>(), Int<N>());
  }
}

// The backward's rows: groups and rows that a work-group takes at a time (as many of its slots as
// can be used, rather more groups, which are neighbours), and its work-groups down the batch, which
// write one partial row each.  One goes down up to four times: it then has the gradients themselves,
// which spares the workspace and a launch (3.3 us for the host).  No more than 128 times where it does
// not: a thread's sums are float32 chains of as many terms.
constexpr int kRowsBlock = 1024;
constexpr int64_t kRowsDown = 128;
struct RowsShape {
  int wide, deep, chunks, down;
};
RowsShape rows_shape(const GroupArgs& a, int tpr) {
  const int slots = kRowsBlock / tpr;
  RowsShape p = {1, 1, a.groups, 1};
  double best = 0;
  for (int w = (int)std::min<int64_t>(a.groups, slots); w >= 1 && best < 0.9; --w) {
    const int chunks = (int)ceil_div(a.groups, w), deep = slots / w;
    const double used = (double)deep * w / slots * a.groups / ((double)chunks * w);
    if (used > best + 0.02) {
      best = used;
      p.wide = w;
      p.deep = deep;
      p.chunks = chunks;
    }
  }
  const int64_t times = ceil_div(a.batch, p.deep);
  const int64_t down = std::max<int64_t>(std::max(1, 256 / p.chunks),
                                         std::min(ceil_div(times, kRowsDown), (1 << 21) / (int64_t)p.chunks));
  p.down = times <= 4 ? 1 : (int)std::min(times, down);
  return p;
}

// Fields: calls f(threads, strip) where a work-group of 64, 256 or 1024 threads holds a group whole,
// the smallest that does; says whether one does.
template <int VEC, int K, typename F>
bool pick_whole(const GroupArgs& a, F&& f) {
  const auto go = [&](auto block) {
    const Strip p = strip_of<VEC, K, block.value>(a);
    if (p.strips > 1 || p.runs > 1) return false;
    f(block, p);
    return true;
  };
  return go(Int<64>()) || go(Int<256>()) || go(Int<1024>());
}

template <typename T>
Pass pass_of(const GroupArgs& a, const Strip& p) {
  return {p, a.batch * a.groups * p.runs * p.parts, p.runs * p.parts, stream_out<T>(a)};
}
// The second pass, with about `strips` strips to a work item: short items run faster than a work-group
// that goes on from strip to strip (2 x 20 x 128^3 float32 backward, which has nothing to join, 264 us
// with one, 269 with two, 310 with as many as the first pass has; 8 x 64 x 512^2 float32 forward 279,
// 264 and 302).
template <typename T>
Pass second_of(const GroupArgs& a, const Strip& p, int strips) {
  Pass q = pass_of<T>(a, p);
  q.p.parts = (int)std::min<int64_t>(ceil_div(p.strips, strips), 1 << 30);
  q.p.by_parts = Divider(q.p.parts);
  q.items = a.batch * a.groups * p.runs * q.p.parts;
  return q;
}

template <typename T>
hipError_t rows_fwd(const GroupArgs& a, const T* x, const float* gamma, const float* beta, T* y,
                    float* stats, hipStream_t s) {
  by_vector<kVec<T>>(a.channels / a.groups, [&](auto vec) {
    pick_rows<vec.value>(a.channels / a.groups, [&](auto tpr, auto nv) {
      constexpr int TPR = tpr.value, kB = TPR < kBlock ? kBlock : TPR, kSlots = kB / TPR;
      // a number of work-groups whose slots are a multiple of the groups, about as many as fill the
      // card, or as there are rows
      int64_t unit = a.groups;
      for (int64_t n = kSlots; n % 2 == 0 && unit % 2 == 0; n /= 2) unit /= 2;
      const int64_t need = ceil_div(a.batch * a.groups, kSlots), most = 1024 * kBlock / kB;
      const int64_t groups = unit * std::max<int64_t>(1, std::min(ceil_div(need, unit), most / unit));
      hipLaunchKernelGGL((k_gn_rows<T, vec.value, TPR, nv.value, kB>), dim3(groups), dim3(kB), 0, s,
                         a, a.channels / a.groups, Divider(a.groups), Scale(a), groups * kSlots,
                         groups * kSlots / a.groups, stream_out<T>(a), x, gamma, beta, y, stats);
    });
  });
  return hipGetLastError();
}

template <typename T>
hipError_t first_fwd(const GroupArgs& a, const T* x, const float* gamma, const float* beta, T* y,
                     float* stats, void* ws, hipStream_t s) {
  by_vector<kVec<T>>(a.npts, [&](auto vec) {
    constexpr int V = vec.value, W = kWhole<V>, K = kAhead;
    const bool whole = pick_whole<V, W>(a, [&](auto block, const Strip& p) {
      hipLaunchKernelGGL((k_gn_whole<T, V, W, block.value>), grid_of(a.batch * a.groups),
                         dim3(block.value), 0, s, a, p, a.batch * a.groups, x, gamma, beta, y, stats);
    });
    if (whole) return;
    const Strip p = strip_of<V, K, kBlock>(a);
    const Pass q = pass_of<T>(a, p), r = second_of<T>(a, p, 2);
    float4* part = static_cast<float4*>(ws);
    const auto go = [&](auto first, auto second) {
      hipLaunchKernelGGL(first, grid_of(q.items), dim3(kBlock), 0, s, a, q, x, part);
      hipLaunchKernelGGL(second, grid_of(r.items), dim3(kBlock), 0, s, a, r, x, gamma, beta, part, y,
                         stats);
    };
    if (p.strips > 1) go(k_gn_stats<T, V, K, true>, k_gn_apply<T, V, K, true>);
    else go(k_gn_stats<T, V, K, false>, k_gn_apply<T, V, K, false>);
  });
  return hipGetLastError();
}

// Where the sums for the weights' gradients go: into `rows` partial rows [2][channels], or where there
// is one row into the gradients themselves.
struct Partial {
  float *g = nullptr, *b = nullptr;
  Partial(const GroupArgs& a, int64_t rows, float* part, float* ggamma, float* gbeta) {
    if (!ggamma && !gbeta) return;
    g = rows == 1 ? ggamma : part;
    b = rows == 1 ? gbeta : part + a.channels;
  }
};

template <typename T>
size_t fwd_bytes(const GroupArgs& a) {
  if (form_of(a) == kRows) return 0;
  if (form_of(a) == kLast) return group_norm_last_fwd_bytes(a);
  return by_vector<kVec<T>>(a.npts, [&](auto vec) {
    constexpr int V = vec.value;
    if (pick_whole<V, kWhole<V>>(a, [](auto, const Strip&) {})) return (size_t)0;
    const Strip p = strip_of<V, kAhead, kBlock>(a);
    return up((int64_t)sizeof(float4) * a.batch * a.groups * p.runs * p.parts);
  });
}

// Workspace of n partial rows alone, and the weights' gradients from them (by a kernel that adds wide
// rows up in four float32 chains).
Fold rows_fold(const GroupArgs& a, int64_t n) { return Fold(n, a.channels >= 4096 ? 512 : kMostRows); }
size_t rows_bytes(const GroupArgs& a, int64_t n) {
  return n == 1 ? 0 : up((int64_t)sizeof(float) * 2 * n * a.channels) + rows_fold(a, n).bytes(a);
}
hipError_t rows_finish(const GroupArgs& a, int64_t n, float* part, float* ggamma, float* gbeta,
                       hipStream_t s) {
  float* to = reinterpret_cast<float*>(reinterpret_cast<char*>(part) +
                                       up((int64_t)sizeof(float) * 2 * n * a.channels));
  const Rows r = fold_rows(a, rows_fold(a, n), n, part, to, s);
  return launch_weight_sums(a.channels, (int)r.n, r.at, ggamma, gbeta, s);
}

template <typename T>
size_t bwd_bytes(const GroupArgs& a) {
  if (form_of(a) == kLast) return group_norm_last_bwd_bytes(a);
  if (form_of(a) == kRows)
    return by_vector<kVec<T>>(a.channels / a.groups, [&](auto vec) {
      return pick_rows<vec.value>(a.channels / a.groups, [&](auto tpr, auto) {
        return rows_bytes(a, rows_shape(a, tpr.value).down);
      });
    });
  return by_vector<kVec<T>>(a.npts, [&](auto vec) {
    constexpr int V = vec.value;
    if (pick_whole<V, kWholeBwd<V>>(a, [](auto, const Strip&) {}))
      return rows_bytes(a, a.batch);
    return Space(a, a.batch * strip_of<V, kAhead, kBlock>(a).parts, 0).bytes();
  });
}

template <typename T>
hipError_t rows_bwd(const GroupArgs& a, const T* x, const float* gamma, const float* beta,
                    const float* stats, const T* gy, T* gx, float* ggamma, float* gbeta, float* part,
                    hipStream_t s) {
  const bool weights = ggamma || gbeta;
  int parts = 0;
  by_vector<kVec<T>>(a.channels / a.groups, [&](auto vec) {
    pick_rows<vec.value>(a.channels / a.groups, [&](auto tpr, auto nv) {
      constexpr int V = vec.value, TPR = tpr.value, NV = nv.value;
      const RowsShape p = rows_shape(a, TPR);
      parts = p.down;
      const Partial to(a, parts, part, ggamma, gbeta);
      const auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(p.chunks * p.down), dim3(kRowsBlock), 0, s, a,
                           a.channels / a.groups, Divider(p.wide), p.wide, p.deep, p.chunks,
                           stream_out<T>(a), x, gamma, beta, stats, gy, gx, to.g, to.b,
                           2 * (int64_t)a.channels);
      };
      if (weights) go(k_gn_rows_bwd<T, V, TPR, NV, kRowsBlock, true>);
      else go(k_gn_rows_bwd<T, V, TPR, NV, kRowsBlock, false>);
    });
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !weights || parts == 1) return e;
  return rows_finish(a, parts, part, ggamma, gbeta, s);
}

template <typename T>
hipError_t first_bwd(const GroupArgs& a, const T* x, const float* gamma, const float* beta,
                     const float* stats, const T* gy, T* gx, float* ggamma, float* gbeta, void* ws,
                     hipStream_t s) {
  const bool weights = ggamma || gbeta;
  float* part = static_cast<float*>(ws);
  bool whole = false;
  by_vector<kVec<T>>(a.npts, [&](auto vec) {
    constexpr int V = vec.value, W = kWholeBwd<V>, K = kAhead;
    const Partial to(a, a.batch, part, ggamma, gbeta);
    whole = pick_whole<V, W>(a, [&](auto block, const Strip& p) {
      hipLaunchKernelGGL((k_gn_whole_bwd<T, V, W, block.value>), grid_of(a.batch * a.groups),
                         dim3(block.value), 0, s, a, p, a.batch * a.groups, x, gamma, beta, stats, gy,
                         gx, to.g, to.b, 2 * (int64_t)a.channels);
    });
    if (whole) return;
    const Strip p = strip_of<V, K, kBlock>(a);
    const Space z(a, a.batch * p.parts, 0);
    const Pass q = pass_of<T>(a, p), r = second_of<T>(a, p, 1);
    const bool own = small(a) && p.cg * p.parts <= 4 * kBlock;
    Between t = z.between(a, ws, gx != nullptr, ggamma, gbeta, own, r.items);
    const Sums sums = {p.cg, p.parts, Divider(p.cg)};
    const auto go = [&](auto first, auto second) {
      hipLaunchKernelGGL(first, grid_of(q.items), dim3(kBlock), 0, s, a, q, x, gamma, beta, stats, gy,
                         part);
      z.fold_in(a, t, ws, s);
      if (!t.own)
        hipLaunchKernelGGL(k_gn_between, Space::grid(a, t), dim3(kBlock), 0, s, a, t, sums, gamma);
      if (gx)
        hipLaunchKernelGGL(second, t.own ? Space::grid(a, t) : grid_of(r.items), dim3(kBlock), 0, s, a,
                           r, x, gamma, beta, stats, gy, t, sums, gx);
    };
    if (p.strips > 1) go(k_gn_sums<T, V, K, true>, k_gn_grad<T, V, K, true>);
    else go(k_gn_sums<T, V, K, false>, k_gn_grad<T, V, K, false>);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !weights || !whole || a.batch == 1) return e;
  return rows_finish(a, a.batch, part, ggamma, gbeta, s);
}

bool none(const GroupArgs& a) { return a.batch == 0 || a.npts == 0; }

__global__ __launch_bounds__(kBlock) void k_gn_zero(int64_t n, float* p) {
  for (int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x; i < n; i += (int64_t)gridDim.x * kBlock)
    p[i] = 0.f;
}

}  // namespace

Rows fold_rows(const GroupArgs& a, const Fold& f, int64_t n, const float* part, float* to,
               hipStream_t s) {
  if (f.size == 1) return {n, part};
  const int64_t width = 2 * (int64_t)a.channels, columns = ceil_div(width, kSumCols);
  hipLaunchKernelGGL(k_gn_fold, grid_of(f.rows * columns), dim3(kBlock), 0, s, width, n, f.size,
                     columns, f.rows * columns, part, to);
  return {f.rows, to};
}

size_t group_norm_fwd_bytes(const GroupArgs& a, int dtype) {
  if (none(a)) return 0;
  return by_type(dtype, [&](auto t) { return fwd_bytes<decltype(t)>(a); });
}

hipError_t launch_group_norm_fwd(const GroupArgs& a, int dtype, const void* x, const float* gamma,
                                 const float* beta, void* y, float* stats, void* ws,
                                 hipStream_t s) {
  if (none(a)) {
    const int64_t n = 2 * a.batch * a.groups;
    if (!stats || n == 0) return hipSuccess;
    hipLaunchKernelGGL(k_gn_zero, grid_of(ceil_div(n, kBlock)), dim3(kBlock), 0, s, n, stats);
    return hipGetLastError();
  }
  const Form form = form_of(a);
  if (form == kLast) return launch_group_norm_last_fwd(a, dtype, x, gamma, beta, y, stats, ws, s);
  return by_type(dtype, [&](auto t) {
    typedef decltype(t) T;
    const T* px = static_cast<const T*>(x);
    if (form == kRows) return rows_fwd<T>(a, px, gamma, beta, static_cast<T*>(y), stats, s);
    return first_fwd<T>(a, px, gamma, beta, static_cast<T*>(y), stats, ws, s);
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
  const Form form = form_of(a);
  if (form == kLast)
    return launch_group_norm_last_bwd(a, dtype, x, gamma, beta, stats, gy, gx, ggamma, gbeta, ws, s);
  return by_type(dtype, [&](auto t) {
    typedef decltype(t) T;
    const T *px = static_cast<const T*>(x), *pg = static_cast<const T*>(gy);
    T* to = static_cast<T*>(gx);
    if (form == kRows)
      return rows_bwd<T>(a, px, gamma, beta, stats, pg, to, ggamma, gbeta, static_cast<float*>(ws), s);
    return first_bwd<T>(a, px, gamma, beta, stats, pg, to, ggamma, gbeta, ws, s);
  });
}

}  // namespace fno
