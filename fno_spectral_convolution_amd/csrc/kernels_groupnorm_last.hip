// Group norm of channels-last data [batch][npts][channels] (and of rows of one point that are longer
// than a work-group holds, the same memory).  groupnorm_device.h has the mathematics.
//
// A thread keeps to four channels and goes down the rows, so that its weights, statistics and sums stay
// in registers.  Two passes: 8 x 256^2 x 128 bfloat16 with SiLU 76.5 us, moments 25 (5.4 TB/s), a launch
// that joins them 5, output 48 to 54 (5 TB/s), the same in float32 49, 5 and 108, backward 102, 5 and
// 161 (all 5 TB/s and more); 4 x 96^2 x 320 half with SiLU and dropout backward 47, sums 21, between 5,
// gradient 25: twelve rows a thread, whose setting out and sums over the work-group are a third of the
// instructions.  There neither the memory (3.2 and 3.7 TB/s) nor the vector units (55 to 70% busy) are
// full: four and five waves a SIMD, with 80 to 90 scalar registers of the arguments kept in vector ones.
#include "groupnorm_device.h"

namespace fno {
namespace {

// ---- channels last -------------------------------------------------------------------------------
// EVEN: vectors are whole, and each lies in one group (its mean and r are then one register each).
// A row is one point's channels.  A work-group takes a block of `cols` channels (tc vectors) and a
// tile of rows, tr of them at a time: a thread keeps to its vector's channels.  The part of a group
// that lies in a block is a segment; group g and block k make segment g + k, so that a group's
// segments are neighbours (numbers that no pair has stay unused).
struct Cut {
  int64_t rows;  // of a tile
  int tiles;
  Divider by_tiles;
};
struct Tiles : Cut {
  int cols, blocks, tc, tr;  // channels of a block, blocks, vectors of a block, rows at a time
  int cg;                    // channels of a group
  int seg_cols, seg_blocks;  // channels of a segment, blocks that a group touches, at most
  int64_t segments;
  bool paired;               // lanes 2 j and 2 j + 1 have neighbouring vectors of eight aligned elements
  Divider by_tc, by_tr, by_cols, by_cg, by_blocks;
  Scale scale;
};
template <int VEC>
Tiles tiles_of(const GroupArgs& a, int least, int most, int longest = 1 << 22) {
  Tiles p;
  p.cg = a.channels / a.groups;
  const int64_t nvec = ceil_div(a.channels, VEC);
  p.blocks = (int)ceil_div(nvec, 32);
  p.tc = (int)ceil_div(nvec, p.blocks);
  p.paired = VEC == 4 && a.channels % 8 == 0;
  if (p.paired) p.tc += p.tc % 2;
  p.cols = p.tc * VEC;
  p.blocks = (int)ceil_div(a.channels, p.cols);
  p.tr = kBlock / p.tc;
  p.segments = (int64_t)a.groups + p.blocks;
  // at most `most` work-groups, with `least` rows to a thread or more: a second, short round costs as
  // much as a whole one; or as many as leave `longest` rows to a thread, up to a million
  const int64_t want =
      std::max<int64_t>(1, most / std::max<int64_t>(1, a.batch * p.blocks));
  const int64_t tiles =  // (rows of a tile fit 31 bits)
      std::max(std::max(ceil_div(a.npts, (int64_t)1 << 30),
                        std::min<int64_t>(ceil_div(a.npts, (int64_t)p.tr * longest), 1 << 20)),
               std::min(ceil_div(a.npts, (int64_t)p.tr * least), want));
  p.rows = std::max<int64_t>(1, ceil_div(a.npts, tiles));
  p.tiles = (int)std::max<int64_t>(1, ceil_div(a.npts, p.rows));
  p.seg_cols = std::min(p.cg, p.cols);
  p.seg_blocks = (int)std::min<int64_t>(p.blocks, ((int64_t)p.cg + p.cols - 1) / p.cols + 1);
  p.by_tc = Divider(p.tc);
  p.by_tr = Divider(p.tr);
  p.by_cols = Divider(p.cols);
  p.by_cg = Divider(p.cg);
  p.by_blocks = Divider(p.blocks);
  p.by_tiles = Divider(p.tiles);
  p.scale = Scale(a);
  return p;
}
// Whether the second pass joins the parts for itself, which saves a launch: few enough for
// a work-group's threads.
bool joins(const Tiles& p) {
  const int64_t in_block = std::min<int64_t>(p.cols, (p.cols + (int64_t)p.cg - 1) / p.cg + 1);
  return in_block * p.seg_blocks * p.tiles <= 1024;
}

// The first pass's tiles: four rows to a thread or more, or eight where the second pass can then join
// the parts.
template <int VEC>
Tiles parts_tiles(const GroupArgs& a, int most, int longest = 1 << 22) {
  const Tiles p = tiles_of<VEC>(a, 4, most, longest);
  if (joins(p)) return p;
  const Tiles q = tiles_of<VEC>(a, 8, most, longest);
  return joins(q) ? q : p;
}
// Work-groups of each pass, two, three and four a compute unit.  The first passes end with sums over
// the work-group: 8 x 256^2 x 128 bf16 moments 24.6 us, 26.8 with 768, 26.9 with 1024; 4 x 96^2 x 320
// half sums with dropout 21.6, 23.2 with 512, 22.8 with 1024.  The second ones only stream: the same two
// 48.4 and 25.4 us, with 768 54.2 and 24.4, with 512 60.3 and 27.0; with 1280 both passes of the latter
// took 8 more.
constexpr int kMoments = 512, kSums = 768, kSecond = 1024;
// Rows to a thread in the second pass, at least: it has no parts of its own (3 x 4095 x 45 half backward
// 23 us with four, 26 with eight, 29 with two; both passes).
constexpr int kLeast = 4;
// And in the sums at most, four of which make one term of a thread's float32 chain.
constexpr int kLongest = 512;

struct Block {
  int64_t b, row0;     // entry, first row
  int k, tile, rows;   // column block, tile, rows of it
  int c0, c1, g0, segs;  // channels, first group, groups that it touches
};
__device__ __forceinline__ Block block_of(int64_t w, const GroupArgs& a, const Tiles& p) {
  Block q;
  const int64_t rest = p.by_blocks.of(w);
  q.k = (int)(w - rest * p.blocks);
  q.b = p.by_tiles.of(rest);
  q.tile = (int)(rest - q.b * p.tiles);
  q.row0 = q.tile * p.rows;
  q.rows = (int)(p.rows < a.npts - q.row0 ? p.rows : a.npts - q.row0);
  q.c0 = q.k * p.cols;
  q.c1 = q.c0 + p.cols < a.channels ? q.c0 + p.cols : a.channels;
  q.g0 = (int)p.by_cg.of((uint32_t)q.c0);
  q.segs = (int)p.by_cg.of((uint32_t)q.c1 - 1) - q.g0 + 1;
  return q;
}
// A thread's vector in a block: its first channel, and its own elements (as Items).
template <int VEC>
__device__ __forceinline__ void vector_of(const Block& q, const Tiles& p, int channels, int& r,
                                          int& c, int& lo) {
  r = (int)p.by_tc.of((uint32_t)threadIdx.x);
  const int at = q.c0 + (threadIdx.x - r * p.tc) * VEC;
  c = at < channels - VEC ? at : channels - VEC;
  lo = r < p.tr && at < channels ? at - c : VEC;
}

// Rows r, r + tr, ... of a tile, K at a time: f(at, n, all) with n of them there, all of them where
// the constant `all` says so; `at` is the element that slot 0's row begins with, the same for the whole
// work-group, so that a thread has one offset of its own for all its rows.  The last rows are loaded
// together like the others (2 x 10^6 x 20 half forward 64 us; one by one 69).
template <int K, typename F>
__device__ __forceinline__ void tile_rows(const Tiles& p, const Block& q, int r, int channels,
                                          F&& f) {
  int i = 0;
  for (; i + K * p.tr <= q.rows; i += K * p.tr) f((q.row0 + i) * channels, K, std::true_type());
  if (i + r < q.rows)
    f((q.row0 + i) * channels, (int)p.by_tr.of((uint32_t)(q.rows - i - r - 1)) + 1,
      std::false_type());
}
template <typename T, int VEC, int K, typename All>
__device__ __forceinline__ void load_rows(const T* p, int64_t step, int64_t own, int n, All all,
                                          Raw<T, VEC> (&raw)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (all.value || k < n) raw[k] = load_raw<T, VEC, true>(p + k * step + own);
}

// The masks of a thread's K rows from element i on, four bits each.
template <int VEC, int K>
__device__ __forceinline__ uint32_t row_masks(const GroupArgs& a, const Dropper& drop, int64_t i,
                                              int64_t step, bool paired) {
  return a.drop.threshold ? drop.masks<VEC, K>((uint64_t)i, step, paired) : 0;
}

// log2 of the lanes to a segment that has at most `terms` to add up, so that the segments take the
// work-group between them.
__device__ __forceinline__ int lanes_of(int segs, int terms) {
  int l = 6;
  while (l > 0 && (segs << l > kBlock || 1 << (l - 1) >= terms)) --l;
  return l;
}
// Calls f(segment, its first channel in the block, its width, lane, lanes) in the lanes of each: for
// sums over a segment's channels, or over the `terms` parts of its group.
template <typename F>
__device__ __forceinline__ void each_segment(const Tiles& p, const Block& q, int terms, F&& f) {
  const int log = lanes_of(q.segs, terms), lane = threadIdx.x & ((1 << log) - 1);
  for (int s = threadIdx.x >> log; s < q.segs; s += kBlock >> log) {
    const int g = q.g0 + s, from = max(q.c0, g * p.cg), to = min(q.c1, (g + 1) * p.cg);
    f(s, from - q.c0, to - from, lane, 1 << log);
  }
}
// The threads of a block's channels, in sets that share the row slots: no more than sixteen, whose sums
// each channel's lane then adds up in a row (256 of them for a single channel put the mean of 1.1s off by
// 42 units of 2^-24; 16 row slots to each of 16 sets are off by 11 at most).
struct Columns {
  int sets, set, c;  // set >= sets: none
  __device__ __forceinline__ explicit Columns(const Tiles& p) {
    sets = max(1, min((int)p.by_cols.of((uint32_t)kBlock), min(p.tr, 16)));
    set = (int)p.by_cols.of((uint32_t)threadIdx.x);
    c = threadIdx.x - set * p.cols;
  }
};

// part [batch][segments][tiles]: mean, squared deviations over m
template <typename T, int VEC, int K>
__global__ __launch_bounds__(kBlock) void k_gn_stats_last(GroupArgs a, Tiles p, int64_t total,
                                                          const T* x, float2* part) {
  __shared__ float2 s_mom[kBlock * VEC];  // [tr][cols]
  __shared__ float s_set[kBlock], s_mean[32 * VEC];
  const Scale scale = p.scale;
  const float inv_m = scale.inv_m;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const Block q = block_of(w, a, p);
    int r, c, lo;
    vector_of<VEC>(q, p, a.channels, r, c, lo);
    float n = 0.f, mean[VEC], var[VEC];
    fill(mean, 0.f);
    fill(var, 0.f);
    if (lo < VEC) {
      const T* from = x + q.b * a.x_stride;
      const int64_t own = (int64_t)r * a.channels + c;
      tile_rows<K>(p, q, r, a.channels, [&](int64_t at, int more, auto all) {
        Raw<T, VEC> raw[K] = {};
        load_rows<T, VEC, K>(from + at, (int64_t)p.tr * a.channels, own, more, all, raw);
        const float rows = (float)more, seen = n + rows;
        const float inv = all.value ? 1.0f / K : __builtin_amdgcn_rcpf(rows);
        const float share = rows * __builtin_amdgcn_rcpf(seen), between = share * (n * inv_m);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float sum = 0.f, sq = 0.f;
#pragma unroll
          for (int k = 0; k < K; ++k) sum += element<T, VEC>(raw[k], e);  // (zeros beyond `more`)
          const float m = sum * inv;
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const float d = scale.deviation(element<T, VEC>(raw[k], e), m);
            sq += all.value || k < more ? d * d : 0.f;
          }
          const float d = m - mean[e];
          mean[e] += d * share;
          var[e] += sq * scale.up + (d * between) * d;
        }
        n = seen;
      });
    }
    __syncthreads();
    if (lo < VEC)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e >= lo) s_mom[r * p.cols + c + e - q.c0] = make_float2(mean[e], var[e]);
    __syncthreads();
    // the row slots' moments of a segment: their mean first, then the deviations about it
    const Columns col(p);
    const int slots = min(p.tr, q.rows), width = q.c1 - q.c0;
    const bool mine = col.set < col.sets && col.c < width;
    // rows that slot i has seen: all rounds, and the last one where it is in it
    const int rounds = (int)p.by_tr.of((uint32_t)q.rows), more = q.rows - rounds * p.tr;
    const auto seen = [&](int i) { return (float)(rounds + (i < more)); };
    float sum = 0.f;
    if (mine) {
#pragma unroll 4
      for (int i = col.set; i < slots; i += col.sets)
        sum += seen(i) * s_mom[i * p.cols + col.c].x;
      s_set[threadIdx.x] = sum;
    }
    __syncthreads();
    each_segment(p, q, p.seg_cols, [&](int s, int from, int wide, int lane, int lanes) {
      float v = 0.f;
      for (int i = 0; i < col.sets; ++i)
#pragma unroll 4
        for (int k = lane; k < wide; k += lanes) v += s_set[i * p.cols + from + k];
      v = lanes_sum(v, lanes);
      if (lane == 0) s_mean[s] = v * __builtin_amdgcn_rcpf((float)q.rows * (float)wide);
    });
    __syncthreads();
    if (mine) {
      const float m = s_mean[(int)p.by_cg.of((uint32_t)(q.c0 + col.c)) - q.g0];
      sum = 0.f;
#pragma unroll 4
      for (int i = col.set; i < slots; i += col.sets) {
        const float2 v = s_mom[i * p.cols + col.c];
        sum += v.y + ((v.x - m) * (seen(i) * inv_m)) * (v.x - m);
      }
      s_set[threadIdx.x] = sum;
    }
    __syncthreads();
    each_segment(p, q, p.seg_cols, [&](int s, int from, int wide, int lane, int lanes) {
      float v = 0.f;
      for (int i = 0; i < col.sets; ++i)
#pragma unroll 4
        for (int k = lane; k < wide; k += lanes) v += s_set[i * p.cols + from + k];
      v = lanes_sum(v, lanes);
      if (lane == 0)
        part[(q.b * p.segments + q.g0 + s + q.k) * p.tiles + q.tile] = make_float2(s_mean[s], v);
    });
  }
}

// The column blocks that group g lies in.
struct Span {
  int first, blocks;
};
__device__ __forceinline__ Span span_of(const Tiles& p, int g) {
  const int k0 = (int)p.by_cols.of((uint32_t)(g * p.cg));
  const int k1 = (int)p.by_cols.of((uint32_t)((g + 1) * p.cg) - 1);
  return {k0, k1 - k0 + 1};
}
// The parts of group g of entry b, one a tile for each of its segments.
__device__ __forceinline__ const float2* parts_of(const Tiles& p, const Cut& cut,
                                                  const float2* part, int64_t b, int g,
                                                  const Span& sp) {
  return part + (b * p.segments + g + sp.first) * cut.tiles;
}
// Calls f(i, from[i]) for a lane's share of n parts, four loads ahead.
template <typename F>
__device__ __forceinline__ void each_part(const float2* from, int n, int lane, int lanes, F&& f) {
  for (int i = lane; i < n; i += 4 * lanes) {
    float2 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * lanes < n) v[u] = from[i + u * lanes];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * lanes < n) f(i + u * lanes, v[u]);
  }
}
// Mean and r of group g of entry b from its parts, in `lanes` lanes.
__device__ __forceinline__ float2 join_parts(const GroupArgs& a, const Tiles& p, const Cut& cut,
                                             const float2* part, int64_t b, int g, int lane,
                                             int lanes) {
  const float inv = 1.0f / ((float)p.cg * (float)a.npts);
  const Span sp = span_of(p, g);
  const float2* from = parts_of(p, cut, part, b, g, sp);
  const auto share = [&](int i) {  // of the group's entries in part i
    const int k = (int)cut.by_tiles.of((uint32_t)i), block = sp.first + k;
    const int width = (int)(min((int64_t)(block + 1) * p.cols, (int64_t)(g + 1) * p.cg) -
                            max((int64_t)block * p.cols, (int64_t)g * p.cg));
    const int64_t row0 = (i - k * cut.tiles) * cut.rows;
    const int64_t rows = cut.rows < a.npts - row0 ? cut.rows : a.npts - row0;
    return (float)rows * inv * (float)width;
  };
  float mean = 0.f, var = 0.f;
  each_part(from, sp.blocks * cut.tiles, lane, lanes,
            [&](int i, const float2& v) { mean += share(i) * v.x; });
  mean = lanes_sum(mean, lanes);
  each_part(from, sp.blocks * cut.tiles, lane, lanes, [&](int i, const float2& v) {
    var += v.y + ((v.x - mean) * share(i)) * (v.x - mean);
  });
  return make_float2(mean, rsqrtf(lanes_sum(var, lanes) + a.eps));
}

// stats [2][batch * groups] from the parts, a wave to a group
__global__ __launch_bounds__(kBlock) void k_gn_finish_last(GroupArgs a, Tiles p,
                                                           Divider by_groups, const float2* part,
                                                           float* stats) {
  const int64_t sides = a.batch * a.groups;
  for (int64_t i = (int64_t)blockIdx.x * kWaves + threadIdx.x / 64; i < sides;
       i += (int64_t)gridDim.x * kWaves) {
    const int64_t b = by_groups.of(i);
    const float2 st = join_parts(a, p, p, part, b, (int)(i - b * a.groups), threadIdx.x % 64, 64);
    if (threadIdx.x % 64 == 0) {
      stats[i] = st.x;
      stats[sides + i] = st.y;
    }
  }
}

// What s holds for the groups of a thread's channels.
template <int VEC, bool EVEN>
__device__ __forceinline__ void by_group(const Tiles& p, const Block& q, int c, const float2* s,
                                         float (&u)[VEC], float (&v)[VEC]) {
  if (EVEN) {
    const float2 t = s[(int)p.by_cg.of((uint32_t)c) - q.g0];
    fill(u, t.x);
    fill(v, t.y);
    return;
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const float2 t = s[max((int)p.by_cg.of((uint32_t)(c + e)) - q.g0, 0)];
    u[e] = t.x;
    v[e] = t.y;
  }
}
// a thread's channels' mean, r, gamma and beta
template <int VEC, bool EVEN>
__device__ __forceinline__ void channel_terms(const Tiles& p, const Block& q, int c,
                                              const float* gamma, const float* beta,
                                              const float2* s_st, float (&mu)[VEC],
                                              float (&rs)[VEC], float (&ga)[VEC],
                                              float (&be)[VEC]) {
  by_group<VEC, EVEN>(p, q, c, s_st, mu, rs);
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    ga[e] = gamma ? gamma[c + e] : 1.f;
    be[e] = beta ? beta[c + e] : 0.f;
  }
}

// the statistics of the groups that a block touches, as they are, into LDS
__device__ __forceinline__ void given_stats(const GroupArgs& a, const Block& q, const float* stats,
                                            float2* s_st) {
  for (int s = threadIdx.x; s < q.segs; s += kBlock)
    s_st[s] = make_float2(stats[q.b * a.groups + q.g0 + s],
                          stats[(a.batch + q.b) * a.groups + q.g0 + s]);
}

// stats: given (part NULL), or made here from the parts and, nullable, written
template <typename T, int VEC, int K, bool EVEN>
__global__ __launch_bounds__(kBlock) void k_gn_apply_last(GroupArgs a, Tiles p, Cut parts,
                                                          int64_t total, bool stream, const T* x,
                                                          const float* gamma, const float* beta,
                                                          const float2* part, T* y, float* stats) {
  __shared__ float2 s_st[32 * VEC];
  const Dropper drop(a.drop);
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const Block q = block_of(w, a, p);
    int r, c, lo;
    vector_of<VEC>(q, p, a.channels, r, c, lo);
    __syncthreads();
    if (part) {
      each_segment(p, q, p.seg_blocks * parts.tiles, [&](int s, int, int, int lane, int lanes) {
        const float2 st = join_parts(a, p, parts, part, q.b, q.g0 + s, lane, lanes);
        if (lane != 0) return;
        s_st[s] = st;
        // the block that has the group's first channel
        if (stats && q.tile == 0 && (q.g0 + s) * (int64_t)p.cg >= q.c0) {
          stats[q.b * a.groups + q.g0 + s] = st.x;
          stats[(a.batch + q.b) * a.groups + q.g0 + s] = st.y;
        }
      });
    } else {
      given_stats(a, q, stats, s_st);
    }
    __syncthreads();
    if (lo >= VEC) continue;
    float mu[VEC], by[VEC], ga[VEC], be[VEC];
    channel_terms<VEC, EVEN>(p, q, c, gamma, beta, s_st, mu, by, ga, be);
#pragma unroll
    for (int e = 0; e < VEC; ++e) by[e] *= ga[e];
    const T* from = x + q.b * a.x_stride;
    T* to = y + q.b * a.y_stride;
    const int64_t index = q.b * a.npts * a.channels, own = (int64_t)r * a.channels + c;
    const int64_t step = (int64_t)p.tr * a.channels;
    const auto put = [&](const Raw<T, VEC>& raw, int64_t at, uint32_t mask) {
      float f[VEC];
      unpack<T, VEC>(raw, f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = fmaf(f[e] - mu[e], by[e], be[e]);
      activate(f, a.act);
      if (a.drop.threshold) drop.apply<VEC>(f, mask);
      store_own<T, VEC>(to + at + own, f, EVEN ? 0 : lo, stream);
    };
    tile_rows<K>(p, q, r, a.channels, [&](int64_t at, int n, auto all) {
      Raw<T, VEC> raw[K];
      load_rows<T, VEC, K>(from + at, step, own, n, all, raw);
      const uint32_t masks = row_masks<VEC, K>(a, drop, index + at + own, step, p.paired);
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (all.value || k < n) put(raw[k], at + k * step, masks >> 4 * k);
    });
  }
}

// A lane's share of the sums of gamma g and gamma g h of group g of entry b.
__device__ __forceinline__ float2 seg_sums(const Tiles& p, const Cut& cut, const float2* seg,
                                           int64_t b, int g, int lane, int lanes) {
  const Span sp = span_of(p, g);
  const float2* from = parts_of(p, cut, seg, b, g, sp);
  double u = 0.0, v = 0.0;
  each_part(from, sp.blocks * cut.tiles, lane, lanes, [&](int, const float2& w) {
    u += w.x;
    v += w.y;
  });
  return make_float2((float)u, (float)v);
}

// part: rows [batch * tiles] of [2][channels], sums of g h and g; seg [batch][segments][tiles]: sums
// of gamma g and gamma g h
template <typename T, int VEC, int K, bool EVEN>
__global__ __launch_bounds__(kBlock) void k_gn_sums_last(GroupArgs a, Tiles p, int64_t total,
                                                         const T* x, const float* gamma,
                                                         const float* beta, const float* stats,
                                                         const T* gy, float* part, float2* seg) {
  __shared__ float2 s_st[32 * VEC], s_sum[kBlock * VEC], s_set[kBlock];
  const Dropper drop(a.drop);
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const Block q = block_of(w, a, p);
    int r, c, lo;
    vector_of<VEC>(q, p, a.channels, r, c, lo);
    __syncthreads();
    given_stats(a, q, stats, s_st);
    __syncthreads();
    if (lo < VEC) {
      float mu[VEC], rs[VEC], ga[VEC], be[VEC], sg[VEC], sb[VEC];
      fill(sg, 0.f);
      fill(sb, 0.f);
      channel_terms<VEC, EVEN>(p, q, c, gamma, beta, s_st, mu, rs, ga, be);
      const T* px = x + q.b * a.x_stride;
      const T* pg = gy + q.b * a.y_stride;
      const int64_t index = q.b * a.npts * a.channels, own = (int64_t)r * a.channels + c;
      const int64_t step = (int64_t)p.tr * a.channels;
      tile_rows<K>(p, q, r, a.channels, [&](int64_t at, int n, auto all) {
        Raw<T, VEC> rx[K], rg[K];
        load_rows<T, VEC, K>(px + at, step, own, n, all, rx);
        load_rows<T, VEC, K>(pg + at, step, own, n, all, rg);
        const uint32_t masks = row_masks<VEC, K>(a, drop, index + at + own, step, p.paired);
        float tg[VEC], tb[VEC];  // of these rows (the first is always there)
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (!all.value && k >= n) continue;
          float h[VEC], g[VEC];
          backward_terms<T, VEC>(a, drop, rx[k], rg[k], mu, rs, ga, be, masks >> 4 * k, h, g);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            tg[e] = k == 0 ? g[e] * h[e] : fmaf(g[e], h[e], tg[e]);
            tb[e] = k == 0 ? g[e] : tb[e] + g[e];
          }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          sg[e] += tg[e];
          sb[e] += tb[e];
        }
      });
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e >= lo) s_sum[r * p.cols + c + e - q.c0] = make_float2(sg[e], sb[e]);
    }
    __syncthreads();
    const Columns col(p);
    const int slots = min(p.tr, q.rows), width = q.c1 - q.c0;
    if (col.set < col.sets && col.c < width) {
      float2 v = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int i = col.set; i < slots; i += col.sets) {
        v.x += s_sum[i * p.cols + col.c].x;
        v.y += s_sum[i * p.cols + col.c].y;
      }
      s_set[threadIdx.x] = v;
    }
    __syncthreads();
    float* row = part + (q.b * p.tiles + q.tile) * 2 * a.channels + q.c0;
    if ((int)threadIdx.x < width) {  // (a block has at most 128 channels)
      float2 v = s_set[threadIdx.x];
      for (int i = 1; i < col.sets; ++i) {
        v.x += s_set[i * p.cols + threadIdx.x].x;
        v.y += s_set[i * p.cols + threadIdx.x].y;
      }
      row[threadIdx.x] = v.x;
      row[a.channels + threadIdx.x] = v.y;
      const float weight = gamma ? gamma[q.c0 + threadIdx.x] : 1.f;
      s_set[threadIdx.x] = make_float2(weight * v.y, weight * v.x);
    }
    __syncthreads();
    each_segment(p, q, p.seg_cols, [&](int s, int from, int wide, int lane, int lanes) {
      float u = 0.f, v = 0.f;
      for (int k = lane; k < wide; k += lanes) {
        u += s_set[from + k].x;
        v += s_set[from + k].y;
      }
      u = lanes_sum(u, lanes);
      v = lanes_sum(v, lanes);
      if (lane == 0)
        seg[(q.b * p.segments + q.g0 + s + q.k) * p.tiles + q.tile] = make_float2(u, v);
    });
  }
}

template <typename T, int VEC, int K, bool EVEN>
__global__ __launch_bounds__(kBlock) void k_gn_grad_last(GroupArgs a, Tiles p, Cut parts,
                                                         int64_t total, bool stream, const T* x,
                                                         const float* gamma, const float* beta,
                                                         const float* stats, const T* gy,
                                                         Between z, const float2* seg, T* gx) {
  __shared__ float2 s_st[32 * VEC], s_m[32 * VEC];
  const Dropper drop(a.drop);
  if (z.own && blockIdx.x >= z.groups) return weight_sums(a, z);
  const int64_t stride = z.own ? z.groups : gridDim.x;
  for (int64_t w = blockIdx.x; w < total; w += stride) {
    const Block q = block_of(w, a, p);
    int r, c, lo;
    vector_of<VEC>(q, p, a.channels, r, c, lo);
    __syncthreads();
    given_stats(a, q, stats, s_st);
    if (z.own) {
      const float inv = 1.0f / ((float)p.cg * (float)a.npts);
      each_segment(p, q, p.seg_blocks * parts.tiles, [&](int s, int, int, int lane, int lanes) {
        float2 v = seg_sums(p, parts, seg, q.b, q.g0 + s, lane, lanes);
        v = make_float2(lanes_sum(v.x, lanes) * inv, lanes_sum(v.y, lanes) * inv);
        if (lane == 0) s_m[s] = v;
      });
    } else {
      for (int s = threadIdx.x; s < q.segs; s += kBlock)
        s_m[s] = z.means[q.b * a.groups + q.g0 + s];
    }
    __syncthreads();
    if (lo >= VEC) continue;
    float mu[VEC], rs[VEC], ga[VEC], be[VEC], m1[VEC], m2[VEC];
    channel_terms<VEC, EVEN>(p, q, c, gamma, beta, s_st, mu, rs, ga, be);
    by_group<VEC, EVEN>(p, q, c, s_m, m1, m2);
    const T* px = x + q.b * a.x_stride;
    const T* pg = gy + q.b * a.y_stride;
    T* to = gx + q.b * a.gx_stride;
    const int64_t index = q.b * a.npts * a.channels, own = (int64_t)r * a.channels + c;
    const int64_t step = (int64_t)p.tr * a.channels;
    const auto put = [&](const Raw<T, VEC>& rx, const Raw<T, VEC>& rg, int64_t at, uint32_t mask) {
      float h[VEC], g[VEC];
      backward_terms<T, VEC>(a, drop, rx, rg, mu, rs, ga, be, mask, h, g);
#pragma unroll
      for (int e = 0; e < VEC; ++e) g[e] = rs[e] * fmaf(ga[e], g[e], -fmaf(h[e], m2[e], m1[e]));
      store_own<T, VEC>(to + at + own, g, EVEN ? 0 : lo, stream);
    };
    tile_rows<K>(p, q, r, a.channels, [&](int64_t at, int n, auto all) {
      Raw<T, VEC> rx[K], rg[K];
      load_rows<T, VEC, K>(px + at, step, own, n, all, rx);
      load_rows<T, VEC, K>(pg + at, step, own, n, all, rg);
      const uint32_t masks = row_masks<VEC, K>(a, drop, index + at + own, step, p.paired);
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (all.value || k < n) put(rx[k], rg[k], at + k * step, masks >> 4 * k);
    });
  }
}

__global__ __launch_bounds__(kBlock) void k_gn_between_last(GroupArgs a, Tiles p, Between z,
                                                            const float2* seg) {
  between(a, z, [&](int64_t b, int g) { return seg_sums(p, p, seg, b, g, threadIdx.x, kBlock); });
}

// ---- launches ------------------------------------------------------------------------------------
// Four elements to a vector: eight halves, whose weights and sums each thread keeps for all its rows,
// need twice the registers.  K rows to a thread at a time, 64 bytes of each field.
constexpr int kVecLast = 4;
template <typename T, int VEC>
constexpr int kRowsAhead = VEC * (int)sizeof(T) == 8 ? 8 : 4;
bool even(const GroupArgs& a) { return a.channels / a.groups % kVecLast == 0; }

// Whether an output goes past the caches: where it is large, and the work-groups' rows begin and end near
// whole lines.  Others are left to the cache to put together.  Forward and backward with the streaming
// stores over without, 134 to 400 MB: rows of 256 bytes 149 us over 155 and 245 over 253, of 96 159 over
// 162 and 265 over 274, but of 90 (45 half) 248 over 232 and 411 over 387, of 40 268 over 251 and 426 over
// 418; 64 bf16 from 32 bytes into a line 186 over 175 and 296 over 290.  (Planes and rows of tokens gain
// at any alignment: 20 x 600001 float32 212 over 218 and 334 over 361.)
template <typename T>
bool stream_rows(const GroupArgs& a, const T* to, int64_t stride) {
  return stream_out<T>(a) && a.channels * sizeof(T) % 32 == 0 &&
         reinterpret_cast<uintptr_t>(to) % 64 == 0 && (a.batch == 1 || stride * sizeof(T) % 64 == 0);
}

template <typename F>
auto pick(const GroupArgs& a, F&& f) {
  return by_vector<kVecLast>(a.channels, f);
}

template <typename T>
hipError_t fwd(const GroupArgs& a, const T* x, const float* gamma, const float* beta, T* y,
               float* stats, void* ws, hipStream_t s) {
  pick(a, [&](auto vec) {
    constexpr int V = vec.value, K = kRowsAhead<T, V>;
    const Tiles p = parts_tiles<V>(a, kMoments), r = tiles_of<V>(a, kLeast, kSecond);
    const int64_t total = a.batch * p.tiles * p.blocks, items = a.batch * r.tiles * r.blocks;
    float2* part = static_cast<float2*>(ws);
    hipLaunchKernelGGL((k_gn_stats_last<T, V, K>), grid_of(total), dim3(kBlock), 0, s, a, p, total,
                       x, part);
    if (!joins(p)) {
      const int64_t sides = a.batch * a.groups;
      if (!stats)
        stats = reinterpret_cast<float*>(
            static_cast<char*>(ws) + up((int64_t)sizeof(float2) * a.batch * p.segments * p.tiles));
      hipLaunchKernelGGL(k_gn_finish_last, grid_of(ceil_div(sides, kWaves)), dim3(kBlock), 0, s, a,
                         p, Divider(a.groups), part, stats);
      part = nullptr;
    }
    const auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid_of(items), dim3(kBlock), 0, s, a, r, p, items,
                         stream_rows(a, y, a.y_stride), x, gamma, beta, part, y, stats);
    };
    if (V > 1 && even(a)) go(k_gn_apply_last<T, V, K, V != 1>);
    else go(k_gn_apply_last<T, V, K, false>);
  });
  return hipGetLastError();
}

template <typename T>
hipError_t bwd(const GroupArgs& a, const T* x, const float* gamma, const float* beta,
               const float* stats, const T* gy, T* gx, float* ggamma, float* gbeta, void* ws,
               hipStream_t s) {
  pick(a, [&](auto vec) {
    constexpr int V = vec.value, K = 4;
    const Tiles p = parts_tiles<V>(a, kSums, kLongest), r = tiles_of<V>(a, kLeast, kSecond);
    const int64_t total = a.batch * p.tiles * p.blocks, items = a.batch * r.tiles * r.blocks;
    const Space z(a, a.batch * p.tiles, a.batch * p.segments * p.tiles);
    Between q = z.between(a, ws, gx != nullptr, ggamma, gbeta,
                                joins(p) && small(a), items);
    const auto go = [&](auto first, auto second) {
      hipLaunchKernelGGL(first, grid_of(total), dim3(kBlock), 0, s, a, p, total, x, gamma, beta,
                         stats, gy, static_cast<float*>(ws), z.segments_at(ws));
      z.fold_in(a, q, ws, s);
      if (!q.own)
        hipLaunchKernelGGL(k_gn_between_last, Space::grid(a, q), dim3(kBlock), 0, s, a, p, q,
                           z.segments_at(ws));
      if (gx)
        hipLaunchKernelGGL(second, q.own ? Space::grid(a, q) : grid_of(items), dim3(kBlock), 0, s, a, r,
                           p, items, stream_rows(a, gx, a.gx_stride), x, gamma, beta, stats, gy,
                           q, z.segments_at(ws), gx);
    };
    if (V > 1 && even(a)) go(k_gn_sums_last<T, V, K, V != 1>, k_gn_grad_last<T, V, K, V != 1>);
    else go(k_gn_sums_last<T, V, K, false>, k_gn_grad_last<T, V, K, false>);
  });
  return hipGetLastError();
}

}  // namespace

size_t group_norm_last_fwd_bytes(const GroupArgs& a) {
  return pick(a, [&](auto vec) {
    const Tiles p = parts_tiles<vec.value>(a, kMoments);
    return up((int64_t)sizeof(float2) * a.batch * p.segments * p.tiles) +
           (joins(p) ? 0 : up((int64_t)sizeof(float) * 2 * a.batch * a.groups));
  });
}

size_t group_norm_last_bwd_bytes(const GroupArgs& a) {
  return pick(a, [&](auto vec) {
    const Tiles p = parts_tiles<vec.value>(a, kSums, kLongest);
    return Space(a, a.batch * p.tiles, a.batch * p.segments * p.tiles).bytes();
  });
}

hipError_t launch_group_norm_last_fwd(const GroupArgs& a, int dtype, const void* x,
                                      const float* gamma, const float* beta, void* y, float* stats,
                                      void* ws, hipStream_t s) {
  return by_type(dtype, [&](auto t) {
    typedef decltype(t) T;
    return fwd<T>(a, static_cast<const T*>(x), gamma, beta, static_cast<T*>(y), stats, ws, s);
  });
}

hipError_t launch_group_norm_last_bwd(const GroupArgs& a, int dtype, const void* x,
                                      const float* gamma, const float* beta, const float* stats,
                                      const void* gy, void* gx, float* ggamma, float* gbeta,
                                      void* ws, hipStream_t s) {
  return by_type(dtype, [&](auto t) {
    typedef decltype(t) T;
    return bwd<T>(a, static_cast<const T*>(x), gamma, beta, stats, static_cast<const T*>(gy),
                  static_cast<T*>(gx), ggamma, gbeta, ws, s);
  });
}

}  // namespace fno
