// The global gradient norm over a list of tensors, clipping, and the AdamW update.
//
//   norm = sqrt(sum g^2) / scale,  factor = min(1, max / norm) / scale,  out = factor g
//   m = b1 m + (1 - b1) factor g,  v = b2 v + (1 - b2) (factor g)^2,
//   p = p - (lr decay p + (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps))
//
// Memory bounds all three: 4 bytes an element read, 8 read and written, 28.  A list is one launch
// whatever its number of tensors: the work-groups share its chunks out evenly, each a run of
// neighbours, so that a work-group meets few tensors and goes through each in 16-byte vectors, four
// (AdamW: two of each of its four operands) under way.  Offsets inside a run are 32 bits, where it
// lies is 64.  The sum of squares is float64: no gradient over- or underflows it, and it costs
// nothing (float32 sums measured the same).  Its order is fixed by the list and the work-groups.
//
// Measured on an MI355X whose large copies run at 4.9 TB/s:
//   norm   300 MB of half gradients 50 us (6.0 TB/s), 400 MB of float32 65 us (6.2)
//   clip   301 half tensors, 150 million entries, into float32, with its norm 217 us (its own 900 MB
//          163 us, 5.5 TB/s; the norm reads 300 MB before)
//   AdamW  52 million float32 entries 304 us (4.8 TB/s), with the norm before it 342 us: what the
//          update before wrote last leaves the 256 MB cache meanwhile
#include <algorithm>

#include "train_device.h"
#include "train_ops.h"

namespace fno {
namespace {

constexpr int kThreads = 256;

// fixed-order sum of one double per thread; every thread gets it
__device__ __forceinline__ double group_sum(double v, double* s_red) {
  constexpr int kWaves = kThreads / 64;
  v = wave_sum(v);
  if (threadIdx.x % 64 == 0) s_red[threadIdx.x / 64] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) s += s_red[w];
  return s;
}

// The record's norm and factor from the partial sums of squares; every thread gets them.
struct Record {
  float norm, factor;
};
__device__ __forceinline__ Record record_of(const double* part, const NormRecord& r,
                                            double* s_red) {
  double a = 0.0;
  for (int i = threadIdx.x; i < r.nparts; i += kThreads) a += part[i];
  const double norm = sqrt(group_sum(a, s_red)) / (double)r.grad_scale;
  double f = norm > (double)r.max_norm ? (double)r.max_norm / norm : 1.0;
  if (!(norm < (double)INFINITY)) f = (double)NAN;
  return {(float)norm, (float)(f / (double)r.grad_scale)};
}

template <typename T>
__device__ __forceinline__ Global<T> data_of(const TensorTable& t, uint32_t k, int64_t at) {
  return (Global<T>)uniform(reinterpret_cast<int64_t>(t.entry[k].data)) + at;
}

// Calls f(entry number, first element, elements) for the spans of this work-group's share of the
// chunks: neighbours, so that a work-group meets few tensors.  A span has at most 2^28 elements,
// so that offsets inside it fit 32 bits; where it lies in its tensor is 64 bits.
template <typename F>
__device__ __forceinline__ void each_span(const TensorTable& t, F&& f) {
  const uint64_t total = t.chunks;
  uint32_t c = (uint32_t)(total * blockIdx.x / gridDim.x);
  const uint32_t end = (uint32_t)(total * (blockIdx.x + 1) / gridDim.x);
  while (c < end) {
    const uint32_t k = uniform(t.of_chunk[c]), first = uniform(t.entry[k].first);
    const int64_t elems = uniform(t.entry[k].elems);
    const int64_t at = (int64_t)(c - first) * kChunk;
    const uint32_t most = end - c < (1u << 28) / kChunk ? end - c : (1u << 28) / kChunk;
    const int64_t n = elems - at < most * kChunk ? elems - at : most * kChunk;
    f(k, at, (int)n);
    c += (uint32_t)((n + kChunk - 1) / kChunk);
  }
}

// Elements of a span until one lies on a 128-byte line: vectors from there on do not straddle
// lines (reads of half gradients packed at odd places 66 -> 58 us for 300 MB), and what is written
// goes in whole lines.
template <typename T>
__device__ __forceinline__ int lead_of(Global<T> p, int n) {
  const int lead = (int)(-(uint64_t)p & 127) / (int)sizeof(T);
  return lead < n ? lead : n;
}

constexpr int kAhead = 4;  // vectors that a thread has in flight of each operand

template <typename T, int V>
__device__ __forceinline__ double squares(const Raw<T, V>& q) {
  double a = 0.0;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const double g = (double)element<T, V>(q, e);
    a += g * g;
  }
  return a;
}

template <typename T, bool Stream>
__device__ __forceinline__ double sum_squares(Global<const T> p, int n) {
  constexpr int V = 16 / (int)sizeof(T);
  double a[kAhead] = {};
  const int lead = lead_of(p, n), nv = (n - lead) / V;
  const auto one = [&](int i) {
    const double g = (double)to_float<T>(p[i]);
    a[1] += g * g;
  };
  if ((int)threadIdx.x < lead) one(threadIdx.x);
  const int rest = lead + nv * V + threadIdx.x;
  if (rest < n) one(rest);
  p += lead;
  int i = threadIdx.x;
  for (; i + (kAhead - 1) * kThreads < nv; i += kAhead * kThreads) {
    Raw<T, V> q[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) q[u] = load_global<T, V, Stream>(p + (i + u * kThreads) * V);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) a[u] += squares<T, V>(q[u]);
  }
  for (; i < nv; i += kThreads) a[0] += squares<T, V>(load_global<T, V, Stream>(p + i * V));
  double s = 0.0;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) s += a[u];
  return s;
}

template <bool Stream>
__global__ __launch_bounds__(kThreads) void k_norm_part(TensorTable t, double* part) {
  __shared__ double s_red[kThreads / 64];
  double a = 0.0;
  each_span(t, [&](uint32_t k, int64_t at, int n) {
    const uint32_t d = uniform((uint32_t)t.entry[k].dtype);
    if (d == FNO_DTYPE_F32) a += sum_squares<float, Stream>(data_of<const float>(t, k, at), n);
    else if (d == FNO_DTYPE_BF16) a += sum_squares<__bf16, Stream>(data_of<const __bf16>(t, k, at), n);
    else a += sum_squares<_Float16, Stream>(data_of<const _Float16>(t, k, at), n);
  });
  a = group_sum(a, s_red);
  if (threadIdx.x == 0) part[blockIdx.x] = a;
}

__global__ __launch_bounds__(kThreads) void k_norm_finish(const double* part, NormRecord r,
                                                          float* record) {
  __shared__ double s_red[kThreads / 64];
  const Record rec = record_of(part, r, s_red);
  if (threadIdx.x == 0) {
    record[0] = rec.norm;
    record[1] = rec.factor;
  }
}

template <typename T, typename U>
__device__ __forceinline__ void scale_chunk(Global<const T> p, Global<U> o, int n, float f,
                                            bool stream) {
  // 16 bytes of the wider type: lanes next to one another write next to one another
  constexpr int V = 16 / (int)(sizeof(T) > sizeof(U) ? sizeof(T) : sizeof(U));
  const int lead = lead_of(o, n), nv = (n - lead) / V;
  const auto one = [&](int i) { o[i] = from_float<U>(to_float<T>(p[i]) * f); };
  if ((int)threadIdx.x < lead) one(threadIdx.x);
  const int rest = lead + nv * V + threadIdx.x;
  if (rest < n) one(rest);
  p += lead;
  o += lead;
  int i = threadIdx.x;
  const auto put = [&](const Raw<T, V>& q, int j) {
    float g[V];
    unpack<T, V>(q, g);
#pragma unroll
    for (int e = 0; e < V; ++e) g[e] *= f;
    store_global<U, V>(o + j * V, g, stream);
  };
  for (; i + (kAhead - 1) * kThreads < nv; i += kAhead * kThreads) {
    Raw<T, V> q[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) q[u] = load_global<T, V>(p + (i + u * kThreads) * V);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) put(q[u], i + u * kThreads);
  }
  for (; i < nv; i += kThreads) put(load_global<T, V>(p + i * V), i);
}

// Every work-group adds up the partial sums for itself (in the same order, and out of its L2),
// which costs less than a launch between the norm and this.
__global__ __launch_bounds__(kThreads) void k_clip(TensorTable t, TensorTable out,
                                                   const double* part, NormRecord r,
                                                   float* record, bool stream) {
  __shared__ double s_red[kThreads / 64];
  const Record rec = record_of(part, r, s_red);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    record[0] = rec.norm;
    record[1] = rec.factor;
  }
  const float f = rec.factor;
  each_span(t, [&](uint32_t k, int64_t at, int n) {
    if (f == 1.0f && data_of<char>(t, k, 0) == data_of<char>(out, k, 0)) return;
    const uint32_t d = uniform((uint32_t)t.entry[k].dtype);
    const bool wide = uniform((uint32_t)out.entry[k].dtype) == FNO_DTYPE_F32;
    if (d == FNO_DTYPE_F32) {
      scale_chunk<float, float>(data_of<const float>(t, k, at), data_of<float>(out, k, at), n, f, stream);
    } else if (d == FNO_DTYPE_BF16) {
      const Global<const __bf16> p = data_of<const __bf16>(t, k, at);
      if (wide) scale_chunk<__bf16, float>(p, data_of<float>(out, k, at), n, f, stream);
      else scale_chunk<__bf16, __bf16>(p, data_of<__bf16>(out, k, at), n, f, stream);
    } else {
      const Global<const _Float16> p = data_of<const _Float16>(t, k, at);
      if (wide) scale_chunk<_Float16, float>(p, data_of<float>(out, k, at), n, f, stream);
      else scale_chunk<_Float16, _Float16>(p, data_of<_Float16>(out, k, at), n, f, stream);
    }
  });
}

// The decay and the step leave the parameter together, in one rounding: a factor 1 - lr decay in
// float32 would be off by up to 2^-25 for all parameters alike, at lr decay below that by all of it.
__device__ __forceinline__ void adamw_one(float& p, float g, float& m, float& v,
                                          const AdamArgs& a, float f) {
  g *= f;
  m = a.beta1 * m + a.one_minus_beta1 * g;
  v = a.beta2 * v + a.one_minus_beta2 * g * g;
  p -= a.decay * p + a.step_size * m / (sqrtf(v) * a.inv_bias2 + a.eps);
}

template <typename T>
__device__ __forceinline__ void adamw_chunk(Global<float> p, Global<const T> g, Global<float> m,
                                            Global<float> v, int n, const AdamArgs& a, float f) {
  constexpr int V = 4, kTwo = 2;
  typedef Raw<float, V> Q;
  const int lead = lead_of(p, n), nv = (n - lead) / V;
  const auto one = [&](int i) {
    float qp = p[i], qm = m[i], qv = v[i];
    adamw_one(qp, to_float<T>(g[i]), qm, qv, a, f);
    p[i] = qp;
    m[i] = qm;
    v[i] = qv;
  };
  if ((int)threadIdx.x < lead) one(threadIdx.x);
  const int rest = lead + nv * V + threadIdx.x;
  if (rest < n) one(rest);
  p += lead;
  g += lead;
  m += lead;
  v += lead;
  int i = threadIdx.x;
  const auto put = [&](const Q& qp, const Raw<T, V>& qg, const Q& qm, const Q& qv, int j) {
    float fp[V], fm[V], fv[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      fp[e] = qp[e];
      fm[e] = qm[e];
      fv[e] = qv[e];
      adamw_one(fp[e], to_float<T>(qg[e]), fm[e], fv[e], a, f);
    }
    store_global<float, V>(p + j, fp, false);
    store_global<float, V>(m + j, fm, false);
    store_global<float, V>(v + j, fv, false);
  };
  for (; i + (kTwo - 1) * kThreads < nv; i += kTwo * kThreads) {
    Q qp[kTwo], qm[kTwo], qv[kTwo];
    Raw<T, V> qg[kTwo];
#pragma unroll
    for (int u = 0; u < kTwo; ++u) {
      const int j = (i + u * kThreads) * V;
      qg[u] = load_global<T, V>(g + j);
      qp[u] = load_global<float, V>(p + j);
      qm[u] = load_global<float, V>(m + j);
      qv[u] = load_global<float, V>(v + j);
    }
#pragma unroll
    for (int u = 0; u < kTwo; ++u) put(qp[u], qg[u], qm[u], qv[u], (i + u * kThreads) * V);
  }
  for (; i < nv; i += kThreads) {
    const int j = i * V;
    put(load_global<float, V>(p + j), load_global<T, V>(g + j), load_global<float, V>(m + j),
        load_global<float, V>(v + j), j);
  }
}

__global__ __launch_bounds__(kThreads) void k_adamw(TensorTable params, TensorTable grads,
                                                    TensorTable exp_avg, TensorTable exp_avg_sq,
                                                    AdamArgs a, const float* record) {
  const float f = record ? record[1] : 1.0f;
  if (!(fabsf(f) < INFINITY)) return;  // the gradients were not finite: no update
  each_span(params, [&](uint32_t k, int64_t at, int n) {
    const uint32_t d = uniform((uint32_t)grads.entry[k].dtype);
    const Global<float> p = data_of<float>(params, k, at);
    const Global<float> m = data_of<float>(exp_avg, k, at);
    const Global<float> v = data_of<float>(exp_avg_sq, k, at);
    if (d == FNO_DTYPE_F32) adamw_chunk<float>(p, data_of<const float>(grads, k, at), m, v, n, a, f);
    else if (d == FNO_DTYPE_BF16) adamw_chunk<__bf16>(p, data_of<const __bf16>(grads, k, at), m, v, n, a, f);
    else adamw_chunk<_Float16>(p, data_of<const _Float16>(grads, k, at), m, v, n, a, f);
  });
}

// Whether what a clip writes outgrows the 256 MB cache behind the L2s: it goes past them (150
// million half entries into float32 226 us against 255, 100 million float32 229 against 246).  AdamW's
// writes measured the same either way.
bool large(const TensorTable& t) { return t.bytes > ((int64_t)256 << 20); }

// Work-groups of the kernels that write: as many as the compute units hold at a time; half of them
// where the writes go past the caches (150 million half entries into float32 211 us against 226,
// bfloat16 into bfloat16 156 against 168, 100 million float32 217 against 229).  Writes that the
// caches take measured the same or 1 us less with all of them.
int write_groups(const TensorTable& t, bool stream) {
  return (int)std::min(t.chunks, stream ? 1024u : 2048u);
}

}  // namespace

// A norm by itself reads a list of more than 128 MB past the caches: 300 MB of half gradients 50 us
// against 58, 600 MB of float32 93 against 107, and so with the AdamW update behind it (52 million
// float32 entries 339 against 346, 150 million 948 against 977; at 100 MB 165 against 162, at 40 MB 74
// against 71).  Where a clip reads the same gradients next, it finds a part of them in the caches:
// 150 million half entries into float32 211 us with plain loads, 233 without.
hipError_t launch_norm_part(const TensorTable& t, int groups, double* part, bool again,
                            hipStream_t s) {
  const auto kernel = !again && t.bytes > ((int64_t)128 << 20) ? k_norm_part<true> : k_norm_part<false>;
  hipLaunchKernelGGL(kernel, dim3(groups), dim3(kThreads), 0, s, t, part);
  return hipGetLastError();
}

hipError_t launch_norm_finish(const double* part, const NormRecord& r, float* record,
                              hipStream_t s) {
  hipLaunchKernelGGL(k_norm_finish, dim3(1), dim3(kThreads), 0, s, part, r, record);
  return hipGetLastError();
}

hipError_t launch_clip(const TensorTable& t, const TensorTable& out, const double* part,
                       const NormRecord& r, float* record, hipStream_t s) {
  const bool stream = large(out);
  hipLaunchKernelGGL(k_clip, dim3(write_groups(t, stream)), dim3(kThreads), 0, s, t, out, part, r,
                     record, stream);
  return hipGetLastError();
}

hipError_t launch_adamw(const TensorTable& params, const TensorTable& grads,
                        const TensorTable& exp_avg, const TensorTable& exp_avg_sq,
                        const AdamArgs& a, const float* record, hipStream_t s) {
  hipLaunchKernelGGL(k_adamw, dim3(write_groups(params, false)), dim3(kThreads), 0, s, params, grads,
                     exp_avg, exp_avg_sq, a, record);
  return hipGetLastError();
}

}  // namespace fno
