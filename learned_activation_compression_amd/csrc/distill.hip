// The last stage's loss: cross-entropy with the labels and the divergence from a
// teacher's top logits, and its gradient.  Formulas: include/mapl_block.h.  Both are
// bound by the logits' traffic: one read of them, and for the gradient one write.
#include "internal.h"
#include "vec8.h"

namespace mapl {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kThreads = 256, kAhead = 4;  // vectors of 8 logits in flight per thread
constexpr int kMaxK = 1024;
constexpr int64_t kSlice = 8 * kThreads;   // the least logits that a block takes of a row

template <typename T>
struct DistillArgs {
  const T* Z;
  const int32_t *labels, *t_ids;
  const float *t_logits, *gloss;
  float *loss, *stats, *part;  // part [N][splits][4]: maximum, the two sums
  T* gZ;
  float inv_T, w_ce, w_kd;
  bool warm;  // temperature other than 1: two sums
  int64_t N, V, per;  // per: logits of a block
  int K, splits;
};

struct Sums {  // sums of exp(z - m) and exp((z - m) / T)
  float m, s1, sT;
};
// a maximum of -inf stands for no finite logit: nothing is scaled by it
__device__ __forceinline__ float ref(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ Sums join(Sums a, Sums b, float inv_T) {
  const float m = fmaxf(a.m, b.m), x = (a.m - ref(m)) * kLog2e, y = (b.m - ref(m)) * kLog2e;
  return {m, a.s1 * exp2f(x) + b.s1 * exp2f(y), a.sT * exp2f(x * inv_T) + b.sT * exp2f(y * inv_T)};
}

// over the block, the same in every thread
__device__ __forceinline__ Sums block_join(Sums v, float inv_T, Sums* lds) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1)
    v = join(v, {__shfl_xor(v.m, s), __shfl_xor(v.s1, s), __shfl_xor(v.sT, s)}, inv_T);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) v = join(v, lds[w], inv_T);
  __syncthreads();
  return v;
}
__device__ __forceinline__ float block_sum(float v, float* lds) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) v += __shfl_xor(v, s);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
  __syncthreads();
  return v;
}
__device__ __forceinline__ float block_max(float v, float* lds) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) v = fmaxf(v, __shfl_xor(v, s));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = fmaxf(fmaxf(lds[0], lds[1]), fmaxf(lds[2], lds[3]));
  __syncthreads();
  return v;
}

// The teacher's entries k = threadIdx.x + 256 j of a row: their ids (-1: none) and the
// logarithms of their probabilities.  An entry with a logit of -inf has none.
struct Teacher {
  int id[kMaxK / kThreads];
  float logq[kMaxK / kThreads];
  bool some;
};
template <typename T>
__device__ __forceinline__ Teacher teacher(const DistillArgs<T>& a, int64_t n, float* lds) {
  Teacher t;
  float top = -INFINITY, bad = 0.f;
#pragma unroll
  for (int j = 0; j < kMaxK / kThreads; ++j) {
    const int k = threadIdx.x + kThreads * j;
    t.id[j] = -1;
    t.logq[j] = -INFINITY;
    if (k < a.K) {
      const int id = a.t_ids[n * a.K + k];
      const float x = a.t_logits[n * a.K + k] * a.inv_T;
      if (id >= 0 && id < a.V && x != -INFINITY) {
        t.id[j] = id;
        t.logq[j] = x;
        top = fmaxf(top, x);
        if (x != x) bad = 1.f;
      }
    }
  }
  top = block_max(top, lds);
  bad = block_max(bad, lds);
  t.some = top != -INFINITY || bad != 0.f;
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < kMaxK / kThreads; ++j)
    if (t.id[j] >= 0) s += exp2f((t.logq[j] - top) * kLog2e);
  s = block_sum(s, lds);
  const float l = top + log2f(s) * kLn2;
#pragma unroll
  for (int j = 0; j < kMaxK / kThreads; ++j) t.logq[j] -= l;
  return t;
}

template <typename T>
__device__ __forceinline__ void finish(const DistillArgs<T>& a, int64_t n, Sums v, float* lds) {
  const float lse1 = ref(v.m) + log2f(v.s1) * kLn2;
  const float lseT = a.warm ? ref(v.m) * a.inv_T + log2f(v.sT) * kLn2 : lse1;
  const T* row = a.Z + n * a.V;
  float loss = 0.f;
  if (a.w_kd != 0.f && a.K > 0) {
    const Teacher t = teacher(a, n, lds);
    float kd = 0.f;
#pragma unroll
    for (int j = 0; j < kMaxK / kThreads; ++j)
      if (t.id[j] >= 0) {
        const float q = exp2f(t.logq[j] * kLog2e);
        if (q != 0.f) kd += q * (t.logq[j] - (to_f32<T>(row[t.id[j]]) * a.inv_T - lseT));
      }
    kd = block_sum(kd, lds);
    if (t.some) loss = a.w_kd * kd;
  }
  if (threadIdx.x == 0) {
    const int y = a.labels ? a.labels[n] : -1;
    if (a.w_ce != 0.f && y >= 0 && y < a.V) loss += a.w_ce * (lse1 - to_f32<T>(row[y]));
    a.loss[n] = loss;
    a.stats[2 * n] = lse1;
    a.stats[2 * n + 1] = lseT;
  }
}

// A block takes a row, or a slice of one where there are few rows.
template <typename T, RowMode MODE>
__global__ __launch_bounds__(kThreads) void k_distill(DistillArgs<T> a) {
  __shared__ Sums sums[kThreads / 64];
  __shared__ float lds[kThreads / 64];
  const int64_t n = blockIdx.x / a.splits, c0 = blockIdx.x % a.splits * a.per, c1 = min(c0 + a.per, a.V);
  const T* row = a.Z + n * a.V;
  Sums v = {-INFINITY, 0.f, 0.f};
  const float cT = kLog2e * a.inv_T;
  for (int64_t c = c0 + 8 * threadIdx.x; c < c1; c += 8 * kThreads * kAhead) {
    Fetch<T, MODE> f[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) f[u].issue(row, c + 8 * kThreads * u < c1 ? c + 8 * kThreads * u : c, a.V);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t at = c + 8 * kThreads * u;
      if (at >= c1) break;
      const Raw8<T> r = f[u].value(at, a.V, true);
      float x[8], top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = at + i < c1 ? r.get(i) : -INFINITY;
        top = fmaxf(top, x[i]);
      }
      if (top > v.m) {
        const float g = v.m - top;
        v.s1 *= exp2f(g * kLog2e);
        v.sT *= exp2f(g * cT);
        v.m = top;
      }
      const float m = ref(v.m);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = x[i] - m;
        v.s1 += __builtin_amdgcn_exp2f(g * kLog2e);
        if (a.warm) v.sT += __builtin_amdgcn_exp2f(g * cT);
      }
    }
  }
  v = block_join(v, a.inv_T, sums);
  if (a.splits == 1) return finish(a, n, v, lds);
  if (threadIdx.x == 0) {
    float* p = a.part + 4 * int64_t(blockIdx.x);
    p[0] = v.m;
    p[1] = v.s1;
    p[2] = v.sT;
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_distill_join(DistillArgs<T> a) {
  __shared__ Sums sums[kThreads / 64];
  __shared__ float lds[kThreads / 64];
  const int64_t n = blockIdx.x;
  Sums v = {-INFINITY, 0.f, 0.f};
  for (int s = threadIdx.x; s < a.splits; s += kThreads) {
    const float* p = a.part + 4 * (n * a.splits + s);
    v = join(v, {p[0], p[1], p[2]}, a.inv_T);
  }
  finish(a, n, block_join(v, a.inv_T, sums), lds);
}

// The gradient: w1 (softmax(z) - 1[y]) + wT (softmax(z / T) - q).  The row's pass writes
// the softmaxes; the places of the label and of the teacher's entries are then
// written again, each by the thread of its first entry with everything that falls on
// it, from the logit read before the pass (gZ may be Z).
template <typename T, RowMode MODE>
__global__ __launch_bounds__(kThreads) void k_distill_bwd(DistillArgs<T> a) {
  __shared__ float lds[kThreads / 64];
  __shared__ int ids[kMaxK];
  __shared__ float qs[kMaxK];
  const int64_t n = blockIdx.x / a.splits, c0 = blockIdx.x % a.splits * a.per, c1 = min(c0 + a.per, a.V);
  const T* row = a.Z + n * a.V;
  T* out = a.gZ + n * a.V;
  const float g = a.gloss[n], lse1 = a.stats[2 * n], lseT = a.stats[2 * n + 1];
  const int label = a.labels ? a.labels[n] : -1;
  const bool has1 = a.w_ce != 0.f && label >= 0 && label < a.V;
  const float w1 = has1 ? a.w_ce * g : 0.f;
  float wT = 0.f, z[kMaxK / kThreads];
  bool mine[kMaxK / kThreads], hasT = false;
  if (a.w_kd != 0.f && a.K > 0) {
    const Teacher t = teacher(a, n, lds);
    hasT = t.some;
    if (hasT) wT = a.w_kd * a.inv_T * g;
#pragma unroll
    for (int j = 0; j < kMaxK / kThreads; ++j) {
      const int k = threadIdx.x + kThreads * j;
      mine[j] = hasT && t.id[j] >= c0 && t.id[j] < c1;
      z[j] = mine[j] ? to_f32<T>(row[t.id[j]]) : 0.f;
      if (k < a.K) {
        ids[k] = t.id[j];
        qs[k] = t.id[j] >= 0 ? exp2f(t.logq[j] * kLog2e) : 0.f;
      }
    }
  }
  const bool label_here = has1 && label >= c0 && label < c1 && threadIdx.x == 0;
  const float zy = label_here ? to_f32<T>(row[label]) : 0.f;
  __syncthreads();
  const auto p1 = [&](float x) { return __builtin_amdgcn_exp2f((x - lse1) * kLog2e); };
  const auto pT = [&](float x) { return __builtin_amdgcn_exp2f(fmaf(x, a.inv_T, -lseT) * kLog2e); };
  const bool one = !a.warm;  // one softmax serves both terms
  const float ws = w1 + wT;
  for (int64_t c = c0 + 8 * threadIdx.x; c < c1; c += 8 * kThreads * kAhead) {
    Fetch<T, MODE> f[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) f[u].issue(row, c + 8 * kThreads * u < c1 ? c + 8 * kThreads * u : c, a.V);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t at = c + 8 * kThreads * u;
      if (at >= c1) break;
      const Raw8<T> r = f[u].value(at, a.V, true);
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = r.get(i);
        if (one)
          x[i] = has1 || hasT ? ws * p1(y) : 0.f;
        else
          x[i] = (has1 ? w1 * p1(y) : 0.f) + (hasT ? wT * pT(y) : 0.f);
      }
      put_row<MODE>(out, at, min(c1, a.V), true, x);
    }
  }
  __syncthreads();
  const auto put = [&](int id, float x, float q, bool y) {
    float v = (has1 ? w1 * (p1(x) - (y ? 1.f : 0.f)) : 0.f);
    if (hasT) v += wT * ((one ? p1(x) : pT(x)) - q);
    out[id] = from_f32<T>(v);
  };
  bool taken = false;  // the label is one of the teacher's entries
  if (hasT) {
#pragma unroll
    for (int j = 0; j < kMaxK / kThreads; ++j) {
      if (!mine[j]) continue;
      const int k = threadIdx.x + kThreads * j, id = ids[k];
      float q = 0.f;
      bool firstOf = true;
      for (int e = 0; e < a.K; ++e) {
        if (ids[e] != id) continue;
        firstOf = firstOf && e >= k;
        q += qs[e];
      }
      if (firstOf) put(id, z[j], q, has1 && id == label);
    }
    if (label_here)
      for (int e = 0; e < a.K; ++e) taken = taken || ids[e] == label;
  }
  if (label_here && !taken) put(label, zy, 0.f, true);
}

// ------------------------------------------------------------------- launches --
// Blocks of a row: one where the rows alone fill the card.
int split(int64_t N, int64_t V) {
  const int64_t want = (1024 + N - 1) / N, most = (V + kSlice - 1) / kSlice;
  return int(std::max<int64_t>(1, std::min(want, most)));
}

template <typename T>
DistillArgs<T> make_args(const Distill& c, float* ws) {
  DistillArgs<T> a;
  a.Z = static_cast<const T*>(c.Z);
  a.labels = c.labels;
  a.t_ids = c.t_ids;
  a.t_logits = c.t_logits;
  a.gloss = c.gloss;
  a.loss = c.loss;
  a.stats = c.stats;
  a.part = ws;
  a.gZ = static_cast<T*>(c.gZ);
  a.inv_T = 1.f / c.temperature;
  a.warm = c.temperature != 1.f;
  a.w_ce = c.w_ce;
  a.w_kd = c.w_kd;
  a.N = c.N;
  a.V = c.V;
  a.K = int(c.K);
  const int s = split(c.N, c.V);
  a.per = ((c.V + s - 1) / s + 7) / 8 * 8;
  a.splits = int((c.V + a.per - 1) / a.per);
  return a;
}

template <typename T>
void distill_t(const Distill& c, float* ws, hipStream_t s) {
  const DistillArgs<T> a = make_args<T>(c, ws);
  by_row_mode<T, true>(a.V, {a.Z}, [&](auto m) {
    hipLaunchKernelGGL((k_distill<T, decltype(m)::value>), dim3(uint32_t(a.N * a.splits)), dim3(kThreads), 0, s, a);
  });
  if (a.splits > 1) hipLaunchKernelGGL((k_distill_join<T>), dim3(uint32_t(a.N)), dim3(kThreads), 0, s, a);
}
template <typename T>
void distill_bwd_t(const Distill& c, hipStream_t s) {
  const DistillArgs<T> a = make_args<T>(c, nullptr);
  by_row_mode<T, true>(a.V, {a.Z, a.gZ}, [&](auto m) {
    hipLaunchKernelGGL((k_distill_bwd<T, decltype(m)::value>), dim3(uint32_t(a.N * a.splits)), dim3(kThreads), 0, s, a);
  });
}

}  // namespace

size_t distill_ws_bytes(int64_t N, int64_t V) {
  const int s = split(N, V);
  return s > 1 ? size_t(4) * N * s * sizeof(float) : 0;
}
void launch_distill(const Distill& c, int bf16, float* ws, hipStream_t s) {
  (bf16 ? distill_t<bf16_t> : distill_t<float>)(c, ws, s);
}
void launch_distill_bwd(const Distill& c, int bf16, hipStream_t s) {
  (bf16 ? distill_bwd_t<bf16_t> : distill_bwd_t<float>)(c, s);
}

}  // namespace mapl
