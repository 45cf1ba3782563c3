// The last stage's loss: cross-entropy with the labels and the divergence from a
// teacher's top logits, and its gradient.  Formulas: include/mapl_block.h.  Both are
// bound by the logits' traffic: one read of them, and for the gradient one write.
#include "internal.h"
#include "vec8.h"

namespace mapl {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kAhead = 4;  // vectors of 8 logits in flight per thread
constexpr int kMaxK = 1024;

template <typename T>
struct DistillArgs {
  const T* Z;
  const int32_t *labels, *t_ids;
  const float *t_logits, *gloss;
  float *loss, *stats, *part;  // part [N][splits][4]: reference, the two sums
  T* gZ;
  float inv_T, w_ce, w_kd;
  bool warm;  // temperature other than 1: two sums
  int64_t N, V, per;  // per: logits of a block
  int K, splits;
};

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float lg2(float x) { return __builtin_amdgcn_logf(x); }

// Sums of exp(z - m) and exp((z - m) / T) for the largest logit m so far.
struct Sums {
  float m, s1, sT;
};
// a largest logit of -inf stands for no finite one: nothing is scaled by it
__device__ __forceinline__ float ref(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ float shift(float from, float to, float c) {  // the factor of a change of m
  return from == to ? 1.f : ex2((from - to) * c);
}
__device__ __forceinline__ Sums join(Sums x, Sums y, float c, float cT) {
  const float m = fmaxf(x.m, y.m);
  return {m, x.s1 * shift(x.m, m, c) + y.s1 * shift(y.m, m, c), x.sT * shift(x.m, m, cT) + y.sT * shift(y.m, m, cT)};
}

// over the block, the same in every thread
template <int THREADS>
__device__ __forceinline__ Sums block_join(Sums v, float c, float cT, Sums* lds) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1)
    v = join(v, {__shfl_xor(v.m, s), __shfl_xor(v.s1, s), __shfl_xor(v.sT, s)}, c, cT);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) v = join(v, lds[w], c, cT);
  return v;
}
template <int THREADS, typename F>
__device__ __forceinline__ float block_all(float v, float* lds, F f) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) v = f(v, __shfl_xor(v, s));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) v = f(v, lds[w]);
  return v;
}
__device__ __forceinline__ float sum2(float x, float y) { return x + y; }
__device__ __forceinline__ float max2(float x, float y) { return fmaxf(x, y); }

// The teacher's entries k = threadIdx.x + THREADS j of a row: their ids (-1: none), their
// logits and the student's logits there.  An entry with a logit of -inf has none.
// Everything that memory has to bring is asked for at once, and early.
template <typename T, int THREADS>
struct Teacher {
  static constexpr int J = kMaxK / THREADS;
  int id[J];
  float x[J], z[J];
  __device__ __forceinline__ void load(const DistillArgs<T>& a, int64_t n) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int k = threadIdx.x + THREADS * j;
      id[j] = -1;
      x[j] = -INFINITY;
      if (THREADS * j < a.K) {
        const int64_t at = n * a.K + min(k, a.K - 1);
        const int i = a.t_ids[at];
        x[j] = a.t_logits[at];
        if (k < a.K && i >= 0 && i < a.V && x[j] != -INFINITY) id[j] = i;
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (THREADS * j < a.K) z[j] = to_f32<T>(a.Z[n * a.V + max(id[j], 0)]);
  }
  // the probabilities e / s of the entries, e = exp((x - top) / T); s = 0: no entry
  __device__ __forceinline__ float norm(const DistillArgs<T>& a, float* lds, float& top, float (&e)[J]) {
    top = -INFINITY;
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (THREADS * j < a.K && id[j] >= 0) top = fmaxf(top, x[j]);
    top = block_all<THREADS>(top, lds, max2);
    const float cT = kLog2e * a.inv_T;
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      e[j] = THREADS * j < a.K && id[j] >= 0 ? ex2((x[j] - top) * cT) : 0.f;
      s += e[j];
    }
    return block_all<THREADS>(s, lds + 16, sum2);
  }
};

// Log-sums and logits enter the loss as differences from the largest logit, the teacher's
// from its own: rounded beside a common offset they would lose the loss.
template <typename T, int THREADS>
__device__ __forceinline__ void finish(const DistillArgs<T>& a, int64_t n, Sums v, const Teacher<T, THREADS>& t, float zy,
                                       bool label, float* lds) {
  const float m = ref(v.m), log1 = lg2(v.s1) * kLn2, logT = a.warm ? lg2(v.sT) * kLn2 : log1;
  float loss = 0.f;
  if (a.w_kd != 0.f && a.K > 0) {
    Teacher<T, THREADS> u = t;
    float e[Teacher<T, THREADS>::J], top, kd = 0.f;
    const float s = u.norm(a, lds, top, e), l = lg2(s) * kLn2;
#pragma unroll
    for (int j = 0; j < Teacher<T, THREADS>::J; ++j)
      if (THREADS * j < a.K && e[j] != 0.f) kd += e[j] * (((u.x[j] - top) * a.inv_T - l) - ((u.z[j] - m) * a.inv_T - logT));
    kd = block_all<THREADS>(kd, lds + 32, sum2);
    if (s != 0.f) loss = a.w_kd * (kd / s);
  }
  if (threadIdx.x == 0) {
    if (label) loss += a.w_ce * ((m - zy) + log1);
    a.loss[n] = loss;
    const float lse1 = fmaf(lg2(v.s1), kLn2, m);
    a.stats[2 * n] = lse1;
    a.stats[2 * n + 1] = a.warm ? fmaf(lg2(v.sT), kLn2, m * a.inv_T) : lse1;
  }
}

// A block takes a row, or a slice of one where there are few rows.  The teacher's entries
// and the logits at them are asked for before the row's pass, whose traffic then hides
// their latency.  Both sums in one pass, by a running maximum as the reference; about 10
// vector operations a logit, two of them exp, which take 130 us of 16384 x 32000 bf16 beside the 186
// of its read: 220-235 us (4.5-4.8 TB/s).  Without the sums the same loads take 177; vectors
// asked for a turn ahead do not help (231 for 223), and whole turns without their bounds
// by 3 us.  4 x 32000 fp32: 9.7 us.
template <typename T, RowMode MODE, int THREADS>
__global__ __launch_bounds__(THREADS) void k_distill(DistillArgs<T> a) {
  __shared__ Sums sums[THREADS / 64];
  __shared__ float lds[48];
  const int64_t n = blockIdx.x / a.splits, c0 = blockIdx.x % a.splits * a.per, c1 = min(c0 + a.per, a.V);
  const T* row = a.Z + n * a.V;
  Teacher<T, THREADS> t;
  float zy = 0.f;
  bool label = false;
  if (a.splits == 1) {
    if (a.w_kd != 0.f && a.K > 0) t.load(a, n);
    const int y = a.labels ? a.labels[n] : -1;
    label = a.w_ce != 0.f && y >= 0 && y < a.V;
    if (label) zy = to_f32<T>(row[y]);
  }
  Sums v = {-INFINITY, 0.f, 0.f};
  float c = kLog2e, cT = kLog2e * a.inv_T;
  asm("" : "+v"(c), "+v"(cT));  // an operand in a vector register: twice the rate of a scalar one
  constexpr int STEP = 8 * THREADS;
  for (int64_t at = c0 + 8 * threadIdx.x; at < c1; at += STEP * kAhead) {
    Fetch<T, MODE> f[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) f[u].issue(row, at + STEP * u < c1 ? at + STEP * u : at, a.V);
    float x[kAhead][8], top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const Raw8<T> r = f[u].value(at + STEP * u, a.V, true);
      const int left = int(min(max(c1 - at - STEP * u, int64_t(0)), int64_t(8)));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[u][i] = (MODE == kVec ? left > 0 : i < left) ? r.get(i) : -INFINITY;
        top = fmaxf(top, x[u][i]);
      }
    }
    if (top > v.m) {
      v.s1 *= shift(v.m, top, c);
      if (a.warm) v.sT *= shift(v.m, top, cT);
      v.m = top;
    }
    // the difference first: exact for a row of one value, the type's lowest too
    const float m = ref(v.m);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[u][i] -= m;
        s[i & 1] += ex2(x[u][i] * c);
      }
    v.s1 += s[0] + s[1];
    if (a.warm) {
      s[0] = s[1] = 0.f;
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i & 1] += ex2(x[u][i] * cT);
      v.sT += s[0] + s[1];
    }
  }
  v = block_join<THREADS>(v, c, cT, sums);
  if (a.splits == 1) return finish<T, THREADS>(a, n, v, t, zy, label, lds);
  if (threadIdx.x == 0) {
    float* p = a.part + 4 * int64_t(blockIdx.x);
    p[0] = v.m;
    p[1] = v.s1;
    p[2] = v.sT;
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_distill_join(DistillArgs<T> a) {
  __shared__ Sums sums[4];
  __shared__ float lds[48];
  const int64_t n = blockIdx.x;
  const float c = kLog2e, cT = kLog2e * a.inv_T;
  Teacher<T, 256> t;
  if (a.w_kd != 0.f && a.K > 0) t.load(a, n);
  const int y = a.labels ? a.labels[n] : -1;
  const bool label = a.w_ce != 0.f && y >= 0 && y < a.V;
  const float zy = label ? to_f32<T>(a.Z[n * a.V + y]) : 0.f;
  Sums v = {-INFINITY, 0.f, 0.f};
  for (int s = threadIdx.x; s < a.splits; s += 256) {
    const float* p = a.part + 4 * (n * a.splits + s);
    v = join(v, {p[0], p[1], p[2]}, c, cT);
  }
  finish<T, 256>(a, n, block_join<256>(v, c, cT, sums), t, zy, label, lds);
}

// The gradient: w1 (softmax(z) - 1[y]) + wT (softmax(z / T) - q).  The row's pass writes
// the softmaxes; the places of the label and of the teacher's entries are then
// written again, each by the thread of its first entry with everything that falls on
// it, from the logit read before the pass (gZ may be Z).  Bound by memory: 8192 x 32000 bf16
// 256 us (4.1 TB/s read and written, a large copy 4.9), 777 x 32003 fp32 39 us (5.1, some of it
// from the last-level cache).
template <typename T, RowMode MODE, int THREADS>
__global__ __launch_bounds__(THREADS) void k_distill_bwd(DistillArgs<T> a) {
  constexpr int J = Teacher<T, THREADS>::J, STEP = 8 * THREADS;
  __shared__ float lds[48];
  __shared__ __attribute__((aligned(16))) int ids[kMaxK];
  __shared__ __attribute__((aligned(16))) float qs[kMaxK];
  __shared__ float zs[kMaxK], zl;
  const int64_t n = blockIdx.x / a.splits, c0 = blockIdx.x % a.splits * a.per, c1 = min(c0 + a.per, a.V);
  const T* row = a.Z + n * a.V;
  T* out = a.gZ + n * a.V;
  Teacher<T, THREADS> t;
  const bool kd = a.w_kd != 0.f && a.K > 0;
  if (kd) t.load(a, n);
  const float g = a.gloss[n], lse1 = a.stats[2 * n], lseT = a.stats[2 * n + 1];
  const int label = a.labels ? a.labels[n] : -1;
  const bool has1 = a.w_ce != 0.f && label >= 0 && label < a.V;
  const float zy = has1 ? to_f32<T>(row[label]) : 0.f;
  int64_t at = c0 + 8 * threadIdx.x;
  Fetch<T, MODE> f[kAhead];
  const auto issue = [&] {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) f[u].issue(row, at + STEP * u < c1 ? at + STEP * u : c0, a.V);
  };
  issue();
  const float w1 = has1 ? a.w_ce * g : 0.f;
  float wT = 0.f;
  bool hasT = false;
  if (kd) {
    float e[J], top;
    const float s = t.norm(a, lds, top, e);
    hasT = s != 0.f;
    if (hasT) {
      wT = a.w_kd * a.inv_T * g;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int k = threadIdx.x + THREADS * j;
        if (THREADS * j < a.K && k < ((a.K + 3) & ~3)) {  // whole fours
          ids[k] = t.id[j];
          qs[k] = e[j] / s;
          zs[k] = t.z[j];
        }
      }
    }
  }
  if (threadIdx.x == 0) zl = zy;
  __syncthreads();  // the logits that are looked at again have been read before any is overwritten
  const auto p1 = [&](float x) { return ex2((x - lse1) * kLog2e); };
  const auto pT = [&](float x) { return ex2(fmaf(x, a.inv_T, -lseT) * kLog2e); };
  const bool one = !a.warm;  // one softmax serves both terms
  const bool none = !has1 && !hasT;
  const float ws = w1 + wT;
  while (at < c1) {
    float x[kAhead][8];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const Raw8<T> r = f[u].value(at + STEP * u, a.V, at + STEP * u < c1);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[u][i] = r.get(i);
    }
    const int64_t here = at;
    at += STEP * kAhead;
    if (at < c1) issue();
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = x[u][i];
        if (one)
          x[u][i] = none ? 0.f : ws * p1(y);
        else
          x[u][i] = (has1 ? w1 * p1(y) : 0.f) + (hasT ? wT * pT(y) : 0.f);
      }
      put_row<MODE>(out, here + STEP * u, a.V, here + STEP * u < c1, x[u]);
    }
  }
  __syncthreads();
  const auto put = [&](int id, float x, float q, bool y) {
    float v = has1 ? w1 * (p1(x) - (y ? 1.f : 0.f)) : 0.f;
    if (hasT) v += wT * ((one ? p1(x) : pT(x)) - q);
    out[id] = from_f32<T>(v);
  };
  if (hasT) {
    typedef int i32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (THREADS * j >= a.K) break;
      const int k = threadIdx.x + THREADS * j, id = t.id[j];
      if (!(id >= c0 && id < c1)) continue;
      float q = 0.f;
      int earliest = k;  // of the entries with this id
      for (int e = ((a.K + 3) & ~3) - 4; e >= 0; e -= 4) {
        const i32x4 i4 = *reinterpret_cast<const i32x4*>(ids + e);
        const f32x4 q4 = *reinterpret_cast<const f32x4*>(qs + e);
#pragma unroll
        for (int x = 3; x >= 0; --x)
          if (i4[x] == id) {
            q += q4[x];
            earliest = min(earliest, e + x);
          }
      }
      if (earliest == k) put(id, zs[k], q, has1 && id == label);
    }
  }
  if (has1 && label >= c0 && label < c1 && threadIdx.x == 0) {
    bool taken = false;  // the label is one of the teacher's entries
    if (hasT)
      for (int e = 0; e < a.K; ++e) taken = taken || ids[e] == label;
    if (!taken) put(label, zl, 0.f, true);
  }
}

// ------------------------------------------------------------------- launches --
// Rows that fill the card have a block of 256 threads each.  Fewer have one of 1024, and
// where those leave half of the CUs without work and a row is long, a row is split into
// slices of 32768 logits at least, where the launch that joins them is paid for (4 rows of fp32:
// 65536 logits 11.5 us in two, 12.3 whole; 131072 11.6 in four, 17.7 whole; slices of 16384 the same).
constexpr int64_t kManyRows = 1024, kSlice = 32768;
int split(int64_t N, int64_t V) {
  const int64_t want = (128 + N - 1) / N, most = V / kSlice;
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
  return a;
}
template <typename T>
void cut(DistillArgs<T>& a, int s) {  // into s slices of whole vectors, or a few less
  a.per = ((a.V + s - 1) / s + 7) / 8 * 8;
  a.splits = int((a.V + a.per - 1) / a.per);
}

template <typename T>
void distill_t(const Distill& c, float* ws, hipStream_t s) {
  DistillArgs<T> a = make_args<T>(c, ws);
  cut(a, split(a.N, a.V));
  const dim3 grid(uint32_t(a.N * a.splits));
  by_row_mode<T, true>(a.V, {a.Z}, [&](auto m) {
    if (a.N >= kManyRows)
      hipLaunchKernelGGL((k_distill<T, decltype(m)::value, 256>), grid, dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((k_distill<T, decltype(m)::value, 1024>), grid, dim3(1024), 0, s, a);
  });
  if (a.splits > 1) hipLaunchKernelGGL((k_distill_join<T>), dim3(uint32_t(a.N)), dim3(256), 0, s, a);
}
template <typename T>
void distill_bwd_t(const Distill& c, hipStream_t s) {
  DistillArgs<T> a = make_args<T>(c, nullptr);
  cut(a, int(std::max<int64_t>(1, std::min((kManyRows + a.N - 1) / a.N, a.V / 4096))));
  by_row_mode<T, true>(a.V, {a.Z, a.gZ}, [&](auto m) {
    hipLaunchKernelGGL((k_distill_bwd<T, decltype(m)::value, 256>), dim3(uint32_t(a.N * a.splits)), dim3(256), 0, s, a);
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
