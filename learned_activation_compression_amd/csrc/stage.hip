// The edge of a transformer block at a pipeline stage: dropout from a
// counter-based generator, and the fused norm - gate - residual - norm with its
// backward pass.  Formulas: include/mapl_stage.h.  All of it is bound by memory
// traffic: every tensor is read or written once, rows stay in registers between
// their sums and their use.
#include <type_traits>

#include "internal.h"
#include "vec8.h"

namespace mapl {
namespace {

// ----------------------------------------------------------------- generator --
struct Drop {
  uint64_t offset;
  uint32_t k0, k1;  // the seed
  uint32_t t;       // keep where the 16-bit value is >= t; 0: no dropout
  float scale;
};

// Philox4x32-10 (Salmon et al., SC 2011) at (c0, c1, c2, 0): 8 values of 16 bits.
__device__ __forceinline__ u32x4 philox(uint32_t c0, uint64_t row, uint32_t k0, uint32_t k1) {
  uint32_t c1 = static_cast<uint32_t>(row), c2 = static_cast<uint32_t>(row >> 32), c3 = 0;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c0, b = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// bit i: element i of the 8 columns at 8 * c8 of row n is kept
__device__ __forceinline__ uint32_t keep8(const Drop& dr, uint32_t c8, uint64_t n) {
  const u32x4 w = philox(c8, dr.offset + n, dr.k0, dr.k1);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m |= ((w[i] & 0xffffu) >= dr.t ? 1u : 0u) << (2 * i);
    m |= ((w[i] >> 16) >= dr.t ? 1u : 0u) << (2 * i + 1);
  }
  return m;
}

Drop make_drop(double p, uint64_t seed, uint64_t offset) {
  Drop d;
  d.offset = offset;
  d.k0 = static_cast<uint32_t>(seed);
  d.k1 = static_cast<uint32_t>(seed >> 32);
  d.t = static_cast<uint32_t>(p * 65536.0 + 0.5);
  d.scale = d.t < 65536 ? 65536.f / float(65536 - d.t) : 0.f;
  return d;
}

// ------------------------------------------------------------------- dropout --
// Units of 8 columns, unit u = row * nb + column / 8: one generator call each, 20
// products of 32 by 32 bits for 16 bits an element, which hides behind the traffic:
// 16384 x 1024 bf16 out of memory in 12.2 us, 5.5 TB/s, as a copy (a fifth more with
// two calls, 32 bits an element).
constexpr int kDropUnits = 4;  // units in flight per thread

template <typename T, RowMode MODE>
__global__ __launch_bounds__(256) void k_dropout(const T* X, T* Y, Drop dr, int64_t units, uint32_t nb, int64_t d) {
  const int64_t u0 = int64_t(blockIdx.x) * (256 * kDropUnits) + threadIdx.x;
  int64_t row[kDropUnits];
  uint32_t b[kDropUnits], keep[kDropUnits];
  row[0] = u0 / nb;
  b[0] = static_cast<uint32_t>(u0 - row[0] * nb);
  const uint32_t step_row = 256 / nb, step_b = 256 % nb;
  Fetch<T, MODE> x[kDropUnits];
#pragma unroll
  for (int k = 0; k < kDropUnits; ++k) {
    if (k > 0) {
      row[k] = row[k - 1] + step_row;
      b[k] = b[k - 1] + step_b;
      if (b[k] >= nb) {
        b[k] -= nb;
        ++row[k];
      }
    }
    x[k].issue(X + (u0 + k * 256 < units ? row[k] : 0) * d, int64_t(b[k]) * 8, d);
  }
#pragma unroll
  for (int k = 0; k < kDropUnits; ++k) keep[k] = dr.t ? keep8(dr, b[k], static_cast<uint64_t>(row[k])) : 0xffu;
#pragma unroll
  for (int k = 0; k < kDropUnits; ++k) {
    const bool in = u0 + k * 256 < units;
    const Raw8<T> r = x[k].value(int64_t(b[k]) * 8, d, in);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (keep[k] >> i) & 1 ? r.get(i) * dr.scale : 0.f;
    put_row<MODE>(Y + row[k] * d, int64_t(b[k]) * 8, d, in, v);
  }
}

// ------------------------------------------------------------------ norm edge --
// A slot of TPR threads holds a row, V vectors of 8 columns per thread (vector
// j of thread l starts at column 8 * (j * TPR + l)); a block has 256 threads, or
// one slot's where 256 is no multiple of it.
template <int TPR>
constexpr int kBlock = 256 % TPR == 0 ? 256 : TPR;

// Sum over the lanes of a slot (or of its wave), the same value and order in
// every lane: data-parallel primitives within 16 lanes, lane swaps beyond.
template <int L>
__device__ __forceinline__ float lane_sum(float v) {
  static_assert(L == 16 || L == 32 || L == 64, "lanes");
  const auto dpp = [](float x, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  v += dpp(v, std::integral_constant<int, 0xB1>{});   // lanes 1 0 3 2 of a quad
  v += dpp(v, std::integral_constant<int, 0x4E>{});   // lanes 2 3 0 1 of a quad
  v += dpp(v, std::integral_constant<int, 0x141>{});  // 8 lanes mirrored
  v += dpp(v, std::integral_constant<int, 0x140>{});  // 16 lanes mirrored
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// K sums over a slot at once.  A slot of several waves exchanges them through
// lds[2][K][16]; `turn` alternates its halves, so that one barrier is enough.
template <int TPR, int K>
__device__ __forceinline__ void slot_sums(float (&v)[K], float* lds, int& turn) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane_sum<(TPR < 64 ? TPR : 64)>(v[k]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float* at = lds + (turn & 1) * (3 * 16);
    ++turn;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) at[k * 16 + (threadIdx.x >> 6)] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v[k] += at[k * 16 + threadIdx.x / TPR * W + w];
    }
  }
}

// 1 / sqrt(x) from the hardware's estimate (one unit in the last place) and one
// Newton step, once a row: the estimate's error would be common to the whole row.
__device__ __forceinline__ float inv_sqrt(float x) {
  const float r = rsqrtf(x);
  return x < 3.0e38f ? fmaf(0.5f * r, fmaf(-(x * r), r, 1.f), r) : r;
}

template <typename T>
struct NormArgs {
  const T *X, *Y, *w_post, *gate, *w_pre;
  T *X_out, *H;
  float res_scale, eps, inv_d;
  Drop dr;
  int64_t N, rows_per_gate;
  int d;
};

// Bound by its traffic, two tensors in and two out: 16384 x 1024 bf16 out of memory
// in 25.8 us (5.2 TB/s) without and 28 us (4.8 TB/s) with dropout, whose generator
// does not quite hide; 8192 x 2048 in 28.4 us.  All loads of a row, weights included,
// are issued before the first sum; the weights come from the caches.
template <typename T, int TPR, int V, RowMode MODE>
__global__ __launch_bounds__(kBlock<TPR>) void k_stage_norm(NormArgs<T> a) {
  constexpr int S = kBlock<TPR> / TPR;
  __shared__ float lds[2 * 3 * 16];
  int turn = 0;
  const int l = threadIdx.x % TPR;
  const auto col = [&](int j) { return 8 * (j * TPR + l); };
  // every thread of a block takes the same number of turns (slot_sums has barriers)
  for (int64_t n0 = int64_t(blockIdx.x) * S; n0 < a.N; n0 += int64_t(gridDim.x) * S) {
    const int64_t n = n0 + threadIdx.x / TPR;
    const bool in = n < a.N;
    const int64_t at = (in ? n : 0) * a.d;
    Fetch<T, MODE> fx[V], fy[V], fg[V];
    Fetch<T, MODE == kOdd ? kAny : MODE> fq[V], fw[V];
#pragma unroll
    for (int j = 0; j < V; ++j) fx[j].issue(a.X + at, col(j), a.d);
    if (a.Y) {
#pragma unroll
      for (int j = 0; j < V; ++j) fy[j].issue(a.Y + at, col(j), a.d);
    }
    if (a.w_post) {
#pragma unroll
      for (int j = 0; j < V; ++j) fq[j].issue(a.w_post, col(j), a.d);
    }
    if (a.gate) {
      const T* g = a.gate + (in ? n / a.rows_per_gate : 0) * a.d;
#pragma unroll
      for (int j = 0; j < V; ++j) fg[j].issue(g, col(j), a.d);
    }
    if (a.H) {
#pragma unroll
      for (int j = 0; j < V; ++j) fw[j].issue(a.w_pre, col(j), a.d);
    }
    float x[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Raw8<T> r = fx[j].value(col(j), a.d, in);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = a.res_scale * r.get(i);
    }
    if (a.Y) {
      float u[V][8], s[1] = {0.f};
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const Raw8<T> r = fy[j].value(col(j), a.d, in);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[j][i] = r.get(i);
        if (a.dr.t) {
          const uint32_t keep = keep8(a.dr, static_cast<uint32_t>(j * TPR + l), static_cast<uint64_t>(n));
#pragma unroll
          for (int i = 0; i < 8; ++i) u[j][i] = (keep >> i) & 1 ? u[j][i] * a.dr.scale : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += u[j][i] * u[j][i];
      }
      if (a.w_post) {
        slot_sums<TPR>(s, lds, turn);
        const float q = inv_sqrt(s[0] * a.inv_d + a.eps);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const Raw8<T> w = fq[j].value(col(j), a.d, true);
#pragma unroll
          for (int i = 0; i < 8; ++i) u[j][i] *= q * w.get(i);
        }
      }
      if (a.gate) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const Raw8<T> w = fg[j].value(col(j), a.d, true);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[j][i] += w.get(i) * u[j][i];
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) x[j][i] += u[j][i];
      }
    }
    if (a.X_out) {
#pragma unroll
      for (int j = 0; j < V; ++j) put_row<MODE>(a.X_out + at, col(j), a.d, in, x[j]);
    }
    if (a.H) {
      float s[1] = {0.f};
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += col(j) + i < a.d ? x[j][i] * x[j][i] : 0.f;
      slot_sums<TPR>(s, lds, turn);
      const float r = inv_sqrt(s[0] * a.inv_d + a.eps);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const Raw8<T> w = fw[j].value(col(j), a.d, true);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] *= r * w.get(i);
        put_row<MODE>(a.H + at, col(j), a.d, in, x[j]);
      }
    }
  }
}

// ------------------------------------------------------------------- backward --
// The rows are split over blocks, and a block's rows over its slots, both into
// contiguous runs, so that the sums over rows have a fixed order.
//  - few gate rows (or no gate), or gate rows of more than kBwdRun rows: a
//    block's rows lie in one gate row; `bpg` blocks share a gate row.  Each block
//    leaves one partial row of every weight gradient, and k_stage_norm_grads
//    joins them.
//  - many gate rows (a gate per token): a slot takes `gps` whole gate rows, of
//    kBwdRun rows at most, and writes their gradients itself.
struct BwdSplit {
  int64_t blocks, bpg, rows_per_block, gps;
  bool many;
};

template <typename T>
struct NormBwdArgs {
  const T *gX_out, *gH, *X_out, *Y, *w_post, *gate, *w_pre;
  T *gX, *gY;
  float *g_gate, *part;  // part [3][blocks][d]: w_post, gate, w_pre
  float res_scale, eps, inv_d;
  Drop dr;
  BwdSplit sp;
  int64_t N, rows_per_gate;
  int d, accumulate;
};

// PRE: with gH and X_out; POST: with Y; MANY: many gate rows.
//
// Four tensors in, two out, and the three weights' sums in registers.  One row is
// four dependent steps (load, sums, gX and the dot product of gY, gY), so the loads
// of the next row are issued before this row's arithmetic: 16384 x 1024 bf16 in 40
// us (5.0 TB/s), against 84 us with each row loaded when its turn comes.  512 blocks,
// two a CU (three would fit a CU's registers at that width): with 768 and 1024 of
// them the call takes 40.3 and 44.1 instead of 39.7 us, for 8192 x 2048 41.2 and
// 45.2 instead of 39.0 (the same tensors again and again).
template <typename T, int TPR, int V, bool PRE, bool POST, bool MANY, RowMode MODE>
__global__ __launch_bounds__(kBlock<TPR>) void k_stage_norm_bwd(NormBwdArgs<T> a) {
  constexpr int S = kBlock<TPR> / TPR;
  __shared__ float lds[2 * 3 * 16];
  __shared__ float acc_lds[S > 1 ? 256 * 8 : 1];
  int turn = 0;
  const int l = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  int64_t r0, r1, turns;  // this slot's rows; the block's turns
  if constexpr (MANY) {
    const int64_t g0 = (int64_t(blockIdx.x) * S + slot) * a.sp.gps;
    r0 = min(g0 * a.rows_per_gate, a.N);
    r1 = min((g0 + a.sp.gps) * a.rows_per_gate, a.N);
    turns = a.sp.gps * a.rows_per_gate;
  } else {
    const int64_t g = blockIdx.x / a.sp.bpg, part = blockIdx.x % a.sp.bpg;
    const int64_t b0 = g * a.rows_per_gate + min(part * a.sp.rows_per_block, a.rows_per_gate);
    const int64_t b1 = g * a.rows_per_gate + min((part + 1) * a.sp.rows_per_block, a.rows_per_gate);
    turns = (a.sp.rows_per_block + S - 1) / S;
    r0 = min(b0 + slot * turns, b1);
    r1 = min(b0 + (slot + 1) * turns, b1);
  }
  const bool norm = a.w_post != nullptr;
  const auto col = [&](int j) { return 8 * (j * TPR + l); };
  const auto weight = [&](Raw8<T>& w, const T* p, int j) {
    Fetch<T, MODE> f;
    f.issue(p, col(j), a.d);
    w = f.value(col(j), a.d, true);
  };
  // the weights stay in registers; an absent one is 1
  Raw8<T> wq[V], wp[V], wg[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    wp[j].ones();
    wg[j].ones();
    if constexpr (PRE) weight(wq[j], a.w_pre, j);
    if (POST && norm) weight(wp[j], a.w_post, j);
    if (POST && !MANY && a.gate) weight(wg[j], a.gate + blockIdx.x / a.sp.bpg * a.d, j);
  }
  struct Row {
    Fetch<T, MODE> t[V], h[V], x[V], y[V], g[V];
  };
  const T* gxo = a.gX_out ? a.gX_out : a.gH;  // without gX_out: read something, use zero
  const bool has_t = a.gX_out != nullptr;
  const auto load = [&](Row& r, int64_t n) {
    const bool in = n < r1;
    const int64_t at = (in ? n : 0) * a.d;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      r.t[j].issue(gxo + at, col(j), a.d);
      if constexpr (PRE) r.h[j].issue(a.gH + at, col(j), a.d);
      if constexpr (PRE) r.x[j].issue(a.X_out + at, col(j), a.d);
      if constexpr (POST) r.y[j].issue(a.Y + at, col(j), a.d);
      if constexpr (MANY) r.g[j].issue(a.gate + (in ? n / a.rows_per_gate : 0) * a.d, col(j), a.d);
    }
  };
  float Q[V][8], Wp[V][8], Hp[V][8];  // sums over rows of t q u (this gate row's), gate t q u (MANY), gH r X_out
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) Q[j][i] = Wp[j][i] = Hp[j][i] = 0.f;

  Row cur, nxt;
  load(cur, r0);
  for (int64_t k = 0; k < turns; ++k) {
    const int64_t n = r0 + k;
    const bool in = n < r1;
    load(nxt, n + 1 < r0 + turns ? n + 1 : r1);
    float t[V][8], u[V][8], s[3] = {0.f, 0.f, 0.f};
    uint32_t keep[V];
    Raw8<T> rt[V], rh[V], rx[V], rg[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      rt[j] = cur.t[j].value(col(j), a.d, in);
      if constexpr (PRE) {
        rh[j] = cur.h[j].value(col(j), a.d, in);
        rx[j] = cur.x[j].value(col(j), a.d, in);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[0] += rx[j].get(i) * rx[j].get(i);
          s[1] += rh[j].get(i) * wq[j].get(i) * rx[j].get(i);
        }
      }
      if constexpr (MANY) rg[j] = cur.g[j].value(col(j), a.d, in);
      if constexpr (POST) {
        const Raw8<T> ry = cur.y[j].value(col(j), a.d, in);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[j][i] = ry.get(i);
        keep[j] = 0xffu;
        if (a.dr.t) {
          keep[j] = keep8(a.dr, static_cast<uint32_t>(j * TPR + l), static_cast<uint64_t>(n));
#pragma unroll
          for (int i = 0; i < 8; ++i) u[j][i] = (keep[j] >> i) & 1 ? u[j][i] * a.dr.scale : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s[2] += u[j][i] * u[j][i];
      }
    }
    slot_sums<TPR>(s, lds, turn);
    const float r = inv_sqrt(s[0] * a.inv_d + a.eps), m = s[1] * a.inv_d * r * r;
    const float q = norm ? inv_sqrt(s[2] * a.inv_d + a.eps) : 1.f;
    float sb[1] = {0.f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t[j][i] = has_t ? rt[j].get(i) : 0.f;
        if constexpr (PRE) {
          t[j][i] += r * (rh[j].get(i) * wq[j].get(i) - rx[j].get(i) * m);
          Hp[j][i] += rh[j].get(i) * (r * rx[j].get(i));
        }
        v[i] = a.res_scale * t[j][i];
        if constexpr (POST) {
          u[j][i] *= q;
          Q[j][i] += t[j][i] * u[j][i];
          t[j][i] *= (MANY ? rg[j] : wg[j]).get(i) * wp[j].get(i);
          sb[0] += t[j][i] * u[j][i];
        }
      }
      put_row<MODE>(a.gX + n * a.d, col(j), a.d, in, v);
    }
    if constexpr (POST) {
      slot_sums<TPR>(sb, lds, turn);
      const float mb = norm ? sb[0] * a.inv_d : 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = q * (t[j][i] - u[j][i] * mb);
          if (a.dr.t) v[i] = (keep[j] >> i) & 1 ? v[i] * a.dr.scale : 0.f;
        }
        put_row<MODE>(a.gY + n * a.d, col(j), a.d, in, v);
      }
      // the last row of a gate row: its gradient is whole, and its part of w_post's
      if constexpr (MANY) {
        if (in && (n + 1) % a.rows_per_gate == 0) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const int c = 8 * (j * TPR + l), left = a.d - c;
            float* g = a.g_gate + n / a.rows_per_gate * a.d + c;
            float v[8];
            Raw8<float> old;
            if (a.accumulate) load8(old, g, left);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
#pragma clang fp contract(off)  // accumulating adds the gradient that is written otherwise
              Wp[j][i] += rg[j].get(i) * Q[j][i];
              v[i] = wp[j].get(i) * Q[j][i];
              if (a.accumulate) v[i] += old.get(i);
              Q[j][i] = 0.f;
            }
            store8(g, v, left);
          }
        }
      }
    }
    cur = nxt;
  }
  // the block's partial rows: its slots' sums in slot order
#pragma unroll
  for (int which = 0; which < 3; ++which) {
    if (which == 0 ? !POST || !norm : which == 1 ? !POST || MANY || !a.gate : !PRE) continue;
    float* out = a.part + (which * a.sp.blocks + blockIdx.x) * a.d;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = 8 * (j * TPR + l);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = which == 2 ? Hp[j][i] : MANY ? Wp[j][i] : Q[j][i] * (which == 0 ? wg[j] : wp[j]).get(i);
      if constexpr (S == 1) {
        store8(out + c, v, a.d - c);
      } else {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) acc_lds[slot * (TPR * 8) + l * 8 + i] = v[i];
        __syncthreads();
        for (int e = threadIdx.x; e < TPR * 8; e += 256) {
          float s = 0.f;
          for (int k = 0; k < S; ++k) s += acc_lds[k * (TPR * 8) + e];
          if (j * TPR * 8 + e < a.d) out[j * TPR * 8 + e] = s;
        }
      }
    }
  }
}

// Joins the partial rows: block (x, y) sums 32 columns of one output row, 4
// columns by 32 runs of rows a thread, in a fixed order, in fp64: it costs nothing
// here.  y = 0: w_post; 1: w_pre; 2 + g: gate row g, counted on over the grid's z.
// (A loop over y in place of z takes 4 us more.)
__global__ __launch_bounds__(256) void k_stage_norm_grads(const float* part, float* g_w_post, float* g_w_pre,
                                                          float* g_gate, int64_t blocks, int64_t bpg, int64_t gates,
                                                          int d, int accumulate) {
  __shared__ double lds[32][33];
  const int64_t y = int64_t(blockIdx.z) * gridDim.y + blockIdx.y;
  if (y >= 2 + gates) return;
  float* out = y == 0 ? g_w_post : y == 1 ? g_w_pre : g_gate + (y - 2) * d;
  if (out == nullptr) return;
  const float* src = part + (y == 0 ? 0 : y == 1 ? 2 * blocks : blocks + (y - 2) * bpg) * d;
  const int64_t rows = y < 2 ? blocks : bpg;
  const int cx = (threadIdx.x & 7) * 4, ry = threadIdx.x >> 3, c = blockIdx.x * 32 + cx;
  double s[4] = {0., 0., 0., 0.};
  if (c + 4 <= d) {
#pragma unroll 8
    for (int64_t r = ry; r < rows; r += 32) {
      const u32x4 v = ld16B(src + r * d + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += __uint_as_float(v[i]);
    }
  } else {
    for (int64_t r = ry; r < rows; r += 32)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < d) s[i] += src[r * d + c + i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) lds[ry][cx + i] = s[i];
  __syncthreads();
  const int e = threadIdx.x;
  if (e < 32 && blockIdx.x * 32 + e < static_cast<uint32_t>(d)) {
    double v = 0.;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += lds[k][e];
    out += blockIdx.x * 32 + e;
    *out = accumulate ? *out + static_cast<float>(v) : static_cast<float>(v);
  }
}

constexpr int64_t kBwdBlocks = 512;
// Rows that a slot adds up in fp32 before the sum is joined with others in fp64: the
// error of a weight gradient is bounded by them, not by the number of rows.  More
// rows than kBwdBlocks blocks hold that way take a multiple of the blocks.
constexpr int64_t kBwdRun = 512;

// slot shape of a width: TPR threads, V vectors of 8 columns each
struct SlotShape {
  int tpr, v;
};
int slots_per_block(SlotShape s) { return s.tpr > 256 ? 1 : 256 / s.tpr; }
SlotShape slot_shape(int64_t d, bool bwd) {
  if (d <= 128) return {16, 1};
  if (d <= 256) return {32, 1};
  if (d <= 512) return {64, 1};
  // two vectors a thread and no barriers, but half the waves: better forward (16384 x 1024 bf16: 27.6 against
  // 33.2 us), worse backward (46.0 against 43.1 us), where a row takes 240 registers that way
  if (d <= 1024) return bwd ? SlotShape{128, 1} : SlotShape{64, 2};
  // three waves rather than four with a quarter idle (16384 x 1536 bf16: forward 40 against 46 us, backward 71, 76)
  if (d <= 1536) return {192, 1};
  if (d <= 2048) return {256, 1};
  if (d <= 4096) return {512, 1};
  // a backward row does not fit the 128 registers that 1024 threads have each (4096 x 8192: bf16 192 against 93 us, fp32
  // 348 against 211; 4096 x 8191 bf16: 300 against 142).  With two vectors a thread fp32, odd rows and a gate per token
  // still spill, up to 344 bytes a thread.
  return bwd ? SlotShape{512, 2} : SlotShape{1024, 1};
}

BwdSplit bwd_split(int64_t N, int64_t d, int64_t gate_rows) {
  BwdSplit s{};
  const int64_t S = slots_per_block(slot_shape(d, true)), G = gate_rows > 0 ? gate_rows : 1, rpg = N / G;
  const auto parts = [](int64_t n, int64_t of) { return (n + of - 1) / of; };
  s.many = G > kBwdBlocks && rpg <= kBwdRun;
  if (s.many) {
    const int64_t turns = parts(parts(G, kBwdBlocks * S) * rpg, kBwdRun);
    s.gps = std::min(parts(G, kBwdBlocks * S * turns), kBwdRun / rpg);
    s.blocks = parts(G, s.gps * S);
    return s;
  }
  s.bpg = std::max<int64_t>(1, std::min(kBwdBlocks / G, parts(rpg, S)));
  s.bpg *= parts(parts(rpg, s.bpg * S), kBwdRun);
  s.rows_per_block = parts(rpg, s.bpg);
  s.blocks = G * s.bpg;
  return s;
}

template <typename T, template <typename, int, int> class L, bool BWD, typename A>
void by_shape(SlotShape sh, const A& args, dim3 grid, hipStream_t s) {
  if (sh.tpr == 16) return L<T, 16, 1>::go(args, grid, s);
  if (sh.tpr == 32) return L<T, 32, 1>::go(args, grid, s);
  if constexpr (BWD) {
    if (sh.tpr == 128) return L<T, 128, 1>::go(args, grid, s);
    if (sh.tpr == 512 && sh.v == 2) return L<T, 512, 2>::go(args, grid, s);
  } else {
    if (sh.tpr == 64 && sh.v == 2) return L<T, 64, 2>::go(args, grid, s);
  }
  if (sh.tpr == 64) return L<T, 64, 1>::go(args, grid, s);
  if (sh.tpr == 192) return L<T, 192, 1>::go(args, grid, s);
  if (sh.tpr == 256) return L<T, 256, 1>::go(args, grid, s);
  if constexpr (!BWD) {
    if (sh.tpr == 1024) return L<T, 1024, 1>::go(args, grid, s);
  }
  return L<T, 512, 1>::go(args, grid, s);
}
template <typename T, int TPR, int V>
struct FwdLaunch {
  static void go(const NormArgs<T>& a, dim3 grid, hipStream_t s) {
    by_row_mode<T, TPR == 16>(a.d, {a.X, a.Y, a.w_post, a.gate, a.w_pre, a.X_out, a.H}, [&](auto m) {
      hipLaunchKernelGGL((k_stage_norm<T, TPR, V, decltype(m)::value>), grid, dim3(kBlock<TPR>), 0, s, a);
    });
  }
};
template <typename T, int TPR, int V>
struct BwdLaunch {
  template <bool PRE, bool POST, bool MANY>
  static void k(const NormBwdArgs<T>& a, dim3 grid, hipStream_t s) {
    by_row_mode<T, TPR == 16>(a.d, {a.gX_out, a.gH, a.X_out, a.Y, a.w_post, a.gate, a.w_pre, a.gX, a.gY}, [&](auto m) {
      hipLaunchKernelGGL((k_stage_norm_bwd<T, TPR, V, PRE, POST, MANY, decltype(m)::value>), grid, dim3(kBlock<TPR>), 0,
                         s, a);
    });
  }
  static void go(const NormBwdArgs<T>& a, dim3 grid, hipStream_t s) {
    if (!a.Y) return k<true, false, false>(a, grid, s);  // with gH (launch_stage_norm_bwd)
    if (a.sp.many) return a.gH ? k<true, true, true>(a, grid, s) : k<false, true, true>(a, grid, s);
    return a.gH ? k<true, true, false>(a, grid, s) : k<false, true, false>(a, grid, s);
  }
};

}  // namespace

template <typename T>
static void dropout_t(const void* X, void* Y, double p, uint64_t seed, uint64_t offset, int64_t N, int64_t d,
                      hipStream_t s) {
  const int64_t nb = (d + 7) / 8, units = N * nb, per = 256 * kDropUnits;
  by_row_mode<T, true>(d, {X, Y}, [&](auto m) {
    hipLaunchKernelGGL((k_dropout<T, decltype(m)::value>), dim3(uint32_t((units + per - 1) / per)), dim3(256), 0, s,
                       static_cast<const T*>(X), static_cast<T*>(Y), make_drop(p, seed, offset), units, uint32_t(nb), d);
  });
}

void launch_dropout(const void* X, void* Y, double p, uint64_t seed, uint64_t offset, int64_t N, int64_t d, int bf16,
                    hipStream_t s) {
  (bf16 ? dropout_t<bf16_t> : dropout_t<float>)(X, Y, p, seed, offset, N, d, s);
}

template <typename T>
static void norm_t(const StageNorm& c, hipStream_t s) {
  NormArgs<T> a;
  a.X = static_cast<const T*>(c.X);
  a.Y = static_cast<const T*>(c.Y);
  a.w_post = static_cast<const T*>(c.w_post);
  a.gate = static_cast<const T*>(c.gate);
  a.w_pre = static_cast<const T*>(c.w_pre);
  a.X_out = static_cast<T*>(c.X_out);
  a.H = static_cast<T*>(c.H);
  a.res_scale = c.res_scale;
  a.eps = c.eps;
  a.inv_d = 1.f / float(c.d);
  a.dr = make_drop(c.p, c.seed, c.offset);
  a.N = c.N;
  a.rows_per_gate = c.gate_rows > 0 ? c.N / c.gate_rows : c.N;
  a.d = int(c.d);
  const SlotShape sh = slot_shape(c.d, false);
  const int64_t S = slots_per_block(sh);
  const uint32_t grid = uint32_t(std::min<int64_t>((c.N + S - 1) / S, 256 * 8));
  by_shape<T, FwdLaunch, false>(sh, a, dim3(grid), s);
}

void launch_stage_norm(const StageNorm& c, int bf16, hipStream_t s) { (bf16 ? norm_t<bf16_t> : norm_t<float>)(c, s); }

size_t stage_norm_bwd_ws_bytes(int64_t N, int64_t d, int64_t gate_rows) {
  return size_t(3) * bwd_split(N, d, gate_rows).blocks * d * sizeof(float);
}

template <typename T>
static void norm_bwd_t(const StageNorm& c, const StageNormGrads& g, hipStream_t s) {
  NormBwdArgs<T> a;
  a.gX_out = static_cast<const T*>(g.gX_out);
  a.gH = static_cast<const T*>(g.gH);
  a.X_out = static_cast<const T*>(c.X_out);
  a.Y = static_cast<const T*>(c.Y);
  a.w_post = static_cast<const T*>(c.w_post);
  a.gate = static_cast<const T*>(c.gate);
  a.w_pre = static_cast<const T*>(c.w_pre);
  a.gX = static_cast<T*>(g.gX);
  a.gY = static_cast<T*>(g.gY);
  a.g_gate = g.g_gate;
  a.part = g.ws;
  a.res_scale = c.res_scale;
  a.eps = c.eps;
  a.inv_d = 1.f / float(c.d);
  a.dr = make_drop(c.p, c.seed, c.offset);
  a.sp = bwd_split(c.N, c.d, c.gate_rows);
  a.N = c.N;
  a.rows_per_gate = c.gate_rows > 0 ? c.N / c.gate_rows : c.N;
  a.d = int(c.d);
  a.accumulate = g.accumulate;
  by_shape<T, BwdLaunch, true>(slot_shape(c.d, true), a, dim3(uint32_t(a.sp.blocks)), s);
  if (c.w_post || c.gate || g.gH) {
    const int64_t gates = c.gate && !a.sp.many ? c.gate_rows : 0;
    const uint32_t ny = uint32_t(std::min<int64_t>(2 + gates, 32768)), nz = uint32_t((2 + gates + ny - 1) / ny);
    hipLaunchKernelGGL(k_stage_norm_grads, dim3(uint32_t((c.d + 31) / 32), ny, nz), dim3(256), 0, s, g.ws,
                       c.w_post ? g.g_w_post : nullptr, g.gH ? g.g_w_pre : nullptr, gates ? g.g_gate : nullptr,
                       a.sp.blocks, a.sp.bpg, gates, a.d, g.accumulate);
  }
}

void launch_stage_norm_bwd(const StageNorm& c, const StageNormGrads& g, int bf16, hipStream_t s) {
  // neither norm nor block: X_out was res_scale X, and gX is res_scale gX_out, the same pass
  if (!c.Y && !g.gH)
    return launch_stage_norm({g.gX_out, nullptr, nullptr, nullptr, nullptr, g.gX, nullptr, c.res_scale, c.eps, 0.0, 0, 0,
                              c.N, c.d, 0}, bf16, s);
  (bf16 ? norm_bwd_t<bf16_t> : norm_bwd_t<float>)(c, g, s);
}

}  // namespace mapl
