// The edge of a transformer block at a pipeline stage: dropout from a
// counter-based generator, and the fused norm - gate - residual - norm with its
// backward pass.  Formulas: include/mapl_stage.h.  All of it is bound by memory
// traffic: every tensor is read or written once, rows stay in registers between
// their sums and their use.
#include "internal.h"

namespace mapl {
namespace {

// ------------------------------------------------------ 8 elements of a row --
// A thread moves 8 consecutive elements.  The vector types ask only for the
// alignment of an element, so rows of any width and tensors of any offset take
// the same 16-byte accesses; only a row's last elements go one by one.
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

template <typename T>
struct Raw8;  // 8 elements as loaded
template <>
struct Raw8<bf16_t> {
  u32x4 a;
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = a[i >> 1];
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  __device__ __forceinline__ void load(const bf16_t* p, int left) {
    if (left >= 8) {
      a = *reinterpret_cast<const u32x4_a2*>(p);
    } else {
      a = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) a[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
    }
  }
};
template <>
struct Raw8<float> {
  u32x4 a, b;
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(i < 4 ? a[i & 3] : b[i & 3]); }
  __device__ __forceinline__ void load(const float* p, int left) {
    if (left >= 8) {
      a = *reinterpret_cast<const u32x4_a4*>(p);
      b = *reinterpret_cast<const u32x4_a4*>(p + 4);
    } else {
      a = b = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) (i < 4 ? a : b)[i & 3] = __float_as_uint(p[i]);
    }
  }
};

__device__ __forceinline__ void store8(bf16_t* p, const float* v, int left) {
  if (left >= 8) {
    *reinterpret_cast<u32x4_a2*>(p) =
        u32x4{pack2bf(v[0], v[1]), pack2bf(v[2], v[3]), pack2bf(v[4], v[5]), pack2bf(v[6], v[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = f2bf(v[i]);
  }
}
__device__ __forceinline__ void store8(float* p, const float* v, int left) {
  if (left >= 8) {
    *reinterpret_cast<u32x4_a4*>(p) = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                            __float_as_uint(v[3])};
    *reinterpret_cast<u32x4_a4*>(p + 4) = u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                                                __float_as_uint(v[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = v[i];
  }
}

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
// Units of 8 columns, unit u = row * nb + column / 8.
constexpr int kDropUnits = 4;  // units in flight per thread

template <typename T>
__global__ __launch_bounds__(256) void k_dropout(const T* X, T* Y, Drop dr, int64_t units, uint32_t nb, int64_t d) {
  const int64_t u0 = int64_t(blockIdx.x) * (256 * kDropUnits) + threadIdx.x;
  int64_t row = u0 / nb;
  uint32_t b = static_cast<uint32_t>(u0 - row * nb);
  const uint32_t step_row = 256 / nb, step_b = 256 % nb;
  Raw8<T> x[kDropUnits];
  int64_t at[kDropUnits];
  uint32_t keep[kDropUnits];
  int left[kDropUnits];
#pragma unroll
  for (int k = 0; k < kDropUnits; ++k) {
    const bool in = u0 + k * 256 < units;
    at[k] = row * d + int64_t(b) * 8;
    left[k] = in ? static_cast<int>(min(d - int64_t(b) * 8, int64_t(8))) : 0;
    if (in) x[k].load(X + at[k], left[k]);
    keep[k] = keep8(dr, b, static_cast<uint64_t>(row));
    b += step_b;
    row += step_row;
    if (b >= nb) {
      b -= nb;
      ++row;
    }
  }
#pragma unroll
  for (int k = 0; k < kDropUnits; ++k) {
    if (left[k] > 0) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (keep[k] >> i) & 1 ? x[k].get(i) * dr.scale : 0.f;
      store8(Y + at[k], v, left[k]);
    }
  }
}

// ------------------------------------------------------------------ norm edge --
// A slot of TPR threads holds a row, V vectors of 8 columns per thread (vector
// j of thread l starts at column 8 * (j * TPR + l)); a block has 256 threads, or
// one slot's if that is more.
template <int TPR>
constexpr int kBlock = TPR > 256 ? TPR : 256;

template <int TPR>
__device__ __forceinline__ float slot_sum(float v, float* lds) {
#pragma unroll
  for (int m = 1; m < (TPR < 64 ? TPR : 64); m <<= 1) v += __shfl_xor(v, m);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += lds[w];
  }
  return v;
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

template <typename T, int TPR, int V>
__global__ __launch_bounds__(kBlock<TPR>) void k_stage_norm(NormArgs<T> a) {
  constexpr int S = kBlock<TPR> / TPR;
  __shared__ float lds[16];
  const int l = threadIdx.x % TPR;
  // every thread of a block takes the same number of turns (slot_sum has barriers)
  for (int64_t n0 = int64_t(blockIdx.x) * S; n0 < a.N; n0 += int64_t(gridDim.x) * S) {
    const int64_t n = n0 + threadIdx.x / TPR;
    const bool in = n < a.N;
    Raw8<T> rx[V], ry[V];
    int left[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = 8 * (j * TPR + l);
      left[j] = in ? a.d - c : 0;
      rx[j].load(a.X + n * a.d + c, left[j]);
      if (a.Y) ry[j].load(a.Y + n * a.d + c, left[j]);
    }
    float x[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = a.res_scale * rx[j].get(i);
    if (a.Y) {
      float u[V][8], s = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[j][i] = ry[j].get(i);
        if (a.dr.t) {
          const uint32_t keep = keep8(a.dr, static_cast<uint32_t>(j * TPR + l), static_cast<uint64_t>(n));
#pragma unroll
          for (int i = 0; i < 8; ++i) u[j][i] = (keep >> i) & 1 ? u[j][i] * a.dr.scale : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s += u[j][i] * u[j][i];
      }
      if (a.w_post) {
        s = slot_sum<TPR>(s, lds);
        const float q = rsqrtf(s * a.inv_d + a.eps);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          Raw8<T> w;
          w.load(a.w_post + 8 * (j * TPR + l), left[j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) u[j][i] *= q * w.get(i);
        }
      }
      if (a.gate) {
        const T* g = a.gate + (in ? n / a.rows_per_gate : 0) * a.d;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          Raw8<T> w;
          w.load(g + 8 * (j * TPR + l), left[j]);
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
      for (int j = 0; j < V; ++j) store8(a.X_out + n * a.d + 8 * (j * TPR + l), x[j], left[j]);
    }
    if (a.H) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += i < left[j] ? x[j][i] * x[j][i] : 0.f;
      s = slot_sum<TPR>(s, lds);
      const float r = rsqrtf(s * a.inv_d + a.eps);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        Raw8<T> w;
        w.load(a.w_pre + 8 * (j * TPR + l), left[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] *= r * w.get(i);
        store8(a.H + n * a.d + 8 * (j * TPR + l), x[j], left[j]);
      }
    }
  }
}

// ------------------------------------------------------------------- backward --
// The rows are split over blocks, and a block's rows over its slots, both into
// contiguous runs, so that the sums over rows have a fixed order.
//  - few gate rows (or no gate): a block's rows lie in one gate row; `bpg`
//    blocks share a gate row.  Each block leaves one partial row of every
//    weight gradient, and k_stage_norm_grads joins them.
//  - many gate rows (a gate per token): a slot takes `gps` whole gate rows and
//    writes their gradients itself.
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

template <typename T, int TPR, int V>
__global__ __launch_bounds__(kBlock<TPR>) void k_stage_norm_bwd(NormBwdArgs<T> a) {
  constexpr int S = kBlock<TPR> / TPR;
  __shared__ float lds[16];
  __shared__ float acc_lds[S > 1 ? 256 * 8 : 1];
  const int l = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  int64_t r0, r1, turns;  // this slot's rows; the block's turns
  if (a.sp.many) {
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
  float Q[V][8], Wp[V][8], Hp[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) Q[j][i] = Wp[j][i] = Hp[j][i] = 0.f;

  for (int64_t k = 0; k < turns; ++k) {
    const int64_t n = r0 + k;
    const bool in = n < r1;
    const int64_t gate_row = a.gate && in ? n / a.rows_per_gate : 0;
    float t[V][8], u[V][8];
    Raw8<T> rx[V], rh[V];
    uint32_t keep[V];
    int left[V];
    float sx = 0.f, sax = 0.f, su = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = 8 * (j * TPR + l);
      left[j] = in ? a.d - c : 0;
      Raw8<T> v;
      if (a.gX_out) {
        v.load(a.gX_out + n * a.d + c, left[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[j][i] = v.get(i);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[j][i] = 0.f;
      }
      if (a.gH) {
        rx[j].load(a.X_out + n * a.d + c, left[j]);
        rh[j].load(a.gH + n * a.d + c, left[j]);
        v.load(a.w_pre + c, left[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sx += rx[j].get(i) * rx[j].get(i);
          sax += rh[j].get(i) * v.get(i) * rx[j].get(i);
        }
      }
      keep[j] = 0xffu;
      if (a.Y) {
        v.load(a.Y + n * a.d + c, left[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[j][i] = v.get(i);
        if (a.dr.t) {
          keep[j] = keep8(a.dr, static_cast<uint32_t>(j * TPR + l), static_cast<uint64_t>(n));
#pragma unroll
          for (int i = 0; i < 8; ++i) u[j][i] = (keep[j] >> i) & 1 ? u[j][i] * a.dr.scale : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) su += u[j][i] * u[j][i];
      }
    }
    if (a.gH) {
      sx = slot_sum<TPR>(sx, lds);
      sax = slot_sum<TPR>(sax, lds);
      const float r = rsqrtf(sx * a.inv_d + a.eps), m = sax * a.inv_d * r * r;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        Raw8<T> w;
        w.load(a.w_pre + 8 * (j * TPR + l), left[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          t[j][i] += r * (rh[j].get(i) * w.get(i) - rx[j].get(i) * m);
          Hp[j][i] += rh[j].get(i) * (r * rx[j].get(i));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = a.res_scale * t[j][i];
      store8(a.gX + n * a.d + 8 * (j * TPR + l), v, left[j]);
    }
    if (a.Y) {
      float q = 1.f, sb = 0.f;
      if (a.w_post) q = rsqrtf(slot_sum<TPR>(su, lds) * a.inv_d + a.eps);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = 8 * (j * TPR + l);
        Raw8<T> w;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          u[j][i] *= q;
          Q[j][i] += t[j][i] * u[j][i];
        }
        if (a.gate) {
          w.load(a.gate + gate_row * a.d + c, left[j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) t[j][i] *= w.get(i);
        }
        if (a.w_post) {
          w.load(a.w_post + c, left[j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            t[j][i] *= w.get(i);
            sb += t[j][i] * u[j][i];
          }
        }
      }
      const float m = a.w_post ? slot_sum<TPR>(sb, lds) * a.inv_d : 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = q * (t[j][i] - u[j][i] * m);
          if (a.dr.t) v[i] = (keep[j] >> i) & 1 ? v[i] * a.dr.scale : 0.f;
        }
        store8(a.gY + n * a.d + 8 * (j * TPR + l), v, left[j]);
      }
    }
    // the last row of a gate row (or of this slot): its sum goes to the weights
    if (in && (n + 1 == r1 || (a.sp.many && (n + 1) % a.rows_per_gate == 0))) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = 8 * (j * TPR + l);
        Raw8<T> wg, wp;
        if (a.gate) wg.load(a.gate + gate_row * a.d + c, left[j]);
        if (a.w_post) wp.load(a.w_post + c, left[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          Wp[j][i] += a.gate ? wg.get(i) * Q[j][i] : Q[j][i];
          if (a.w_post) Q[j][i] *= wp.get(i);
        }
        if (a.sp.many) {
          float* g = a.g_gate + gate_row * a.d + c;
          float v[8];
          Raw8<float> old;
          if (a.accumulate) old.load(g, left[j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[i] = a.accumulate ? old.get(i) + Q[j][i] : Q[j][i];
            Q[j][i] = 0.f;
          }
          store8(g, v, left[j]);
        }
      }
    }
  }
  // the block's partial rows: its slots' sums in slot order
#pragma unroll
  for (int which = 0; which < 3; ++which) {
    if (which == 0 ? a.w_post == nullptr : which == 1 ? (a.gate == nullptr || a.sp.many) : a.gH == nullptr) continue;
    float* out = a.part + (which * a.sp.blocks + blockIdx.x) * a.d;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float* v = which == 0 ? Wp[j] : which == 1 ? Q[j] : Hp[j];
      const int c = 8 * (j * TPR + l);
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

// Joins the partial rows: block (x, y) sums 16 columns of one output row, 16
// threads a column, in a fixed order.  y = 0: w_post; 1: w_pre; 2 + g: gate row g.
__global__ __launch_bounds__(256) void k_stage_norm_grads(const float* part, float* g_w_post, float* g_w_pre,
                                                          float* g_gate, int64_t blocks, int64_t bpg, int d,
                                                          int accumulate) {
  __shared__ float lds[16][17];
  const int64_t y = int64_t(blockIdx.y);
  float* out = y == 0 ? g_w_post : y == 1 ? g_w_pre : g_gate ? g_gate + (y - 2) * d : nullptr;
  if (out == nullptr) return;
  const float* src = part + (y == 0 ? 0 : y == 1 ? 2 * blocks : blocks + (y - 2) * bpg) * d;
  const int64_t rows = y < 2 ? blocks : bpg;
  const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4, c = blockIdx.x * 16 + cx;
  float s = 0.f;
  if (c < d)
    for (int64_t r = ry; r < rows; r += 16) s += src[r * d + c];
  lds[ry][cx] = s;
  __syncthreads();
  if (ry == 0 && c < d) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += lds[k][cx];
    out[c] = accumulate ? out[c] + s : s;
  }
}

constexpr int64_t kBwdBlocks = 512;

// slot shape of a width: TPR threads, V vectors of 8 columns each
struct SlotShape {
  int tpr, v;
};
int slots_per_block(SlotShape s) { return s.tpr > 256 ? 1 : 256 / s.tpr; }
SlotShape slot_shape(int64_t d) {
  if (d <= 64) return {8, 1};
  if (d <= 128) return {16, 1};
  if (d <= 256) return {32, 1};
  if (d <= 512) return {64, 1};
  if (d <= 1024) return {64, 2};
  if (d <= 2048) return {256, 1};
  if (d <= 4096) return {512, 1};
  return {1024, 1};
}

BwdSplit bwd_split(int64_t N, int64_t d, int64_t gate_rows) {
  BwdSplit s{};
  const int64_t S = slots_per_block(slot_shape(d)), G = gate_rows > 0 ? gate_rows : 1, rpg = N / G;
  s.many = G > kBwdBlocks;
  if (s.many) {
    s.gps = (G + kBwdBlocks * S - 1) / (kBwdBlocks * S);
    s.blocks = (G + s.gps * S - 1) / (s.gps * S);
    return s;
  }
  s.bpg = std::max<int64_t>(1, std::min(kBwdBlocks / G, (rpg + S - 1) / S));
  s.rows_per_block = (rpg + s.bpg - 1) / s.bpg;
  s.blocks = G * s.bpg;
  return s;
}

template <typename T, template <typename, int, int> class L, typename A>
void by_shape(SlotShape sh, const A& args, dim3 grid, hipStream_t s) {
  switch (sh.tpr * 16 + sh.v) {
    case 8 * 16 + 1: return L<T, 8, 1>::go(args, grid, s);
    case 16 * 16 + 1: return L<T, 16, 1>::go(args, grid, s);
    case 32 * 16 + 1: return L<T, 32, 1>::go(args, grid, s);
    case 64 * 16 + 1: return L<T, 64, 1>::go(args, grid, s);
    case 64 * 16 + 2: return L<T, 64, 2>::go(args, grid, s);
    case 256 * 16 + 1: return L<T, 256, 1>::go(args, grid, s);
    case 512 * 16 + 1: return L<T, 512, 1>::go(args, grid, s);
    default: return L<T, 1024, 1>::go(args, grid, s);
  }
}
template <typename T, int TPR, int V>
struct FwdLaunch {
  static void go(const NormArgs<T>& a, dim3 grid, hipStream_t s) {
    hipLaunchKernelGGL((k_stage_norm<T, TPR, V>), grid, dim3(kBlock<TPR>), 0, s, a);
  }
};
template <typename T, int TPR, int V>
struct BwdLaunch {
  static void go(const NormBwdArgs<T>& a, dim3 grid, hipStream_t s) {
    hipLaunchKernelGGL((k_stage_norm_bwd<T, TPR, V>), grid, dim3(kBlock<TPR>), 0, s, a);
  }
};

}  // namespace

template <typename T>
static void dropout_t(const void* X, void* Y, double p, uint64_t seed, uint64_t offset, int64_t N, int64_t d,
                      hipStream_t s) {
  const int64_t nb = (d + 7) / 8, units = N * nb, per = 256 * kDropUnits;
  hipLaunchKernelGGL(k_dropout<T>, dim3(uint32_t((units + per - 1) / per)), dim3(256), 0, s,
                     static_cast<const T*>(X), static_cast<T*>(Y), make_drop(p, seed, offset), units, uint32_t(nb), d);
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
  const SlotShape sh = slot_shape(c.d);
  const int64_t S = slots_per_block(sh);
  const uint32_t grid = uint32_t(std::min<int64_t>((c.N + S - 1) / S, 256 * 8));
  by_shape<T, FwdLaunch>(sh, a, dim3(grid), s);
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
  by_shape<T, BwdLaunch>(slot_shape(c.d), a, dim3(uint32_t(a.sp.blocks)), s);
  if (c.w_post || c.gate || g.gH) {
    const uint32_t gates = c.gate && !a.sp.many ? uint32_t(c.gate_rows) : 0;
    hipLaunchKernelGGL(k_stage_norm_grads, dim3(uint32_t((c.d + 15) / 16), 2 + gates), dim3(256), 0, s, g.ws,
                       c.w_post ? g.g_w_post : nullptr, g.gH ? g.g_w_pre : nullptr, gates ? g.g_gate : nullptr,
                       a.sp.blocks, a.sp.bpg, a.d, g.accumulate);
  }
}

void launch_stage_norm_bwd(const StageNorm& c, const StageNormGrads& g, int bf16, hipStream_t s) {
  (bf16 ? norm_bwd_t<bf16_t> : norm_bwd_t<float>)(c, g, s);
}

}  // namespace mapl
