// Causal attention over packed sequences with grouped heads, and its backward
// pass.  Formulas: include/mapl_block.h.
//
// The three kernels are alike.  A wave owns the rows of 32-row blocks (query rows
// in the forward pass and for gQ, key rows for gK and gV) as matrix operands in
// registers and walks over the rows of the other side in tiles that the block
// stages in LDS.  Every product has the owned rows as its columns (lane l holds
// column l & 31), so that
//   - a row's statistics live in its lane: the softmax's maximum and sum are taken
//     over registers and one swap of half-waves;
//   - the scores' registers are the operand of the next product as they stand: the
//     16 values of a half-wave at rows 8 (v >> 2) + 4 h + (v & 3) serve as
//     contraction slots, and the other operand is read in the same order, its 4
//     consecutive rows by LDS reads that transpose (bf16) or one by one (fp32).
// fp32 operands go through the fp32 matrix instruction, in the same slots.
//
// Packed rows are tiled as they lie in memory, whatever the sequences' edges: row i
// sees the rows [start(i), i], and a tile's range begins at its first row's start.
// Short sequences share tiles, and no list of tiles is needed.
//
// A row outside the sequences, or beyond N, is read at a row that exists; its
// products are masked or not stored.  A masked product is replaced before the
// softmax, but a zero weight times an infinity or NaN in a masked place would still
// spoil a sum of products: rows of an output block that holds a NaN are computed again, one
// by one over their visible rows alone (in the forward pass those whose NaN no value that
// they see explains).  So are rows with an infinity in a product's padding:
// behind its D columns an aligned tile repeats a row's first ones, which meet zeros of the
// other side.  That makes a NaN of a score, and of everything that it enters, so a
// log-sum that is NaN is formed again as well.  And so are rows of very large scores (far)
// and those whose sum of weighted values, up to 2^8 times their number of keys as large as
// its mean, is infinite: by means of the keys so far, which are no larger than the values.
#pragma once

#include <type_traits>

#include "internal.h"
#include "vec8.h"

namespace mapl {
namespace {

typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kCuLds = 1024;  // sequence edges kept in LDS

// ------------------------------------------------------------------ operands --
// 16 contraction indices of 32 rows or columns: lane l holds row l & 31 and 8 of
// the indices, which ones is the same for both operands of a product.
template <typename T>
struct Operand;
template <>
struct Operand<bf16_t> {
  bf16x8 v;
};
template <>
struct Operand<float> {
  f32x8 v;
};

__device__ __forceinline__ f32x16 mma(Operand<bf16_t> a, Operand<bf16_t> b, f32x16 c) {
  return mfma_bf16_32x32x16(a.v, b.v, c);
}
__device__ __forceinline__ f32x16 mma(Operand<float> a, Operand<float> b, f32x16 c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c = mfma_f32_32x32x2(a.v[i], b.v[i], c);
  return c;
}

// the registers 8 u .. 8 u + 7 of a product as an operand; bf16: rounded to nearest
// even, the same relative error as the output's own rounding
template <typename T>
__device__ __forceinline__ Operand<T> as_operand(const f32x16& x, int u) {
  if constexpr (sizeof(T) == 2) {
    return {__builtin_bit_cast(bf16x8, u32x4{cvt2bf(x[8 * u], x[8 * u + 1]), cvt2bf(x[8 * u + 2], x[8 * u + 3]),
                                             cvt2bf(x[8 * u + 4], x[8 * u + 5]), cvt2bf(x[8 * u + 6], x[8 * u + 7])})};
  } else {
    Operand<float> o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = x[8 * u + i];
    return o;
  }
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// columns 16 t + 8 h .. + 7 of a row in memory, zeros from column D on
template <typename T, bool ALIGNED>
__device__ __forceinline__ Operand<T> load_row(const T* row, int c, int D) {
  Raw8<T> r;
  if constexpr (ALIGNED) {  // 16-byte chunks are whole or absent
    constexpr int E = 16 / sizeof(T);
    const u32x4 z = {0u, 0u, 0u, 0u};
    r.a = c < D ? *reinterpret_cast<const u32x4*>(row + c) : z;
    if constexpr (sizeof(T) == 4) r.b = c + E < D ? *reinterpret_cast<const u32x4*>(row + c + E) : z;
  } else {
    load8(r, row + c, max(0, min(8, D - c)));
  }
  Operand<T> o;
  if constexpr (sizeof(T) == 2) {
    o.v = __builtin_bit_cast(bf16x8, r.a);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = r.get(i);
  }
  return o;
}

// --------------------------------------------------------------------- tiles --
// Rows of a tile in LDS: kSlots chunks of 16 bytes, chunk c of row r at slot
// c ^ turn(r).  The copies to LDS are contiguous, so the lanes' global addresses carry
// the permutation.  It keeps apart in the banks
//   - 8 consecutive rows at one column (operands by rows, 16 bytes a lane);
//   - bf16: 4 rows at 16 columns (reads that transpose, 8 bytes a lane);
//   - fp32: rows r and r + 4 at 32 columns (operands by columns);
// measured in a loop of such reads on every SIMD: 4.2 cycles for 16 bytes a lane, 2.6 for
// 8 and for 4, as without any permutation in contiguous reads.
template <typename T, int DP>
struct Tile {
  static constexpr int E = 16 / sizeof(T);                               // elements of a chunk
  static constexpr int kSlots = DP <= 64 ? 64 / E : 128 / E;             // a power of two
  static constexpr int kRowBytes = kSlots * 16;
  static __device__ __forceinline__ int turn(int r) {
    if constexpr (kSlots == 8) return ((r & 2) << 1) | ((r >> 1) & 2) | ((r >> 3) & 1);
    return ((r & 3) << 2) | ((r >> 2) & 3);
  }
  static __device__ __forceinline__ int at(int r, int c) { return r * kRowBytes + ((c ^ turn(r)) << 4); }

  // rows r0 + (l & 31), columns 16 t + 8 h .. + 7
  static __device__ __forceinline__ Operand<T> by_rows(const char* lds, int r0, int t) {
    const int lane = threadIdx.x & 63, r = r0 + (lane & 31), h = lane >> 5;
    if constexpr (sizeof(T) == 2) {
      return {__builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(lds + at(r, 2 * t + h)))};
    } else {
      const f32x4 a = *reinterpret_cast<const f32x4*>(lds + at(r, 4 * t + 2 * h));
      const f32x4 b = *reinterpret_cast<const f32x4*>(lds + at(r, 4 * t + 2 * h + 1));
      return {f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
    }
  }

  // columns 32 db + (l & 31), rows r0 + 4 h .. + 3 and r0 + 8 + 4 h .. + 3 (r0 a multiple of 16)
  static __device__ __forceinline__ Operand<T> by_cols(const char* lds, int r0, int db) {
    const int lane = threadIdx.x & 63, h = lane >> 5;
    if constexpr (sizeof(T) == 2) {
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const int i = lane & 15, r = r0 + 4 * h + (i >> 2);
      const int c = 4 * db + 2 * ((lane >> 4) & 1) + ((i >> 1) & 1), off = 8 * (i & 1);
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + at(r, c) + off));
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + at(r + 8, c) + off));
      const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
      return {__builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]})};
    } else {
      Operand<float> o;
      const int c = 8 * db + ((lane & 31) >> 2), off = 4 * (lane & 3);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o.v[e] = *reinterpret_cast<const float*>(lds + at(r0 + 8 * (e >> 2) + 4 * h + (e & 3), c) + off);
      return o;
    }
  }
};

// The copies of a tile's rows to LDS, a wave's share of them: lane offsets once, the
// tile's place in a uniform base.  Rows behind the last are read at the last.
template <typename T, int DP, int ROWS, int WAVES, bool ALIGNED>
struct Stager {
  using L = Tile<T, DP>;
  static constexpr int PER = ROWS * L::kSlots / 64 / WAVES;
  static_assert(PER > 0 && ROWS * L::kSlots % (64 * WAVES) == 0, "whole copies");
  static_assert(uint64_t(ROWS) * (sizeof(float) << 22) <= 1ull << 31, "a tile's offsets, rows of 2^22 elements, have 32 bits");
  uint32_t ld;  // bytes of a row
  int D;
  uint32_t off[PER];

  static __device__ __forceinline__ int slot(int k) { return (wave_id() + k * WAVES) * 64 + (threadIdx.x & 63); }
  __device__ __forceinline__ uint32_t chunk(int k) const {  // byte offset within a row
    const int c = (slot(k) % L::kSlots) ^ L::turn(slot(k) / L::kSlots);
    return c * L::E < D ? c * 16 : 0;
  }
  __device__ __forceinline__ Stager(int64_t ld_elems, int D_) : ld(uint32_t(ld_elems) * sizeof(T)), D(D_) {
    if constexpr (ALIGNED) {
#pragma unroll
      for (int k = 0; k < PER; ++k) off[k] = uint32_t(slot(k) / L::kSlots) * ld + chunk(k);
    }
  }
  // rows r0 .. of the tensor's rows at `base` to the tile `lds`
  __device__ __forceinline__ void operator()(char* lds, const T* base, int r0, int N) const {
    const char* at = reinterpret_cast<const char*>(base) + int64_t(r0) * ld;
    if constexpr (ALIGNED) {
      const uint32_t to = lds_address(lds) + wave_id() * 1024;
      if (r0 + ROWS <= N) {
#pragma unroll
        for (int k = 0; k < PER; ++k) copy_lane16_to_lds(at, off[k], to + k * WAVES * 1024);
      } else {
#pragma unroll
        for (int k = 0; k < PER; ++k)
          copy_lane16_to_lds(at, uint32_t(min(slot(k) / L::kSlots, N - 1 - r0)) * ld + chunk(k), to + k * WAVES * 1024);
      }
    } else {
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int r = slot(k) / L::kSlots, c = (slot(k) % L::kSlots) ^ L::turn(r);
        const T* row = reinterpret_cast<const T*>(at + int64_t(min(r, N - 1 - r0)) * ld);
        const int left = max(0, D - c * L::E);
        u32x4 v;
        if constexpr (sizeof(T) == 2) {
          Raw8<T> x;
          load8(x, row + (left > 0 ? c * L::E : 0), min(8, left));
          v = x.a;
        } else {
          v = left >= 4 ? ld16B(row + c * L::E) : ld_tail4(row + (left > 0 ? c * L::E : 0), left);
        }
        *reinterpret_cast<u32x4*>(lds + slot(k) * 16) = v;
      }
    }
  }
};

// both half-waves' values of a column joined
template <typename F>
__device__ __forceinline__ float join_halves(float v, F f) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum2(float a, float b) { return a + b; }
__device__ __forceinline__ float max2(float a, float b) { return fmaxf(a, b); }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) v = fmaxf(v, __shfl_xor(v, s));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) v += __shfl_xor(v, s);
  return v;
}

// ----------------------------------------------------------------- sequences --
struct Seq {
  int start, end;  // of the row's sequence, [i, i + 1) for a row of none
  bool inside;
};
// edges in ascending order; any values give a range around i within [0, N)
__device__ __forceinline__ Seq find_seq(const int32_t* cu, int S, int i, int N) {
  int lo = 0, n = S + 1;  // the number of edges <= i
  while (n > 0) {
    const int half = n >> 1;
    if (cu[lo + half] <= i) {
      lo += half + 1;
      n -= half + 1;
    } else {
      n = half;
    }
  }
  Seq s;
  s.inside = lo >= 1 && lo <= S && i < N;
  s.start = s.inside ? min(max(cu[lo - 1], 0), i) : i;
  s.end = s.inside ? min(max(cu[lo], i + 1), N) : i + 1;
  return s;
}
// the edges in LDS where they fit; ends with a barrier
__device__ __forceinline__ const int32_t* edges(const int32_t* cu, int S, int32_t* lds) {
  if (S + 1 > kCuLds) return cu;
  for (int i = threadIdx.x; i <= S; i += blockDim.x) lds[i] = cu[i];
  __syncthreads();
  return lds;
}

// The tile of BM rows at place `rank` in the order of falling work(t), so that the longest
// ranges begin first and the last blocks are short ones; every thread of the block calls it.
// Beyond kRanked tiles there are blocks enough to even out: the tiles from the last.
// 16384 rows in sequences of 1 to 4099, 16 x 64 bf16, against the tiles from the last:
// forward 143 for 162 us, gQ 175 for 198, gK and gV 281 for 360.
constexpr int kRanked = 256;
template <typename F>
__device__ __forceinline__ int ranked_tile(int tiles, int rank, F work) {
  if (tiles > kRanked) return tiles - 1 - rank;
  __shared__ int w[kRanked], at;
  const int t = threadIdx.x;
  int mine = 0;
  if (t < tiles) w[t] = mine = work(t);
  __syncthreads();
  if (t < tiles) {
    int before = 0;
    for (int x = 0; x < tiles; ++x) before += w[x] > mine || (w[x] == mine && x > t) ? 1 : 0;
    if (before == rank) at = t;
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(at);
}

template <typename T>
struct AttnArgs {
  const T *Q, *K, *V, *O, *gO;
  T *out, *gQ, *gK, *gV;
  const int32_t* cu;
  float *lse, *rows;  // lse [Hq][N]; rows [Hq][2][N]: -lse / scale and -delta
  float* part;        // sums of a split: gQ [splits][N][Hq D]; gK, gV [splits][N][2][Hkv D]
  int splits;
  int64_t ldq, ldk, ldv, ldo, ldgo, ldgq, ldgk, ldgv;
  float scale;
  int S, N, Hq, Hkv, D;
};

// 4 consecutive columns from c of a row, as many as there are
template <typename T, bool ALIGNED>
__device__ __forceinline__ void put4(T* row, int c, int D, float a, float b, float x, float y) {
  if (c >= D) return;
  if constexpr (ALIGNED) {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<u32x2*>(row + c) = u32x2{cvt2bf(a, b), cvt2bf(x, y)};
    else
      *reinterpret_cast<f32x4*>(row + c) = f32x4{a, b, x, y};
  } else {
    row[c] = from_f32<T>(a);
    if (c + 1 < D) row[c + 1] = from_f32<T>(b);
    if (c + 2 < D) row[c + 2] = from_f32<T>(x);
    if (c + 3 < D) row[c + 3] = from_f32<T>(y);
  }
}

// a product's columns as rows of memory: column l & 31 in `row`, column block db
template <typename T, bool ALIGNED>
__device__ __forceinline__ void put_block(T* row, int db, int D, const f32x16& x, float f) {
  const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int g = 0; g < 4; ++g)
    put4<T, ALIGNED>(row, 32 * db + 8 * g + 4 * h, D, x[4 * g] * f, x[4 * g + 1] * f, x[4 * g + 2] * f, x[4 * g + 3] * f);
}

template <int NB>
__device__ __forceinline__ bool any_nan(const f32x16 (&x)[NB], bool in) {
  bool bad = false;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int v = 0; v < 16; ++v) bad = bad || x[b][v] != x[b][v];
  return __any(in && bad);
}

// One row at a time, by a wave: 64 rows of the other side in its lanes for their products
// with it, then the columns l and l + 64 of the sum in its lanes.  Some 250 times as slow as
// the matrix products, for the few rows beside a masked NaN or at the ends of fp32; a sum
// that is NaN throughout, as in a step whose gradients are, ends the row at once.
template <typename T>
__device__ __forceinline__ float dot_row(const T* x, const T* y, int D) {
  float s = 0.f;
#pragma unroll 8
  for (int e = 0; e < D; ++e) s = fmaf(to_f32<T>(x[e]), to_f32<T>(y[e]), s);
  return s;
}
struct LaneSum {
  float a = 0.f, b = 0.f;
  // the n rows at x, weighted by w of the lanes 0 .. n - 1
  template <typename T>
  __device__ __forceinline__ void add(const T* x, int64_t ld, int n, float w, int D) {
    const int l = threadIdx.x & 63, la = min(l, D - 1), lb = min(l + 64, D - 1);
#pragma unroll 8
    for (int t = 0; t < n; ++t, x += ld) {
      const float f = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), t));
      a = fmaf(f, to_f32<T>(x[la]), a);
      b = fmaf(f, to_f32<T>(x[lb]), b);
    }
  }
  __device__ __forceinline__ bool lost() const { return __all(a != a && b != b); }
  template <typename T>
  __device__ __forceinline__ void put(T* row, int D, float f) const {
    const int l = threadIdx.x & 63;
    if (l < D) row[l] = from_f32<T>(a * f);
    if (l + 64 < D) row[l + 64] = from_f32<T>(b * f);
  }
};

// Of the columns l and l + 64 of the rows from .. to: the last that holds a NaN, and the last
// that holds an infinity (-1: none).
struct Spoilt {
  int nan[2] = {-1, -1}, inf[2] = {-1, -1};
};
template <typename T>
__device__ __forceinline__ Spoilt last_spoilt(const T* x, int64_t ld, int from, int to, int D) {
  const int l = threadIdx.x & 63, col[2] = {min(l, D - 1), min(l + 64, D - 1)};
  Spoilt s;
  constexpr int AHEAD = 16;
  for (int j = to; j >= from && !__all(s.nan[0] >= 0 && s.nan[1] >= 0); j -= AHEAD) {
    T y[AHEAD][2];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
#pragma unroll
      for (int c = 0; c < 2; ++c) y[u][c] = x[max(j - u, from) * ld + col[c]];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float v = fabsf(to_f32<T>(y[u][c]));
        if (s.nan[c] < 0 && v != v) s.nan[c] = max(j - u, from);
        if (s.inf[c] < 0 && v == INFINITY) s.inf[c] = max(j - u, from);
      }
  }
  return s;
}
// Whether a sum x at column c of a row that begins at `start` comes from what the row does not
// see, or is an infinity that no value is: a NaN (an infinity) among the values it sees
// explains it.  Every lane of the wave calls it, each with a column of its own.
__device__ __forceinline__ bool unexplained(float x, const Spoilt& s, int c, int start) {
  const int n0 = __shfl(s.nan[0], c & 63), n1 = __shfl(s.nan[1], c & 63);
  const int f0 = __shfl(s.inf[0], c & 63), f1 = __shfl(s.inf[1], c & 63);
  if (x != x) return (c < 64 ? n0 : n1) < start;
  return fabsf(x) == INFINITY && (c < 64 ? f0 : f1) < start;
}

// ------------------------------------------------------------------- forward --
// The weights exp2(s c - m c) take m c as rounded: a factor that all of a row's weights share,
// and its sum with them, so that it cancels.  Up to 2^28 it is 2^8 at most, either way;
// later it would end in 0 or infinity, and the row is formed again, by differences, which
// for every score would be one vector operation more of 5.
__device__ __forceinline__ bool far(float m, float c) { return fabsf(m * c) > 0x1p28f && m != -INFINITY; }

// One row of O, and of lse where `sum_lost`.
template <typename T>
__device__ __forceinline__ void fwd_row(const AttnArgs<T>& a, int h, int kv, int i, int start, bool sum_lost) {
  const T* q = a.Q + i * a.ldq + int64_t(h) * a.D;
  const int64_t kd = int64_t(kv) * a.D;
  float m = -INFINITY, l = 0.f;
  LaneSum o;
  for (int j = start; j <= i && (!o.lost() || (sum_lost && l == l)); j += 64) {
    const int n = min(64, i + 1 - j), at = min(int(threadIdx.x & 63), n - 1);
    const float s = a.scale * dot_row(q, a.K + (j + at) * a.ldk + kd, a.D);
    const float mn = fmaxf(m, wave_max(s)), f = m == mn ? 1.f : exp2f((m - mn) * kLog2e);
    const float p = int(threadIdx.x & 63) >= n || s == -INFINITY ? 0.f : exp2f((s - mn) * kLog2e);
    const float before = l * f;
    m = mn;
    l = before + wave_sum(p);
    const float inv = l == 0.f ? 0.f : 1.f / l;  // no weight yet: the sums stay 0
    o.a *= before * inv;
    o.b *= before * inv;
    o.add(a.V + j * a.ldv + kd, a.ldv, n, p * inv, a.D);
  }
  o.put(a.out + i * a.ldo + int64_t(h) * a.D, a.D, l == 0.f ? NAN : 1.f);
  if (sum_lost && (threadIdx.x & 63) == 0) a.lse[int64_t(h) * a.N + i] = fmaf(__builtin_amdgcn_logf(l), kLn2, m);
}

// o = sum exp(s - m) v / l with l = sum exp(s - m), in one pass over the keys: a running
// reference m per row, the sums scaled where it moves.  Two products a pair of rows, 4 D
// operations, and 5 vector operations a score (factor and difference, exp, sum, maximum,
// half a rounding).  32 query rows a wave and two waves a SIMD: one wave's softmax runs
// beside the other's products.  No unit is full: at 64 columns a vector instruction is
// being issued in 60 % of a SIMD's cycles and its matrix unit is busy in 30 % (at 128: 52 and
// 55), while a wave waits for a barrier or for LDS through 33 % (19) of its cycles and, ready,
// for its turn through 29 (35).  64 rows a wave, 8 waves a block, tiles of 128
// keys, and a loop without the turn's overlap were measured and none is faster.
// bf16: 16384 rows of 16 x 64 in sequences of 2048 101 us (681 TFLOP/s of unmasked pairs),
// 16384 rows of 16 x 128 in one sequence 1.03-1.09 ms (1.01-1.07 PFLOP/s; the library's product
// of 16384^3 reaches 1.40).
template <typename T, int DP, int WAVES, int BN, int OCC, bool ALIGNED>
__global__ __launch_bounds__(64 * WAVES, OCC) void k_attn_fwd(AttnArgs<T> a) {
  using L = Tile<T, DP>;
  constexpr int NT = DP / 16, NB = DP / 32, KB = BN / 32, BM = 32 * WAVES;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  __shared__ int32_t cu_lds[kCuLds];
  constexpr int TILE = BN * L::kRowBytes;
  const auto k_tile = [&](int b) { return smem + b * 2 * TILE; };
  const auto v_tile = [&](int b) { return smem + b * 2 * TILE + TILE; };

  const int tiles = (a.N + BM - 1) / BM;
  const int32_t* cu = edges(a.cu, a.S, cu_lds);
  const int t = ranked_tile(tiles, blockIdx.x / a.Hq, [&](int x) { return min((x + 1) * BM, a.N) - find_seq(cu, a.S, x * BM, a.N).start; });
  const int h = xcd_swizzle(blockIdx.x % a.Hq, a.Hq), kv = h / (a.Hq / a.Hkv);
  const int lane = threadIdx.x & 63, col = lane & 31, hi = lane >> 5;
  const int i0 = t * BM, w0 = i0 + wave_id() * 32;
  const T *Kb = a.K + int64_t(kv) * a.D, *Vb = a.V + int64_t(kv) * a.D;

  const int kmin = __builtin_amdgcn_readfirstlane(find_seq(cu, a.S, i0, a.N).start);
  const int kmax = min(i0 + BM, a.N);  // behind the last key
  const int turns = (kmax - kmin + BN - 1) / BN;
  const Stager<T, DP, BN, WAVES, ALIGNED> stage_k(a.ldk, a.D), stage_v(a.ldv, a.D);
  stage_k(k_tile(0), Kb, kmin, a.N);

  Operand<T> q[NT];
  const int i = w0 + col;
  const Seq seq = find_seq(cu, a.S, i, a.N);
  const T* qr = a.Q + int64_t(min(i, a.N - 1)) * a.ldq + int64_t(h) * a.D;
#pragma unroll
  for (int u = 0; u < NT; ++u) q[u] = load_row<T, ALIGNED>(qr, 16 * u + 8 * hi, a.D);
  // the wave's tiles nb .. ne - 1, from its first row's start to its last row; all of its
  // rows see a tile that begins at or behind the last row's start and ends at or before
  // the first row
  const int nb = min((max(__builtin_amdgcn_readfirstlane(seq.start), kmin) - kmin) / BN, turns);  // rows beyond N: none
  const int ne = min((w0 + 32 - kmin + BN - 1) / BN, turns);
  const int lastStart = __builtin_amdgcn_readlane(seq.start, 31);

  f32x16 o[NB];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int d = 0; d < NB; ++d) o[d] = zero16();
  const float c = a.scale * kLog2e, slack = 8.f / c;

  f32x16 s[KB];         // scores of a tile, then its weights
  Operand<T> p[KB][2];  // the weights as operands
  float mc;
  const auto scores = [&](int x, const char* kt) {
    s[x] = zero16();
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const Operand<T> k = L::by_rows(kt, 32 * x, u);
      s[x] = mma(k, q[u], s[x]);
    }
  };
  const auto values = [&](const char* vt) {
#pragma unroll
    for (int x = 0; x < KB; ++x)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int d = 0; d < NB; ++d) {
          const Operand<T> v = L::by_cols(vt, 32 * x + 16 * u, d);
          o[d] = mma(v, p[x][u], o[d]);
        }
  };
  const auto mask = [&](int k0) {
    // start <= j <= i in one comparison
    const uint32_t most = i - seq.start, at = k0 + 4 * hi - seq.start;
#pragma unroll
    for (int x = 0; x < KB; ++x)
#pragma unroll
      for (int v = 0; v < 16; ++v) s[x][v] = at + (32 * x + mfma32_row(v, 0)) <= most ? s[x][v] : -INFINITY;
  };
  // The reference m of a row's weights exp(s - m) stays until a score passes it by 2^8:
  // weights up to 2^8 lose nothing in a float, and the sums are seldom scaled (by f).
  const auto reference = [&] {
    float top = s[0][0];
#pragma unroll
    for (int x = 0; x < KB; ++x)
#pragma unroll
      for (int v = 0; v < 16; ++v) top = fmaxf(top, s[x][v]);
    top = join_halves(top, max2);
    const float mn = top > m + slack ? top : m;
    const float f = m == mn ? 1.f : __builtin_amdgcn_exp2f((m - mn) * c);
    l *= f;
    m = mn;
    mc = mn == -INFINITY ? 0.f : mn * c;
    return f;
  };
  const auto weights = [&](int x) {
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      s[x][v] = __builtin_amdgcn_exp2f(fmaf(s[x][v], c, -mc));
      sum[v & 1] += s[x][v];
    }
    l += sum[0] + sum[1];
  };
  const auto operands = [&](int x) {
    p[x][0] = as_operand<T>(s[x], 0);
    p[x][1] = as_operand<T>(s[x], 1);
  };
  const auto begin = [&](int n) {  // a turn's wait and copies
    wait_vmcnt<0>();
    __syncthreads();
    if (n + 2 < turns) stage_k(k_tile(n & 1), Kb, kmin + (n + 2) * BN, a.N);
    if (n >= 0 && n < turns) stage_v(v_tile(n & 1), Vb, kmin + n * BN, a.N);
  };
  // Turn n: the values of tile n - 1, the softmax of tile n and the scores of tile n + 1,
  // which are independent of each other, so that the matrix and the vector units work
  // at a time.
  int n = -1;
  for (; n < nb - 1; ++n) begin(n);
  begin(n);
#pragma unroll
  for (int x = 0; x < KB; ++x) scores(x, k_tile((n + 1) & 1));
  for (n = nb; n < ne; ++n) {
    begin(n);
    const int k0 = kmin + n * BN;
    if (!(k0 + BN - 1 <= w0 && k0 >= lastStart)) mask(k0);
    float f;
    if (n > nb) {
      const char* vt = v_tile((n + 1) & 1);
      values(vt);
      f = reference();
      weights(0);
    } else {
      f = reference();
      weights(0);
    }
    if (__any(f != 1.f)) {
#pragma unroll
      for (int d = 0; d < NB; ++d)
#pragma unroll
        for (int v = 0; v < 16; ++v) o[d][v] *= f;
    }
    // behind the wave's last tile the next scores are of no use
    const char* kt = k_tile((n + 1) & 1);
#pragma unroll
    for (int x = 0; x < KB; ++x) {
      operands(x);
      scores(x, kt);
      if (x + 1 < KB) weights(x + 1);
    }
  }
  begin(n);
  values(v_tile((n + 1) & 1));
  for (++n; n <= turns; ++n) begin(n);

  const bool in = seq.inside;
  const float sum = join_halves(l, sum2), inv = 1.f / sum;
  T* row = a.out + int64_t(min(i, a.N - 1)) * a.ldo + int64_t(h) * a.D;
  if (in) {
#pragma unroll
    for (int d = 0; d < NB; ++d) put_block<T, ALIGNED>(row, d, a.D, o[d], inv);
    if (hi == 0) a.lse[int64_t(h) * a.N + i] = fmaf(m, c, __builtin_amdgcn_logf(sum)) * kLn2;
  }
  // a NaN of the sum is one of a weight, and in every column
  const bool lost = sum != sum || far(m, c);
  bool bad = false;
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int v = 0; v < 16; ++v) bad = bad || !(fabsf(o[d][v]) < INFINITY);
  if (__any(in && (bad || lost))) {
    bool again = lost;
    if (__any(in && bad && !lost)) {
      const Spoilt sp = last_spoilt(Vb, a.ldv, min(__builtin_amdgcn_readfirstlane(seq.start), w0), w0, a.D);
#pragma unroll
      for (int d = 0; d < NB; ++d)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int at = 32 * d + mfma32_row(v, hi);
          const bool odd = unexplained(o[d][v], sp, at, seq.start);
          again = again || (at < a.D && odd);
        }
    }
    const uint64_t both = __ballot(in && again);
    for (uint32_t rows = uint32_t(both) | uint32_t(both >> 32); rows != 0; rows &= rows - 1) {
      const int r = __ffs(rows) - 1;
      fwd_row(a, h, kv, w0 + r, __builtin_amdgcn_readlane(seq.start, r), __builtin_amdgcn_readlane(int(lost), r));
    }
  }
}

// Few rows: a block owns 32 query rows, and its waves take a part of every tile of
// 32 WAVES keys each, with a softmax of their own; their sums are joined at the end.  Bound by
// the latency of one block's turns, a copy and two short products each: all of a tile's
// keys at a time make a quarter as many.  128 rows of 4 x 64 fp32 in one sequence: 7.8 us.
template <typename T, int DP, int WAVES, bool ALIGNED>
__global__ __launch_bounds__(64 * WAVES) void k_attn_fwd_few(AttnArgs<T> a) {
  using L = Tile<T, DP>;
  constexpr int NT = DP / 16, NB = DP / 32, BN = 32 * WAVES;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  __shared__ int32_t cu_lds[kCuLds];
  __shared__ float ms[WAVES][2][32];  // of each wave: reference and sum
  __shared__ uint32_t again[WAVES];   // rows to form again, for the sake of the wave's columns
  constexpr int TILE = BN * L::kRowBytes;
  char *const kt = smem, *const vt = smem + TILE;

  const int t = (a.N + 31) / 32 - 1 - blockIdx.x / a.Hq;
  const int h = xcd_swizzle(blockIdx.x % a.Hq, a.Hq), kv = h / (a.Hq / a.Hkv);
  const int lane = threadIdx.x & 63, col = lane & 31, hi = lane >> 5, w = wave_id();
  const int i0 = t * 32, i = i0 + col;
  const int32_t* cu = edges(a.cu, a.S, cu_lds);
  const T *Kb = a.K + int64_t(kv) * a.D, *Vb = a.V + int64_t(kv) * a.D;
  const Seq seq = find_seq(cu, a.S, i, a.N);
  const int kmin = __builtin_amdgcn_readfirstlane(seq.start);
  const int turns = (min(i0 + 32, a.N) - kmin + BN - 1) / BN;
  const Stager<T, DP, BN, WAVES, ALIGNED> stage_k(a.ldk, a.D), stage_v(a.ldv, a.D);
  const auto stage = [&](int n) {
    stage_k(kt, Kb, kmin + n * BN, a.N);
    stage_v(vt, Vb, kmin + n * BN, a.N);
  };
  stage(0);
  Operand<T> q[NT];
  const T* qr = a.Q + int64_t(min(i, a.N - 1)) * a.ldq + int64_t(h) * a.D;
#pragma unroll
  for (int u = 0; u < NT; ++u) q[u] = load_row<T, ALIGNED>(qr, 16 * u + 8 * hi, a.D);
  f32x16 o[NB];
#pragma unroll
  for (int d = 0; d < NB; ++d) o[d] = zero16();
  float m = -INFINITY, l = 0.f;
  const float c = a.scale * kLog2e;
  for (int n = 0; n < turns; ++n) {
    wait_vmcnt<0>();
    __syncthreads();
    const int k0 = kmin + n * BN + 32 * w;
    if (k0 < i0 + 32) {
      f32x16 s = zero16();
#pragma unroll
      for (int u = 0; u < NT; ++u) s = mma(L::by_rows(kt, 32 * w, u), q[u], s);
      const uint32_t most = i - seq.start, at = k0 + 4 * hi - seq.start;
      float top = -INFINITY;
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        s[v] = at + mfma32_row(v, 0) <= most ? s[v] : -INFINITY;
        top = fmaxf(top, s[v]);
      }
      const float mn = fmaxf(m, join_halves(top, max2));
      const float f = m == mn ? 1.f : __builtin_amdgcn_exp2f((m - mn) * c);
      const float mc = mn == -INFINITY ? 0.f : mn * c;
      m = mn;
      l *= f;
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        s[v] = __builtin_amdgcn_exp2f(fmaf(s[v], c, -mc));
        l += s[v];
      }
#pragma unroll
      for (int d = 0; d < NB; ++d) {
        o[d] *= f;
#pragma unroll
        for (int u = 0; u < 2; ++u) o[d] = mma(L::by_cols(vt, 32 * w + 16 * u, d), as_operand<T>(s, u), o[d]);
      }
    }
    if (n + 1 < turns) {
      __syncthreads();
      stage(n + 1);
    }
  }
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);  // [WAVES][DP][32]
  static_assert(WAVES * DP * 32 * 4 <= 2 * TILE, "the tiles' room");
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int v = 0; v < 16; ++v) part[(w * DP + 32 * d + mfma32_row(v, hi)) * 32 + col] = o[d][v];
  l = join_halves(l, sum2);
  if (hi == 0) {
    ms[w][0][col] = m;
    ms[w][1][col] = l;
  }
  __syncthreads();
  float f[WAVES], sum = 0.f;
  m = ms[0][0][col];
#pragma unroll
  for (int x = 1; x < WAVES; ++x) m = fmaxf(m, ms[x][0][col]);
#pragma unroll
  for (int x = 0; x < WAVES; ++x) {
    const float mx = ms[x][0][col];
    f[x] = mx == m ? 1.f : __builtin_amdgcn_exp2f((mx - m) * c);
    sum += f[x] * ms[x][1][col];
  }
  const float inv = 1.f / sum;
  // a thread's columns: a 2 WAVES-th of its row
  constexpr int PER = DP / (2 * WAVES);
  static_assert(PER % 4 == 0, "whole stores");
  const int c0 = (2 * w + hi) * PER;
  T* row = a.out + int64_t(min(i, a.N - 1)) * a.ldo + int64_t(h) * a.D;
  bool bad = false;
  float y[PER];
#pragma unroll
  for (int e = 0; e < PER; e += 4) {
#pragma unroll
    for (int k = e; k < e + 4; ++k) {
      y[k] = 0.f;
#pragma unroll
      for (int x = 0; x < WAVES; ++x) y[k] += f[x] * part[(x * DP + c0 + k) * 32 + col];
      bad = bad || (c0 + k < a.D && !(fabsf(y[k]) < INFINITY));
    }
    if (seq.inside)
      put4<T, ALIGNED>(row, c0 + e, a.D, y[e] * inv, y[e + 1] * inv, y[e + 2] * inv, y[e + 3] * inv);
  }
  if (seq.inside && hi == 0 && w == 0) a.lse[int64_t(h) * a.N + i] = fmaf(m, c, __builtin_amdgcn_logf(sum)) * kLn2;
  const bool lost = sum != sum || far(m, c);
  if (__syncthreads_or(seq.inside && (bad || lost))) {
    bool odd = lost;
    if (__any(seq.inside && bad && !lost)) {
      const Spoilt sp = last_spoilt(Vb, a.ldv, kmin, i0, a.D);
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const bool x = unexplained(y[k], sp, c0 + k, seq.start);
        odd = odd || (c0 + k < a.D && x);
      }
    }
    const uint64_t both = __ballot(seq.inside && odd);
    if (lane == 0) again[w] = uint32_t(both) | uint32_t(both >> 32);
    __syncthreads();
    uint32_t rows = 0;
#pragma unroll
    for (int x = 0; x < WAVES; ++x) rows |= again[x];
    for (int r = w; r < 32; r += WAVES)
      if ((rows >> r) & 1)
        fwd_row(a, h, kv, i0 + r, __builtin_amdgcn_readlane(seq.start, r), __builtin_amdgcn_readlane(int(lost), r));
  }
}

// ----------------------------------------------------------------- gradients --
// One row of gQ, in a wave, over its visible keys alone.
template <typename T>
__device__ __forceinline__ void dq_row(const AttnArgs<T>& a, int h, int kv, int i, int start) {
  const int64_t hd = int64_t(h) * a.D, kd = int64_t(kv) * a.D;
  const T *q = a.Q + i * a.ldq + hd, *go = a.gO + i * a.ldgo + hd;
  const float delta = dot_row(go, a.O + i * a.ldo + hd, a.D), lse = a.lse[int64_t(h) * a.N + i];
  LaneSum g;
  for (int j = start; j <= i && !g.lost(); j += 64) {
    const int n = min(64, i + 1 - j), at = j + min(int(threadIdx.x & 63), n - 1);
    const float p = exp2f((a.scale * dot_row(q, a.K + at * a.ldk + kd, a.D) - lse) * kLog2e);
    g.add(a.K + j * a.ldk + kd, a.ldk, n, p * (dot_row(go, a.V + at * a.ldv + kd, a.D) - delta) * a.scale, a.D);
  }
  g.put(a.gQ + i * a.ldgq + hd, a.D, 1.f);
}

// delta_i = gO_i . O_i, and gQ = scale sum_j p (gO . v - delta) k with p = exp(s - lse): three
// products a pair of rows, a wave's rows being query rows.  gQ, gK and gV in one pass
// would be five products for the seven of two kernels, but its other side's sums would
// have to be added in memory: by atomics, whose order changes the results, or as a
// partial matrix a block.  For k_attn_dkv the kernel leaves -lse / scale and -delta of every row.
// bf16: 16384 rows of 16 x 64 in sequences of 1 to 4099 171 us (753 TFLOP/s); 8192 of 16 x 128 in
// sequences of 2048 130 us (793).
// The matrix unit is busy in 38 % of the cycles, and vector instructions are issued in 53 % (128
// columns: 31), 4 a score: a tile's scores, weights, roundings and second products are one
// chain, with the other wave of the SIMD alone beside it.
template <typename T, int DP, int WAVES, int BN, int OCC, bool ALIGNED>
__global__ __launch_bounds__(64 * WAVES, OCC) void k_attn_dq(AttnArgs<T> a) {
  using L = Tile<T, DP>;
  constexpr int NT = DP / 16, NB = DP / 32, KB = BN / 32, BM = 32 * WAVES;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  __shared__ int32_t cu_lds[kCuLds];
  constexpr int TILE = BN * L::kRowBytes;
  const auto k_tile = [&](int b) { return smem + b * 2 * TILE; };
  const auto v_tile = [&](int b) { return smem + b * 2 * TILE + TILE; };

  const int tiles = (a.N + BM - 1) / BM;
  const int heads = a.Hq * a.splits;
  const int32_t* cu = edges(a.cu, a.S, cu_lds);
  const int t = ranked_tile(tiles, blockIdx.x / heads, [&](int x) { return min((x + 1) * BM, a.N) - find_seq(cu, a.S, x * BM, a.N).start; });
  const int sp = blockIdx.x % heads / a.Hq, h = xcd_swizzle(blockIdx.x % a.Hq, a.Hq), kv = h / (a.Hq / a.Hkv);
  const int lane = threadIdx.x & 63, col = lane & 31, hi = lane >> 5;
  const int i0 = t * BM, w0 = i0 + wave_id() * 32;
  const T *Kb = a.K + int64_t(kv) * a.D, *Vb = a.V + int64_t(kv) * a.D;

  // the split's tiles: sp, sp + splits, ... of the block's range
  const int kmin = __builtin_amdgcn_readfirstlane(find_seq(cu, a.S, i0, a.N).start) + sp * BN, step = a.splits * BN;
  const int kmax = min(i0 + BM, a.N);
  const int turns = (kmax - kmin + step - 1) / step;  // none where kmin is behind the range
  const Stager<T, DP, BN, WAVES, ALIGNED> stage_k(a.ldk, a.D), stage_v(a.ldv, a.D);
  const auto stage = [&](int n) {
    stage_k(k_tile(n & 1), Kb, kmin + n * step, a.N);
    stage_v(v_tile(n & 1), Vb, kmin + n * step, a.N);
  };
  if (turns > 0) stage(0);

  Operand<T> q[NT], go[NT];
  const int i = w0 + col;
  const int64_t r = min(i, a.N - 1);
  const Seq seq = find_seq(cu, a.S, i, a.N);
  const T *qr = a.Q + r * a.ldq + int64_t(h) * a.D, *gr = a.gO + r * a.ldgo + int64_t(h) * a.D;
  const T* orow = a.O + r * a.ldo + int64_t(h) * a.D;
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    q[u] = load_row<T, ALIGNED>(qr, 16 * u + 8 * hi, a.D);
    go[u] = load_row<T, ALIGNED>(gr, 16 * u + 8 * hi, a.D);
    const Operand<T> x = load_row<T, ALIGNED>(orow, 16 * u + 8 * hi, a.D);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(static_cast<float>(go[u].v[e]), static_cast<float>(x.v[e]), s);
  }
  const float delta = join_halves(s, sum2), lse2 = a.lse[int64_t(h) * a.N + r] * kLog2e;
  if (sp == 0 && hi == 0 && i < a.N) {
    a.rows[int64_t(2 * h) * a.N + i] = seq.inside ? -a.lse[int64_t(h) * a.N + i] / a.scale : 0.f;
    a.rows[int64_t(2 * h + 1) * a.N + i] = seq.inside ? -delta : 0.f;
  }
  const int first = __builtin_amdgcn_readfirstlane(seq.start);
  const int lastStart = __builtin_amdgcn_readlane(seq.start, 31);

  f32x16 g[NB];
#pragma unroll
  for (int d = 0; d < NB; ++d) g[d] = zero16();
  const float c = a.scale * kLog2e;

  for (int n = 0; n < turns; ++n) {
    wait_vmcnt<0>();
    __syncthreads();
    if (n + 1 < turns) stage(n + 1);
    const int k0 = kmin + n * step;
    if (k0 + BN <= first || k0 >= w0 + 32) continue;
    const bool whole = k0 + BN - 1 <= w0 && k0 >= lastStart;
    const char *kt = k_tile(n & 1), *vt = v_tile(n & 1);
#pragma unroll
    for (int x = 0; x < KB; ++x) {
      f32x16 s = zero16(), dp = zero16();
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        const Operand<T> k = L::by_rows(kt, 32 * x, u), v = L::by_rows(vt, 32 * x, u);
        s = mma(k, q[u], s);
        dp = mma(v, go[u], dp);
      }
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const float p = __builtin_amdgcn_exp2f(fmaf(s[v], c, -lse2));
        s[v] = p * (dp[v] - delta);
      }
      if (!whole) {
        const uint32_t most = i - seq.start, at = k0 + 32 * x + 4 * hi - seq.start;
#pragma unroll
        for (int v = 0; v < 16; ++v) s[v] = at + mfma32_row(v, 0) <= most ? s[v] : 0.f;
      }
      const Operand<T> ds[2] = {as_operand<T>(s, 0), as_operand<T>(s, 1)};
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int d = 0; d < NB; ++d) {
          const Operand<T> k = L::by_cols(kt, 32 * x + 16 * u, d);
          g[d] = mma(k, ds[u], g[d]);
        }
    }
  }

  const bool in = seq.inside;
  if (a.splits > 1) {
    float* row = a.part + ((int64_t(sp) * a.N + r) * a.Hq + h) * a.D;
    if (in) {
#pragma unroll
      for (int d = 0; d < NB; ++d) put_block<float, ALIGNED>(row, d, a.D, g[d], a.scale);
    }
    return;
  }
  T* row = a.gQ + r * a.ldgq + int64_t(h) * a.D;
  if (in) {
#pragma unroll
    for (int d = 0; d < NB; ++d) put_block<T, ALIGNED>(row, d, a.D, g[d], a.scale);
  }
  if (any_nan<NB>(g, in)) {
    for (int r = 0; r < 32; ++r)
      if (__builtin_amdgcn_readlane(int(in), r)) dq_row(a, h, kv, w0 + r, __builtin_amdgcn_readlane(seq.start, r));
  }
}

// One row of gK (V: of gV), in a wave, over the query rows that see it.
template <bool V, typename T>
__device__ __forceinline__ void dkv_row(const AttnArgs<T>& a, int kv, int j, int end) {
  const int64_t kd = int64_t(kv) * a.D;
  const int G = a.Hq / a.Hkv;
  const T *k = a.K + j * a.ldk + kd, *v = a.V + j * a.ldv + kd;
  LaneSum g;
  for (int h = kv * G; h < (kv + 1) * G; ++h) {
    const int64_t hd = int64_t(h) * a.D;
    const float* row = a.rows + int64_t(2 * h) * a.N;
    for (int i = j; i < end && !g.lost(); i += 64) {
      const int n = min(64, end - i), at = i + min(int(threadIdx.x & 63), n - 1);
      const float p = exp2f(a.scale * kLog2e * (dot_row(k, a.Q + at * a.ldq + hd, a.D) + row[at]));
      if constexpr (V)
        g.add(a.gO + i * a.ldgo + hd, a.ldgo, n, p, a.D);
      else
        g.add(a.Q + i * a.ldq + hd, a.ldq, n, p * (dot_row(v, a.gO + at * a.ldgo + hd, a.D) + row[a.N + at]) * a.scale, a.D);
    }
  }
  g.put(V ? a.gV + j * a.ldgv + kd : a.gK + j * a.ldgk + kd, a.D, 1.f);
}

// gV = sum_i p gO and gK = scale sum_i p (gO . v - delta) q: four products a pair of rows, a
// wave's rows being key rows; the query heads of a group one after the other, into the
// same sums, so that shared heads need no further pass.
// One chain a tile as for gQ (matrix unit busy in 37 to 38 % of the cycles, vector instructions
// issued in 35 %, at 128 columns 28) and, at 128 columns, few registers.  fp32 has one wave a
// SIMD and no other beside its chain (matrix unit 37 %).  bf16: 16384 rows of 16 x 64 in 4 key heads,
// sequences of 1 to 4099, 220-235 us and 16 to join (730-780 TFLOP/s); 8192 of 16 x 128, sequences
// of 2048, 156-174 us (790-880).  K in LDS and 8 waves a block (313 us for 257), operands read
// ahead of their products (243 for 252 at 64 columns, registers spilled at 128) and masks
// without a branch (283 for 255) were measured as well.
// K, V, gK and gV of 32 rows of 128 columns are 192 of the 256 registers that two waves a SIMD
// leave, and one pair of operands at a time can be on its way from LDS.  There V stays in LDS,
// another read for each of its products: 8192 rows of 16 x 128 156-174 us, 205-225 with V in
// registers.  Up to 96 columns both fit.
template <typename T, int DP>
constexpr bool v_in_lds = sizeof(T) == 2 && DP > 96;

template <typename T, int DP, int WAVES, int BN, int OCC, bool ALIGNED>
__global__ __launch_bounds__(64 * WAVES, OCC) void k_attn_dkv(AttnArgs<T> a) {
  using L = Tile<T, DP>;
  constexpr int NT = DP / 16, NB = DP / 32, QB = BN / 32, BM = 32 * WAVES;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  __shared__ int32_t cu_lds[kCuLds];
  __shared__ __attribute__((aligned(16))) float stats[2][2][BN];  // of the tile's rows: -lse / scale and -delta
  constexpr int TILE = BN * L::kRowBytes;
  const auto q_tile = [&](int b) { return smem + b * 2 * TILE; };
  const auto g_tile = [&](int b) { return smem + b * 2 * TILE + TILE; };
  constexpr bool VL = v_in_lds<T, DP>;  // the block's rows of V stay in LDS
  char* const vl = smem + 4 * TILE;

  const int heads = a.Hkv * a.splits;
  const int32_t* cu = edges(a.cu, a.S, cu_lds);
  const int t = ranked_tile((a.N + BM - 1) / BM, blockIdx.x / heads,
                            [&](int x) { return find_seq(cu, a.S, min((x + 1) * BM, a.N) - 1, a.N).end - x * BM; });
  const int sp = blockIdx.x % heads / a.Hkv, kv = xcd_swizzle(blockIdx.x % a.Hkv, a.Hkv);
  const int G = a.Hq / a.Hkv;
  const int lane = threadIdx.x & 63, col = lane & 31, hi = lane >> 5;
  const int j0 = t * BM, w0 = j0 + wave_id() * 32;

  const int last = min(j0 + BM, a.N) - 1;
  const int qmax = __builtin_amdgcn_readfirstlane(find_seq(cu, a.S, last, a.N).end);
  // the tiles of all heads one after the other; the split's are sp, sp + splits, ...
  const int per = (qmax - j0 + BN - 1) / BN, turns = (per * G - sp + a.splits - 1) / a.splits;
  const Stager<T, DP, BN, WAVES, ALIGNED> stage_q(a.ldq, a.D), stage_g(a.ldgo, a.D);
  const auto stage = [&](int n) {
    const int at = sp + n * a.splits, h = kv * G + at / per, i0 = j0 + at % per * BN;
    stage_q(q_tile(n & 1), a.Q + int64_t(h) * a.D, i0, a.N);
    stage_g(g_tile(n & 1), a.gO + int64_t(h) * a.D, i0, a.N);
    constexpr int UNITS = 2 * BN / 64;  // both rows' statistics, 4 bytes a lane
    if (wave_id() < UNITS) {
      const int x = wave_id() * 64 + lane;
      const uint32_t off = (uint32_t(x / BN) * a.N + min(x % BN, a.N - 1 - i0)) * 4;
      copy_lane4_to_lds(a.rows + int64_t(2 * h) * a.N + i0, off, lds_address(&stats[n & 1][0][0]) + wave_id() * 256);
    }
  };
  if (turns > 0) stage(0);
  if constexpr (VL)  // through registers, which puts zeros behind column D: gO's tile has none there
    Stager<T, DP, BM, WAVES, false>(a.ldv, a.D)(vl, a.V + int64_t(kv) * a.D, j0, a.N);

  Operand<T> k[NT], v[VL ? 1 : NT];
  const int j = w0 + col;
  const int64_t r = min(j, a.N - 1);
  const Seq seq = find_seq(cu, a.S, j, a.N);
  const T *kr = a.K + r * a.ldk + int64_t(kv) * a.D, *vr = a.V + r * a.ldv + int64_t(kv) * a.D;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    k[u] = load_row<T, ALIGNED>(kr, 16 * u + 8 * hi, a.D);
    if constexpr (!VL) v[u] = load_row<T, ALIGNED>(vr, 16 * u + 8 * hi, a.D);
  }
  const int firstEnd = __builtin_amdgcn_readfirstlane(seq.end);
  const int lastEnd = __builtin_amdgcn_readlane(seq.end, 31);

  f32x16 gk[NB], gv[NB];
#pragma unroll
  for (int d = 0; d < NB; ++d) gk[d] = gv[d] = zero16();
  const float c = a.scale * kLog2e;

  for (int n = 0; n < turns; ++n) {
    wait_vmcnt<0>();
    __syncthreads();
    if (n + 1 < turns) stage(n + 1);
    const int i0 = j0 + (sp + n * a.splits) % per * BN;
    if (i0 + BN <= w0 || i0 >= lastEnd) continue;
    const bool whole = i0 >= w0 + 31 && i0 + BN <= firstEnd;
    const char *qt = q_tile(n & 1), *gt = g_tile(n & 1);
#pragma unroll
    for (int x = 0; x < QB; ++x) {
      // the sums begin at the rows' -lse / scale and -delta, so that exp(scale s) is the weight
      // and the other the difference; fp32 adds the log-sum last, to lose nothing beside it
      f32x16 y, z;
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const f32x4 y4 = *reinterpret_cast<const f32x4*>(&stats[n & 1][0][32 * x + 2 * r + 4 * hi]);
        const f32x4 z4 = *reinterpret_cast<const f32x4*>(&stats[n & 1][1][32 * x + 2 * r + 4 * hi]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[r + e] = y4[e];
          z[r + e] = z4[e];
        }
      }
      constexpr bool LATE = sizeof(T) == 4;
      f32x16 s = LATE ? zero16() : y, dp = z;
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        const Operand<T> q = L::by_rows(qt, 32 * x, u), go = L::by_rows(gt, 32 * x, u);
        s = mma(q, k[u], s);
        if constexpr (VL)
          dp = mma(go, L::by_rows(vl, 32 * wave_id(), u), dp);
        else
          dp = mma(go, v[u], dp);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[r] = __builtin_amdgcn_exp2f((LATE ? s[r] + y[r] : s[r]) * c);
        dp[r] *= s[r];
      }
      if (!whole) {
        // j <= i < end in one comparison
        const uint32_t most = seq.end - j, at = i0 + 32 * x + 4 * hi - j;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const bool seen = at + mfma32_row(r, 0) < most;
          s[r] = seen ? s[r] : 0.f;
          dp[r] = seen ? dp[r] : 0.f;
        }
      }
      Operand<T> p[2], ds[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        p[u] = as_operand<T>(s, u);
        ds[u] = as_operand<T>(dp, u);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int d = 0; d < NB; ++d) {
          const Operand<T> go = L::by_cols(gt, 32 * x + 16 * u, d), q = L::by_cols(qt, 32 * x + 16 * u, d);
          gv[d] = mma(go, p[u], gv[d]);
          gk[d] = mma(q, ds[u], gk[d]);
        }
    }
  }

  const bool in = seq.inside;
#pragma unroll
  for (int y = 0; y < 2; ++y) {  // gK, then gV
    const f32x16(&g)[NB] = y == 0 ? gk : gv;
    const float f = y == 0 ? a.scale : 1.f;
    if (a.splits > 1) {
      float* row = a.part + (((int64_t(sp) * a.N + r) * 2 + y) * a.Hkv + kv) * a.D;
      if (in) {
#pragma unroll
        for (int d = 0; d < NB; ++d) put_block<float, ALIGNED>(row, d, a.D, g[d], f);
      }
      continue;
    }
    T* row = (y == 0 ? a.gK + r * a.ldgk : a.gV + r * a.ldgv) + int64_t(kv) * a.D;
    if (in) {
#pragma unroll
      for (int d = 0; d < NB; ++d) put_block<T, ALIGNED>(row, d, a.D, g[d], f);
    }
    if (!any_nan<NB>(g, in)) continue;
    for (int x = 0; x < 32; ++x) {
      if (!__builtin_amdgcn_readlane(int(in), x)) continue;
      const int end = __builtin_amdgcn_readlane(seq.end, x);
      if (y == 0)
        dkv_row<false>(a, kv, w0 + x, end);
      else
        dkv_row<true>(a, kv, w0 + x, end);
    }
  }
}

// The splits' sums, four columns a thread where they are aligned; ROWS rows a block, which
// looks at its rows again, head by head, where a sum is NaN.  In the order of the splits, so
// that results repeat.  Bound by memory: 16384 rows of 2 x 4 x 64 by two 16 us, 67 MB of sums read
// and 17 MB of bf16 written.  8 rows a block there (18 us by 4, 21 by 2: the edges are read
// by more blocks), 2 where rows are fewer (1999 rows of 2 x 2 x 80 by 16 8.6 us; 16.4 by 8, one
// split's load behind the other).
template <typename T, bool ALIGNED, int ROWS>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs<T> a, int keys) {
  constexpr int C = ALIGNED ? 4 : 1;
  __shared__ int32_t cu_lds[kCuLds];
  __shared__ Seq seq[ROWS];
  const int32_t* cu = edges(a.cu, a.S, cu_lds);
  const int H = keys ? a.Hkv : a.Hq, i0 = blockIdx.x * ROWS;
  if (threadIdx.x < ROWS) seq[threadIdx.x] = find_seq(cu, a.S, i0 + threadIdx.x, a.N);
  __syncthreads();
  const int half = H * a.D, width = keys ? 2 * half : half;  // of a partial row
  const int64_t plane = int64_t(a.N) * width;
  bool bad[2] = {false, false};  // of gQ or gK, and of gV
  for (int u = threadIdx.x; u < ROWS * (width / C); u += 256) {
    const int r = u / (width / C), c = u % (width / C) * C;
    if (!seq[r].inside) continue;
    const float* p = a.part + int64_t(i0 + r) * width + c;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    const auto part = [&](int s) {
      if constexpr (ALIGNED)
        return *reinterpret_cast<const f32x4*>(p + s * plane);
      else
        return f32x4{p[s * plane], 0.f, 0.f, 0.f};
    };
    int s = 0;
    for (; s + 4 <= a.splits; s += 4) {
      const f32x4 y[4] = {part(s), part(s + 1), part(s + 2), part(s + 3)};
#pragma unroll
      for (int k = 0; k < 4; ++k) x += y[k];
    }
    for (; s < a.splits; ++s) x += part(s);
    T* row = !keys ? a.gQ + (i0 + r) * a.ldgq : c < half ? a.gK + (i0 + r) * a.ldgk : a.gV + (i0 + r) * a.ldgv;
    const int at = c < half ? c : c - half;
    if constexpr (ALIGNED) {
      put4<T, true>(row, at, half, x[0], x[1], x[2], x[3]);
#pragma unroll
      for (int k = 1; k < 4; ++k) x[0] = x[k] != x[k] ? x[k] : x[0];
    } else {
      row[at] = from_f32<T>(x[0]);
    }
    (c < half ? bad[0] : bad[1]) |= x[0] != x[0];
  }
  const bool first = __syncthreads_or(bad[0]), second = __syncthreads_or(bad[1]);
  if (!first && !second) return;
  for (int u = wave_id(); u < ROWS * H; u += 4) {
    const int r = u / H, h = u % H;
    if (!seq[r].inside) continue;
    if (!keys) {
      dq_row(a, h, h / (a.Hq / a.Hkv), i0 + r, seq[r].start);
    } else {
      if (first) dkv_row<false>(a, h, i0 + r, seq[r].end);
      if (second) dkv_row<true>(a, h, i0 + r, seq[r].end);
    }
  }
}

// ------------------------------------------------------------------- launches --
template <auto K, int LDS, typename T>
void go(const AttnArgs<T>& a, int64_t blocks, int waves, hipStream_t s) {
  hipLaunchKernelGGL(K, dim3(uint32_t(blocks)), dim3(64 * waves), (LdsLimit<K, LDS>::bytes()), s, a);
}
template <typename T, int DP, int BN>
constexpr int kLds = 4 * BN * Tile<T, DP>::kRowBytes;  // two buffers of two tiles

constexpr int kWaves = 4, kRows = 32 * kWaves;  // rows of a block of the three kernels
int64_t row_blocks(int64_t N, int64_t heads) { return (N + kRows - 1) / kRows * heads; }

// Below 256 blocks of 128 rows, one a CU, blocks of 32 rows whose waves share the keys
// (1024 rows of 8 x 64 bf16: 12.7 against 18.5 us, 2000 of 8 x 128: 35 against 48; with 512
// blocks, 4096 of 16 x 64, 87 against 68).
template <typename T, int DP, bool ALIGNED>
void fwd_t(const AttnArgs<T>& a, hipStream_t s) {
  const int64_t blocks = row_blocks(a.N, a.Hq);
  if (blocks < 256)
    return go<k_attn_fwd_few<T, DP, kWaves, ALIGNED>, 2 * kRows * Tile<T, DP>::kRowBytes>(
        a, (int64_t(a.N) + 31) / 32 * a.Hq, kWaves, s);
  constexpr int BN = sizeof(T) == 2 ? 64 : 32, OCC = sizeof(T) == 2 ? 2 : 1;
  go<k_attn_fwd<T, DP, kWaves, BN, OCC, ALIGNED>, kLds<T, DP, BN>>(a, blocks, kWaves, s);
}

// Backward with few blocks: the range of a block is split over several, and their sums
// are joined by a further launch.  gQ: up to 400 blocks (1999 rows of 6 x 80 fp32, 96 blocks: 194
// us whole, 64 by 4, 69 by 6, 70 by 8, and the join).  gK and gV, whose blocks walk over all rows of
// all heads of a group: up to 1024 (the same with 2 key heads, 32 blocks: 771 us whole, 126 by 8,
// 83 by 16, 82 by 24, 94 by 32;
// 16384 rows of 16 x 64 in 4 key heads, bf16, 512 blocks and sequences of 1 to 4099: 376 us whole, 291
// by 2, 289 by 4; 8192 rows of 16 x 128, 1024 blocks: 257 whole, 412 by 2).
int splits(int64_t blocks, int64_t want) { return int(std::max<int64_t>(1, std::min<int64_t>(16, want / blocks))); }
int dq_splits(int64_t N, int64_t Hq) { return splits(row_blocks(N, Hq), 400); }
int dkv_splits(int64_t N, int64_t Hkv) { return splits(row_blocks(N, Hkv), 1024); }

// Two waves a SIMD in bf16: 256 registers a thread, and at 128 columns 80 KB of LDS a block, which
// the block's V and tiles of 32 rows take (before V was there 225 us; by 64, one wave a SIMD, 255).  Elsewhere
// tiles of 64 (16384 rows of 16 x 64: 251 us against 296 by 32; 8192 of 16 x 96: 154, 168).
template <typename T, int DP, bool ALIGNED>
void bwd_t(AttnArgs<T> a, hipStream_t s) {
  constexpr bool B = sizeof(T) == 2;
  constexpr int OCC = B ? 2 : 1, BQ = B ? 64 : 32, BK = B && DP <= 96 ? 64 : 32;
  a.splits = dq_splits(a.N, a.Hq);
  go<k_attn_dq<T, DP, kWaves, BQ, OCC, ALIGNED>, kLds<T, DP, BQ>>(a, row_blocks(a.N, a.Hq) * a.splits, kWaves, s);
  const auto join = [&](int keys) {
    if (a.splits == 1) return;
    if (a.N >= 8192)
      hipLaunchKernelGGL((k_attn_join<T, ALIGNED, 8>), dim3(uint32_t((a.N + 7) / 8)), dim3(256), 0, s, a, keys);
    else
      hipLaunchKernelGGL((k_attn_join<T, ALIGNED, 2>), dim3(uint32_t((a.N + 1) / 2)), dim3(256), 0, s, a, keys);
  };
  join(0);
  a.splits = dkv_splits(a.N, a.Hkv);
  constexpr int VL = v_in_lds<T, DP> ? kRows * Tile<T, DP>::kRowBytes : 0;
  go<k_attn_dkv<T, DP, kWaves, BK, OCC, ALIGNED>, kLds<T, DP, BK> + VL>(a, row_blocks(a.N, a.Hkv) * a.splits, kWaves, s);
  join(1);
}

// workspace: two floats a row and query head, then the partial sums
int64_t attn_rows_floats(int64_t N, int64_t Hq) { return (2 * N * Hq + 3) / 4 * 4; }

template <typename T, bool BWD>
void attn_t(const Attn& c, hipStream_t s) {
  AttnArgs<T> a;
  a.Q = static_cast<const T*>(c.Q);
  a.K = static_cast<const T*>(c.K);
  a.V = static_cast<const T*>(c.V);
  a.O = static_cast<const T*>(c.O);
  a.gO = static_cast<const T*>(c.gO);
  a.out = static_cast<T*>(c.out);
  a.gQ = static_cast<T*>(c.gQ);
  a.gK = static_cast<T*>(c.gK);
  a.gV = static_cast<T*>(c.gV);
  a.cu = c.cu;
  a.lse = c.lse;
  a.rows = c.rows;
  a.part = c.rows ? c.rows + attn_rows_floats(c.N, c.Hq) : nullptr;
  a.splits = 1;
  a.ldq = c.ldq;
  a.ldk = c.ldk;
  a.ldv = c.ldv;
  a.ldo = c.ldo;
  a.ldgo = c.ldgo;
  a.ldgq = c.ldgq;
  a.ldgk = c.ldgk;
  a.ldgv = c.ldgv;
  a.scale = c.scale;
  a.S = int(c.S);
  a.N = int(c.N);
  a.Hq = int(c.Hq);
  a.Hkv = int(c.Hkv);
  a.D = int(c.D);
  uintptr_t at = 0;
  for (const void* p : {c.Q, c.K, c.V, c.O, c.gO, static_cast<const void*>(c.out), static_cast<const void*>(c.gQ),
                        static_cast<const void*>(c.gK), static_cast<const void*>(c.gV)})
    at |= reinterpret_cast<uintptr_t>(p);
  for (int64_t n : {c.D, c.ldq, c.ldk, c.ldv, c.ldo, c.ldgo, c.ldgq, c.ldgk, c.ldgv}) at |= uintptr_t(n) * sizeof(T);
  const auto with = [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    if constexpr (BWD)
      at % 16 == 0 ? bwd_t<T, DP, true>(a, s) : bwd_t<T, DP, false>(a, s);
    else
      at % 16 == 0 ? fwd_t<T, DP, true>(a, s) : fwd_t<T, DP, false>(a, s);
  };
  if (c.D <= 64) return with(std::integral_constant<int, 64>{});
  if (c.D <= 96) return with(std::integral_constant<int, 96>{});
  with(std::integral_constant<int, 128>{});
}

}  // namespace

}  // namespace mapl
