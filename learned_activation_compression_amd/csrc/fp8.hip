// Matrix products in 8-bit floating point (e4m3) with a power-of-two scale for
// each block of 128.  Formulas and roles of the packs: include/mapl_stage.h.
// The packs' layout and the rounding: e4m3.h.
#include <type_traits>

#include "e4m3.h"
#include "internal.h"
#include "vec8.h"

namespace mapl {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------- pack --
// A block takes 128 rows x 128 columns of X.  Thread (i, j) = (tid / 8, tid % 8)
// holds rows i + 32 k (k = 0..3), columns 16 j .. 16 j + 15.  The row operand
// needs the sizes of 8 neighbouring lanes only.  The column operand goes through
// LDS: wave w then holds rows 32 w .. 32 w + 31 of two columns per lane.  16384 x
// 1024 bf16 out of memory: the column operand 13.8 us (3.6 TB/s), both 17.0 (3.9);
// with every value tested for infinity and NaN (abs_max) 15.7 and 19.7.
template <typename T, RowMode MODE, bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void k_fp8_pack(const T* X, View pr, View pc, int square, int64_t R, int64_t C) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  T* tile = reinterpret_cast<T*>(smem);
  __shared__ float red[4 * 128];
  const int tid = threadIdx.x, i0 = tid >> 3, j = tid & 7;
  const uint32_t nkb = static_cast<uint32_t>((C + 127) / 128);
  const int64_t kb = blockIdx.x % nkb, rb = blockIdx.x / nkb;
  const int64_t c = kb * 128 + 16 * j;
  float v[4][16], am[4];
  bool bad[4];
  Fetch<T, MODE> f[4][2];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const T* row = X + min(rb * 128 + 32 * k + i0, R - 1) * C;
    f[k][0].issue(row, c, C);
    f[k][1].issue(row, c + 8, C);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool in = rb * 128 + 32 * k + i0 < R;
    const Raw8<T> lo = f[k][0].value(c, C, in), hi = f[k][1].value(c + 8, C, in);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[k][i] = lo.get(i);
      v[k][8 + i] = hi.get(i);
    }
    float m = abs_max<16>(v[k], bad[k]);
    m = fmaxf(m, __shfl_xor(m, 1));
    m = fmaxf(m, __shfl_xor(m, 2));
    am[k] = fmaxf(m, __shfl_xor(m, 4));
  }
  if (square) {
    float m = fmaxf(fmaxf(am[0], am[1]), fmaxf(am[2], am[3]));
#pragma unroll
    for (int s = 8; s < 64; s <<= 1) m = fmaxf(m, __shfl_xor(m, s));
    if ((tid & 63) == 0) red[tid >> 6] = m;
    __syncthreads();
    am[0] = am[1] = am[2] = am[3] = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    __syncthreads();
  }
  if constexpr (ROWS) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t rt = rb * 4 + k;
      if (rt < pr.RT) {
        const int e = block_exp(am[k]);
        *reinterpret_cast<u32x4*>(pr.code + (rt * pr.KB + kb) * 4096 + unit_off(i0, j)) = codes16(v[k], pow2_neg(e), bad[k]);
        if (j == 0) pr.exp[kb * pr.exp_stride + rt * 32 + i0] = static_cast<uint8_t>(e);
      }
    }
  }
  if constexpr (COLS) {
    // row stride 130 elements: a wave's rows start in different banks
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        T* q = tile + (32 * k + i0) * 130 + 16 * j + i;
        if constexpr (sizeof(T) == 2)
          *reinterpret_cast<uint32_t*>(q) = pack2bf(v[k][i], v[k][i + 1]);
        else
          *reinterpret_cast<u32x2*>(q) = u32x2{__float_as_uint(v[k][i]), __float_as_uint(v[k][i + 1])};
      }
    __syncthreads();
    const int w = tid >> 6, l = tid & 63;
    float a0[32], a1[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const T* q = tile + (32 * w + i) * 130 + 2 * l;
      if constexpr (sizeof(T) == 2) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(q);
        a0[i] = __uint_as_float(u << 16);
        a1[i] = __uint_as_float(u & 0xffff0000u);
      } else {
        const u32x2 u = *reinterpret_cast<const u32x2*>(q);
        a0[i] = __uint_as_float(u[0]);
        a1[i] = __uint_as_float(u[1]);
      }
    }
    bool bad0, bad1;
    float m0 = abs_max<32>(a0, bad0), m1 = abs_max<32>(a1, bad1);
    if (square) {
      m0 = m1 = am[0];
    } else {
      red[w * 128 + 2 * l] = m0;
      red[w * 128 + 2 * l + 1] = m1;
      __syncthreads();
      m0 = m1 = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        m0 = fmaxf(m0, red[k * 128 + 2 * l]);
        m1 = fmaxf(m1, red[k * 128 + 2 * l + 1]);
      }
    }
    // operand row kb * 128 + 2 l (+ 1), columns rb * 128 + 32 w + 0..31: j = 2 w, 2 w + 1
    const int e0 = block_exp(m0), e1 = block_exp(m1);
    const int64_t rt = kb * 4 + (l >> 4);
    if (rt < pc.RT) {
      uint8_t* base = pc.code + (rt * pc.KB + rb) * 4096;
      const int r = (2 * l) & 31;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        *reinterpret_cast<u32x4*>(base + unit_off(r, 2 * w + h)) = codes16(a0 + 16 * h, pow2_neg(e0), bad0);
        *reinterpret_cast<u32x4*>(base + unit_off(r + 1, 2 * w + h)) = codes16(a1 + 16 * h, pow2_neg(e1), bad1);
      }
      if (w == 0) {
        uint8_t* ex = pc.exp + rb * pc.exp_stride + rt * 32 + r;
        ex[0] = static_cast<uint8_t>(e0);
        ex[1] = static_cast<uint8_t>(e1);
      }
    }
  }
}

// The row operand alone, scaled by rows: 32 rows x 512 columns a block, so that a
// row is read 1 KB at a time and the codes leave as 16 KB in one piece (32768 x 2048
// bf16 out of memory: 39 us, 5.2 TB/s; by 128 x 128 tiles 4 us more).
template <typename T, RowMode MODE>
__global__ __launch_bounds__(256) void k_fp8_pack_rows(const T* X, View p, int64_t R, int64_t C) {
  const int i0 = threadIdx.x >> 3, j = threadIdx.x & 7;
  const uint32_t nq = static_cast<uint32_t>((p.KB + 3) / 4);
  const int64_t kb0 = int64_t(blockIdx.x % nq) * 4, rt = blockIdx.x / nq;
  const bool in = rt * 32 + i0 < R;
  const T* row = X + min(rt * 32 + i0, R - 1) * C;
  Fetch<T, MODE> f[4][2];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[k][0].issue(row, (kb0 + k) * 128 + 16 * j, C);
    f[k][1].issue(row, (kb0 + k) * 128 + 16 * j + 8, C);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t kb = kb0 + k, c = kb * 128 + 16 * j;
    const Raw8<T> lo = f[k][0].value(c, C, in), hi = f[k][1].value(c + 8, C, in);
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = lo.get(i);
      v[8 + i] = hi.get(i);
    }
    bool bad;
    float m = abs_max<16>(v, bad);
    m = fmaxf(m, __shfl_xor(m, 1));
    m = fmaxf(m, __shfl_xor(m, 2));
    m = fmaxf(m, __shfl_xor(m, 4));
    if (kb < p.KB) {
      const int e = block_exp(m);
      *reinterpret_cast<u32x4*>(p.code + (rt * p.KB + kb) * 4096 + unit_off(i0, j)) = codes16(v, pow2_neg(e), bad);
      if (j == 0) p.exp[kb * p.exp_stride + rt * 32 + i0] = static_cast<uint8_t>(e);
    }
  }
}

// -------------------------------------------------------------------- unpack --
// As k_fp8_pack_rows: 32 rows x 512 columns a block, 16 columns a thread and step.
// 16384 x 1024 to bf16 in 11 us, 4.6 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void k_fp8_unpack(View p, T* X, int64_t rows, int64_t cols) {
  const uint32_t nq = static_cast<uint32_t>((p.KB + 3) / 4);
  const int64_t kb0 = int64_t(blockIdx.x % nq) * 4, rt = blockIdx.x / nq;
  const int r = threadIdx.x >> 3, j = threadIdx.x & 7;
  const int64_t row = rt * 32 + r;
  if (row >= rows) return;
  u32x4 code[4];
  uint8_t e[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t kb = min(kb0 + k, p.KB - 1);
    code[k] = *reinterpret_cast<const u32x4*>(p.code + (rt * p.KB + kb) * 4096 + unit_off(r, j));
    e[k] = p.exp[kb * p.exp_stride + row];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t c = (kb0 + k) * 128 + 16 * j;
    if (c >= cols) break;
    const float s = __uint_as_float(static_cast<uint32_t>(e[k]) << 23);
    float v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(code[k][i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(code[k][i], true);
      v[4 * i] = lo[0] * s;
      v[4 * i + 1] = lo[1] * s;
      v[4 * i + 2] = hi[0] * s;
      v[4 * i + 3] = hi[1] * s;
    }
    T* out = X + row * cols + c;
    store8(out, v, static_cast<int>(min(cols - c, int64_t(8))));
    if (cols - c > 8) store8(out + 8, v + 8, static_cast<int>(min(cols - c - 8, int64_t(8))));
  }
}

// ---------------------------------------------------------------------- gemm --
__device__ __forceinline__ f32x16 mfma_e4m3(i32x8 a, i32x8 b, f32x16 c, int ea, int eb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, ea, 0, eb);
}

__device__ __forceinline__ i32x8 ld_frag(const char* p) {  // pieces h = 0 and 1 of a step, this lane's 16 bytes each
  const u32x4 a = *reinterpret_cast<const u32x4*>(p), b = *reinterpret_cast<const u32x4*>(p + 1024);
  return i32x8{int(a[0]), int(a[1]), int(a[2]), int(a[3]), int(b[0]), int(b[1]), int(b[2]), int(b[3])};
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// 8 codes times a power of two, as bf16: exact (4 significant bits)
__device__ __forceinline__ bf16x8 widen8(int lo, int hi, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// acc += a b^T of one MFMA tile over 64 columns; see Tile for EXACT
template <bool EXACT>
__device__ __forceinline__ f32x16 mac64(i32x8 b, i32x8 a, int eb, int ea, f32x16 acc) {
  if constexpr (!EXACT) {
    return mfma_e4m3(b, a, acc, eb, ea);
  } else {
    const float sa = __uint_as_float(uint32_t(ea) << 23), sb = __uint_as_float(uint32_t(eb) << 23);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      acc = mfma_bf16_32x32x16(widen8(b[2 * c], b[2 * c + 1], sb), widen8(a[2 * c], a[2 * c + 1], sa), acc);
    return acc;
  }
}

struct GemmArgs {
  View A, B;
  void* C;
  int64_t M, N;
  int accumulate;
  int splits;      // parts of the contraction; more than one: partial sums [splits][M][N] fp32 in C
  int64_t kb_per;  // blocks of 128 in each part
};

// Tile of (WM FM) x (WN FN) units of 32: WM x WN waves of FM x FN MFMA tiles.
// B (columns of C) is the matrix cores' row operand and A their column operand,
// so a lane's accumulators run along a row of C.
//
// Two ways to multiply, by the output's type (EXACT):
//  - bf16: the scaled e4m3 matrix instruction, 2.0x the rate of the other.  Before
//    they enter the fp32 accumulator it cuts the products of each 8 columns,
//    towards zero, to multiples of 2^(e - 13), e the largest sum of two factors'
//    exponents among the 8 (measured with factors placed one by one): less than
//    7 2^-13 = 8.5e-4 of the sum of absolute values at worst.  On data of random
//    sign that averages out: 1.6e-5 of it at K = 64, 2.0e-6 at 1024, 7e-7 at 8192
//    (the largest of 65536 outputs, beyond their rounding), against 2^-8 of the
//    output for its own rounding and 2^-4 for that of the codes.
//  - fp32 (weight gradients): the codes times their scales are widened to bf16,
//    which holds them exactly, and go through the bf16 instruction, whose sums
//    are fp32 throughout (1e-8 on the same data).
template <int WM, int WN, int FM, int FN, int NS>
struct Tile {
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int kBM = WM * FM, kBN = WN * FN;  // units of 32 rows
  static constexpr int kUnits = kBM + kBN;
  static constexpr int kStage = kUnits * 4096 + 512;   // codes, then 256 + 256 bytes of exponents
  static constexpr int kPieces = kUnits * 4 / kWaves;  // 1 KB pieces each wave copies per stage
  static constexpr int kLds = NS * kStage;
  static_assert(kUnits * 4 % kWaves == 0 && kPieces % 4 == 0 && kPieces % FM == 0, "every wave copies whole units");
  static_assert(kLds <= kMaxLdsBytes && kBM <= 8 && kBN <= 8, "tile");
};

// One row of a wave's output block from LDS to C: 16 bytes per lane.
__device__ __forceinline__ void put16(bf16_t* c, const char* src, int left, int) {
  const u32x4 v = *reinterpret_cast<const u32x4*>(src);
  if (left >= 8)
    st8_any(c, v);
  else
    st_tail(c, v, left);
}
__device__ __forceinline__ void put16(float* c, const char* src, int left, int accumulate) {
  f32x4 v = *reinterpret_cast<const f32x4*>(src);
  if (accumulate) v += __builtin_bit_cast(f32x4, left >= 4 ? ld16B(c) : ld_tail4(c, left));
  if (left >= 4)
    st16B(c, __builtin_bit_cast(u32x4, v));
  else
    st_tail4(c, __builtin_bit_cast(u32x4, v), left);
}

// The loop runs NS - 1 stages (of 128 columns) ahead in LDS and one step (64
// columns) ahead in registers, with one barrier a stage: behind it the stage just
// read is free for the copy of the stage NS later, and the next one is complete.
// 8192 x 8192 x 8192: 389 us, 2830 TFLOP/s, where MFMAs alone on zeros reach 5000.
// Without the copies (the same operands over and over) 4096 x 4096 x 8192 takes 90
// instead of 101 us, without the reads from LDS 99: the matrix cores are the bound,
// at the clock that random data leaves them.  32768 x 8192 x 2048 takes 520 to 555 us,
// as its 512 MB of C leave in bursts; 128 x 256 tiles, two workgroups a CU, spread them
// and gain nothing (565 us).  Widened operands (EXACT): 8192 x 8192 x 4096 in 400 us,
// 1370 TFLOP/s.
template <typename T, bool EXACT, int WM, int WN, int FM, int FN, int NS>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_fp8_gemm(GemmArgs g) {
  using TL = Tile<WM, WN, FM, FN, NS>;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int w = wave_id(), l = threadIdx.x & 63, wm = w / WN, wn = w % WN;
  const uint32_t tiles_m = static_cast<uint32_t>((g.A.RT + TL::kBM - 1) / TL::kBM);
  const uint32_t tiles_n = static_cast<uint32_t>((g.B.RT + TL::kBN - 1) / TL::kBN);
  // the tiles of an XCD are neighbours: groups of 8 tile rows, column by column
  uint32_t id = xcd_swizzle(blockIdx.x, gridDim.x);
  const uint32_t split = id / (tiles_m * tiles_n);
  id -= split * tiles_m * tiles_n;
  const uint32_t grp = id / (8 * tiles_n), gh = min(8u, tiles_m - 8 * grp), in = id - grp * 8 * tiles_n;
  const int64_t tm = int64_t(8 * grp + in % gh) * TL::kBM, tn = int64_t(in / gh) * TL::kBN;  // first unit rows
  const int64_t KB = g.A.KB, k0 = split * g.kb_per, k1 = min(k0 + g.kb_per, KB);

  // this wave's units of a stage (unit rows past the end repeat the last one)
  const uint8_t* src[TL::kPieces / 4];
#pragma unroll
  for (int i = 0; i < TL::kPieces / 4; ++i) {
    const int u = w * (TL::kPieces / 4) + i;
    const bool isA = u < TL::kBM;
    const int64_t rt = isA ? min(tm + u, g.A.RT - 1) : min(tn + (u - TL::kBM), g.B.RT - 1);
    src[i] = (isA ? g.A.code : g.B.code) + rt * KB * 4096;
  }
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)(smem)));
  const uint8_t* exps = (w & 1) ? g.B.exp + tn * 32 : g.A.exp + tm * 32;
  const int64_t exp_stride = (w & 1) ? g.B.exp_stride : g.A.exp_stride;
  const auto slot = [](int64_t kb) { return static_cast<uint32_t>(kb) % NS; };
  // part i of FM of the copies of a stage
  auto fetch = [&](int64_t kb, int i) {
    const uint32_t st = lds0 + slot(kb) * TL::kStage;
#pragma unroll
    for (int p = i * (TL::kPieces / FM); p < (i + 1) * (TL::kPieces / FM); ++p)
      copy_lane16_to_lds(src[p >> 2] + kb * 4096 + (p & 3) * 1024, l * 16, st + (w * TL::kPieces + p) * 1024);
    // even waves copy A's exponents, odd ones B's: more often than needed, but without a branch
    if (i == 0) copy_lane4_to_lds(exps + kb * exp_stride, l * 4, st + TL::kUnits * 4096 + (w & 1) * 256);
  };

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int k = 0; k < FN; ++k)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][k][e] = 0.f;

  struct Step {  // operands of 64 columns
    i32x8 a[FM], b[FN];
    int ea[FM], eb[FN];
  };
  Step s0, s1;
  // part i of FM of the operands of step s of stage kb; the column operand first, every row needs it
  auto read = [&](Step& st, int64_t kb, int s, int i) {
    const char* at = smem + slot(kb) * TL::kStage + s * 2048 + l * 16;
#pragma unroll
    for (int f = i * (FM + FN) / FM; f < (i + 1) * (FM + FN) / FM; ++f) {
      if (f < FN)
        st.b[f] = ld_frag(at + (TL::kBM + wn * FN + f) * 4096);
      else
        st.a[f - FN] = ld_frag(at + (wm * FM + f - FN) * 4096);
    }
  };
  auto read_exp = [&](Step& st, int64_t kb) {
    const char* ex = smem + slot(kb) * TL::kStage + TL::kUnits * 4096 + (l & 31);
#pragma unroll
    for (int i = 0; i < FM; ++i) st.ea[i] = static_cast<uint8_t>(ex[(wm * FM + i) * 32]);
#pragma unroll
    for (int i = 0; i < FN; ++i) st.eb[i] = static_cast<uint8_t>(ex[256 + (wn * FN + i) * 32]);
  };
  // row i of the wave's MFMA tiles
  auto multiply = [&](const Step& st, int i) {
    if constexpr (!EXACT) {
#pragma unroll
      for (int k = 0; k < FN; ++k) acc[i][k] = mfma_e4m3(st.b[k], st.a[i], acc[i][k], st.eb[k], st.ea[i]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bf16x8 wa = widen8(st.a[i][2 * c], st.a[i][2 * c + 1], __uint_as_float(uint32_t(st.ea[i]) << 23));
#pragma unroll
        for (int k = 0; k < FN; ++k)
          acc[i][k] = mfma_bf16_32x32x16(
              widen8(st.b[k][2 * c], st.b[k][2 * c + 1], __uint_as_float(uint32_t(st.eb[k]) << 23)), wa, acc[i][k]);
      }
    }
  };

  for (int64_t kb = k0; kb < min(k0 + NS, k1); ++kb)
#pragma unroll
    for (int i = 0; i < FM; ++i) fetch(kb, i);
  if (k0 + NS <= k1)
    wait_vmcnt<(NS - 1) * (TL::kPieces + 1)>();  // the first stage: the others may be on their way
  else
    wait_vmcnt<0>();
  __syncthreads();
  read_exp(s0, k0);
#pragma unroll
  for (int i = 0; i < FM; ++i) read(s0, k0, 0, i);
  // One stage.  sched_barrier: each part's reads and copies are issued beside its
  // MFMAs, not in one run ahead of them.  A branch in here would let the compiler
  // sink the MFMAs below it, so the last NS stages are bodies of their own.
  auto stage = [&](int64_t kb, auto next, auto copy) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      read(s1, kb, 1, i);
      multiply(s0, i);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) s1.ea[i] = s0.ea[i];
#pragma unroll
    for (int i = 0; i < FN; ++i) s1.eb[i] = s0.eb[i];
    if constexpr (next) {
      // stage kb + 1 is there when only the NS - 2 behind it are outstanding; none is issued any more near the end
      wait_vmcnt<copy ? (NS - 2) * (TL::kPieces + 1) : 0>();
      __syncthreads();
      read_exp(s0, kb + 1);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if constexpr (copy) fetch(kb + NS, i);
      if constexpr (next) read(s0, kb + 1, 0, i);
      multiply(s1, i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int64_t kb = k0;
  for (; kb + NS < k1; ++kb) stage(kb, std::true_type{}, std::true_type{});
  for (; kb + 1 < k1; ++kb) stage(kb, std::true_type{}, std::false_type{});
  stage(kb, std::false_type{}, std::false_type{});

  // acc[i][k]: row (tm + wm FM + i) * 32 + (l & 31) of C, columns (tn + wn FN + k) * 32 + mfma32_row(v, l >> 5).
  // 32 rows at a time go through LDS, so that a row's columns leave in 16-byte pieces.
  T* C = static_cast<T*>(g.C) + (g.splits > 1 ? split * g.M * g.N : 0);
  constexpr int kRow = FN * 32 * int(sizeof(T)) + 16;  // bytes of a row, and 16 to spread the banks
  static_assert(TL::kWaves * 32 * kRow <= TL::kLds, "epilogue staging");
  constexpr int kPer = 16 / int(sizeof(T)), kLanes = FN * 32 / kPer, kRows = 64 / kLanes;  // lanes of a row, rows at once
  char* block = smem + w * (32 * kRow);
  const int64_t n0 = (tn + wn * FN) * 32 + (l % kLanes) * kPer;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m0 = (tm + wm * FM + i) * 32;
#pragma unroll
    for (int k = 0; k < FN; ++k)
#pragma unroll
      for (int v = 0; v < 16; v += 4) {
        char* q = block + (l & 31) * kRow + (k * 32 + mfma32_row(v, l >> 5)) * int(sizeof(T));
        if constexpr (sizeof(T) == 2)
          *reinterpret_cast<u32x2*>(q) = u32x2{pack2bf(acc[i][k][v], acc[i][k][v + 1]), pack2bf(acc[i][k][v + 2], acc[i][k][v + 3])};
        else
          *reinterpret_cast<f32x4*>(q) = f32x4{acc[i][k][v], acc[i][k][v + 1], acc[i][k][v + 2], acc[i][k][v + 3]};
      }
    // the block is this wave's own: its LDS operations complete in order
#pragma unroll
    for (int r = 0; r < 32; r += kRows) {
      const int64_t m = m0 + r + l / kLanes;
      if (m < g.M && n0 < g.N)
        put16(C + m * g.N + n0, block + (r + l / kLanes) * kRow + (l % kLanes) * 16, static_cast<int>(g.N - n0), g.accumulate);
    }
  }
}

// Few rows (M <= 32 FM): the weight's bytes are what counts.  A block has 32
// columns of C; its 8 waves take every 8th block of 128 columns of the operands,
// straight from memory into registers (the pack's order is the operand order), and
// add up through LDS.  One launch, no partial sums in memory.
constexpr int kFewWaves = 8;
template <int FM>
constexpr int kFewLds = kFewWaves * FM * 16 * 65 * 4;  // 64 lanes and one more, against bank conflicts

template <typename T, bool EXACT, int FM>
__global__ __launch_bounds__(64 * kFewWaves) void k_fp8_few(GemmArgs g) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  float* sums = reinterpret_cast<float*>(smem);
  const int w = wave_id(), l = threadIdx.x & 63;
  const int64_t tn = blockIdx.x, KB = g.A.KB;
  struct Operands {
    u32x4 b[4], a[FM][4];
    int eb, ea[FM];
  };
  const auto load = [&](Operands& o, int64_t kb) {
    const uint8_t* pb = g.B.code + (tn * KB + kb) * 4096 + l * 16;
#pragma unroll
    for (int p = 0; p < 4; ++p) o.b[p] = *reinterpret_cast<const u32x4*>(pb + p * 1024);
    o.eb = g.B.exp[kb * g.B.exp_stride + tn * 32 + (l & 31)];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t rt = min(int64_t(i), g.A.RT - 1);
      const uint8_t* pa = g.A.code + (rt * KB + kb) * 4096 + l * 16;
#pragma unroll
      for (int p = 0; p < 4; ++p) o.a[i][p] = *reinterpret_cast<const u32x4*>(pa + p * 1024);
      o.ea[i] = g.A.exp[kb * g.A.exp_stride + rt * 32 + (l & 31)];
    }
  };
  const auto pair = [](u32x4 x, u32x4 y) {
    return i32x8{int(x[0]), int(x[1]), int(x[2]), int(x[3]), int(y[0]), int(y[1]), int(y[2]), int(y[3])};
  };
  f32x16 acc[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[i][e] = 0.f;
  Operands cur, nxt;
  if (w < KB) load(cur, w);
  for (int64_t kb = w; kb < KB; kb += kFewWaves) {
    if (kb + kFewWaves < KB) load(nxt, kb + kFewWaves);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < FM; ++i)
        acc[i] = mac64<EXACT>(pair(cur.b[2 * s], cur.b[2 * s + 1]), pair(cur.a[i][2 * s], cur.a[i][2 * s + 1]), cur.eb,
                              cur.ea[i], acc[i]);
    cur = nxt;
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) sums[((w * FM + i) * 16 + v) * 65 + l] = acc[i][v];
  __syncthreads();
  T* C = static_cast<T*>(g.C);
  const int n = threadIdx.x & 31, v = 4 * (n >> 3) + (n & 3), hi = (n >> 2) & 1;  // column n: register v, half hi
  for (int m = threadIdx.x >> 5; m < FM * 32; m += 2 * kFewWaves) {
    if (m >= g.M || tn * 32 + n >= g.N) continue;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kFewWaves; ++k) s += sums[((k * FM + (m >> 5)) * 16 + v) * 65 + hi * 32 + (m & 31)];
    T* c = C + m * g.N + tn * 32 + n;
    *c = from_f32<T>(g.accumulate ? to_f32<T>(*c) + s : s);
  }
}

// C (+)= sum of the splits' partial sums, in order; no splits: zeros.  A thread
// has 4 neighbouring elements of the whole.
template <typename T>
__global__ __launch_bounds__(256) void k_fp8_join(const float* part, int splits, T* C, int64_t n, int accumulate) {
  for (int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4; i < n; i += int64_t(gridDim.x) * 1024) {
    const int left = static_cast<int>(min(n - i, int64_t(4)));
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < splits; ++k)
      s += __builtin_bit_cast(f32x4, left == 4 ? ld16B(part + k * n + i) : ld_tail4(part + k * n + i, left));
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) C[i + e] = from_f32<T>(accumulate ? to_f32<T>(C[i + e]) + s[e] : s[e]);
  }
}

template <typename T>
void join_t(const float* part, int splits, T* C, int64_t n, int accumulate, hipStream_t s) {
  hipLaunchKernelGGL(k_fp8_join<T>, dim3(uint32_t(std::min<int64_t>((n + 1023) / 1024, 2048))), dim3(256), 0, s, part,
                     splits, C, n, accumulate);
}

// How a product is cut (times: one MI355X, bf16 C unless stated, the same operands
// again and again, as far as they fit in the last-level cache):
//  - few rows, M <= 64, and M <= 128 while K is below 8192: k_fp8_few (128 x 2048 x 2048: 6.4 us, 64 x 64 tiles
//    6.7, 128 x 128 tiles 10; 20 x 4096 x 16384 fp32: 15.6 us, split tiles 22; but 100 x 4000 x 16000: 32 us, split
//    tiles 20, as a block there goes through all of K);
//  - 256 x 256 tiles where they fill the 256 CUs (4000 x 4096 x 4096: 52 us, 128 x 128 tiles 62);
//  - 128 x 128 tiles from 160 of them (2000 x 2048 x 2048, 256 tiles: 12.4 us, 64 x 64 tiles 16): with two
//    workgroups a CU and 2 stages each, or with one and 4 (2048 x 2048 x 8192: 35 us, with 2 stages 43);
//  - fewer: 64 x 64 tiles (1000 x 2048 x 2048: 9.5 us, 128 x 128 tiles 11.0), or, for K of 8192 and more,
//    128 x 128 tiles with K split into parts of 2048 at least, one or two workgroups a CU (1024 x 1024 x 8192 fp32:
//    28 us, 64 x 64 tiles 34).  Partial sums in memory and a second launch cost 5 to 10 us, which a shorter K does
//    not pay for (1000 x 1024 x 4096: 16.5 us, 64 x 64 tiles 10.6).
enum CutKind { kFew, kTile64, kTile128, kTile256 };
struct Cut {
  CutKind kind;
  bool deep;  // 128 x 128 tiles: at most one workgroup a CU
  int splits;
  int64_t kb_per;
};
Cut cut(int64_t M, int64_t N, int64_t K) {
  constexpr int64_t kCus = 256;
  const int64_t KB = (K + 127) / 128;
  const auto tiles = [&](int64_t t) { return ((M + t - 1) / t) * ((N + t - 1) / t); };
  const int64_t t128 = tiles(128), parts = std::min((2 * t128 <= kCus ? 1 : 2) * kCus / t128, KB / 16);
  Cut c{kFew, false, 1, KB};
  if (M <= 64 || (M <= 128 && KB < 64)) return c;
  if (tiles(256) >= kCus) {
    c.kind = kTile256;
  } else if (t128 >= 160) {
    c.kind = kTile128;
    c.deep = t128 <= kCus;
  } else if (KB >= 64 && parts >= 2) {
    c.kind = kTile128;
    c.kb_per = (KB + parts - 1) / parts;
    c.splits = int((KB + c.kb_per - 1) / c.kb_per);
    c.deep = t128 * c.splits <= kCus;
  } else {
    c.kind = kTile64;
  }
  return c;
}

template <typename T, bool EXACT, int WM, int WN, int FM, int FN, int NS>
void gemm_k(const GemmArgs& g, hipStream_t s) {
  using TL = Tile<WM, WN, FM, FN, NS>;
  constexpr auto K = k_fp8_gemm<T, EXACT, WM, WN, FM, FN, NS>;
  const int64_t tiles = (g.A.RT + TL::kBM - 1) / TL::kBM * ((g.B.RT + TL::kBN - 1) / TL::kBN);
  hipLaunchKernelGGL(K, dim3(uint32_t(tiles * g.splits)), dim3(TL::kThreads), (LdsLimit<K, TL::kLds>::bytes()), s, g);
}

template <typename T, bool EXACT, int FM>
void few_k(const GemmArgs& g, hipStream_t s) {
  constexpr auto K = k_fp8_few<T, EXACT, FM>;
  hipLaunchKernelGGL(K, dim3(uint32_t(g.B.RT)), dim3(64 * kFewWaves), (LdsLimit<K, kFewLds<FM>>::bytes()), s, g);
}

template <typename T>
void gemm_t(GemmArgs g, const Cut& c, float* ws, hipStream_t s) {
  constexpr bool kExact = sizeof(T) == 4;
  if (c.kind == kFew) {
    if (g.A.RT == 1)
      few_k<T, kExact, 1>(g, s);
    else if (g.A.RT == 2)
      few_k<T, kExact, 2>(g, s);
    else
      few_k<T, kExact, 4>(g, s);
  } else if (c.splits > 1) {
    T* C = static_cast<T*>(g.C);
    const int accumulate = g.accumulate;
    g.C = ws;
    g.accumulate = 0;
    if (c.deep)
      gemm_k<float, kExact, 2, 2, 2, 2, 4>(g, s);
    else
      gemm_k<float, kExact, 2, 2, 2, 2, 2>(g, s);
    join_t(ws, c.splits, C, g.M * g.N, accumulate, s);
  } else if (c.kind == kTile256) {
    gemm_k<T, kExact, 2, 4, 4, 2, 2>(g, s);
  } else if (c.kind == kTile64) {
    gemm_k<T, kExact, 2, 2, 1, 1, 4>(g, s);
  } else if (c.deep) {
    gemm_k<T, kExact, 2, 2, 2, 2, 4>(g, s);
  } else {
    gemm_k<T, kExact, 2, 2, 2, 2, 2>(g, s);
  }
}

template <typename T, RowMode MODE, bool ROWS, bool COLS>
void pack_m(const T* X, uint8_t* pk, uint8_t* pkT, int square, int64_t R, int64_t C, hipStream_t s) {
  constexpr auto K = k_fp8_pack<T, MODE, ROWS, COLS>;
  constexpr int kTile = COLS ? int(128 * 130 * sizeof(T)) : 16;
  hipLaunchKernelGGL(K, dim3(uint32_t((C + 127) / 128 * ((R + 127) / 128))), dim3(256), (LdsLimit<K, kTile>::bytes()), s,
                     X, View(pk, R, C), View(pkT, C, R), square, R, C);
}
template <typename T, bool ROWS, bool COLS>
void pack_k(const T* X, uint8_t* pk, uint8_t* pkT, int square, int64_t R, int64_t C, hipStream_t s) {
  by_row_mode<T, true>(C, {X}, [&](auto m) { pack_m<T, decltype(m)::value, ROWS, COLS>(X, pk, pkT, square, R, C, s); });
}
template <typename T>
void pack_t(const T* X, uint8_t* pk, uint8_t* pkT, int square, int64_t R, int64_t C, hipStream_t s) {
  if (pk && pkT)
    pack_k<T, true, true>(X, pk, pkT, square, R, C, s);
  else if (pk && !square)
    by_row_mode<T, true>(C, {X}, [&](auto m) {
      const View v(pk, R, C);
      hipLaunchKernelGGL((k_fp8_pack_rows<T, decltype(m)::value>), dim3(uint32_t((v.KB + 3) / 4 * v.RT)), dim3(256), 0,
                         s, X, v, R, C);
    });
  else if (pk)
    pack_k<T, true, false>(X, pk, pkT, square, R, C, s);
  else
    pack_k<T, false, true>(X, pk, pkT, square, R, C, s);
}

}  // namespace

size_t fp8_bytes(int64_t rows, int64_t cols) {
  const View v(rows, cols);
  return size_t(v.RT) * v.KB * 4096 + size_t(v.KB) * v.exp_stride + 256;
}

void launch_fp8_pack(const void* X, uint8_t* pk, uint8_t* pkT, int square, int64_t R, int64_t C, int bf16,
                     hipStream_t s) {
  if (bf16)
    pack_t(static_cast<const bf16_t*>(X), pk, pkT, square, R, C, s);
  else
    pack_t(static_cast<const float*>(X), pk, pkT, square, R, C, s);
}

void launch_fp8_unpack(const uint8_t* pk, void* X, int64_t rows, int64_t cols, int bf16, hipStream_t s) {
  const View v(pk, rows, cols);
  const dim3 grid(uint32_t((v.KB + 3) / 4 * v.RT));
  if (bf16)
    hipLaunchKernelGGL(k_fp8_unpack<bf16_t>, grid, dim3(256), 0, s, v, static_cast<bf16_t*>(X), rows, cols);
  else
    hipLaunchKernelGGL(k_fp8_unpack<float>, grid, dim3(256), 0, s, v, static_cast<float*>(X), rows, cols);
}

size_t fp8_gemm_ws_bytes(int64_t M, int64_t N, int64_t K) {
  const Cut c = cut(M, N, K);
  return c.splits > 1 ? size_t(c.splits) * M * N * sizeof(float) : 0;
}

void launch_fp8_gemm(const uint8_t* A, const uint8_t* B, void* C, int accumulate, int64_t M, int64_t N, int64_t K,
                     int bf16, float* ws, hipStream_t s) {
  if (K == 0) {
    if (bf16)
      join_t(ws, 0, static_cast<bf16_t*>(C), M * N, 0, s);
    else
      join_t(ws, 0, static_cast<float*>(C), M * N, accumulate, s);
    return;
  }
  const Cut c = cut(M, N, K);
  const GemmArgs g{View(A, M, K), View(B, N, K), C, M, N, accumulate, c.splits, c.kb_per};
  if (bf16)
    gemm_t<bf16_t>(g, c, ws, s);
  else
    gemm_t<float>(g, c, ws, s);
}

}  // namespace mapl
