// Rounding to 8 bits (e4m3 with a power-of-two scale per block of 128) and the
// layout of the packs that hold the result, for every kernel that writes one.
//
// Pack of an operand [rows][cols], KB = ceil(cols / 128), RT = ceil(rows / 32):
//  - codes, RT x KB units of 4 KB, unit (rt, kb) at (rt * KB + kb) * 4096: the
//    32 rows x 128 columns that two v_mfma_scale_f32_32x32x64_f8f6f4 consume.
//    Step s (64 columns) and half h are pieces of 1 KB, 64 lanes x 16 bytes:
//    lane l holds row l & 31, columns 64 s + 32 (l >> 5) + 16 h + 0..15.  Every
//    operand load of a wave is one contiguous kilobyte, from memory or LDS.
//  - exponents, one byte each, [KB][rows rounded up to 256], then 256 bytes of
//    slack, so that 256 bytes from the first row of any tile can be read.
// Codes and exponents of padding rows only reach output rows that are not stored: codes
// up to the next multiple of 32 rows are zero, exponents behind it whatever was there.
// Padding columns are zero in every pack.
#pragma once

#include "common.h"

namespace mapl {

struct View {  // device view of a pack
  uint8_t* code = nullptr;
  uint8_t* exp = nullptr;
  int64_t KB = 0, RT = 0, exp_stride = 0;
  View() = default;
  View(int64_t rows, int64_t cols) : KB((cols + 127) / 128), RT((rows + 31) / 32), exp_stride((rows + 255) / 256 * 256) {}
  View(const uint8_t* pk, int64_t rows, int64_t cols) : View(rows, cols) {
    if (pk == nullptr) return;
    code = const_cast<uint8_t*>(pk);
    exp = code + RT * KB * 4096;
  }
};

// byte offset, in a unit, of row r (0..31) and columns 16 j .. 16 j + 15
__device__ __forceinline__ int unit_off(int r, int j) {
  return ((j >> 2) * 2 + (j & 1)) * 1024 + (((j >> 1) & 1) * 32 + r) * 16;
}

// Largest finite magnitude of a block -> biased exponent of the smallest power
// of two 2^s >= 2^-126 with amax <= 448 * 2^s.  448 = 1.75 * 2^8, so s is the
// exponent of amax less 8, one more if its significand is above 1.75.
__device__ __forceinline__ int block_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e > 1 ? e : 1;
}
__device__ __forceinline__ float pow2_neg(int biased) { return __uint_as_float(static_cast<uint32_t>(254 - biased) << 23); }

__device__ __forceinline__ float finite_abs(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? __uint_as_float(b) : 0.f;
}

// Largest finite magnitude of n values; `bad`: some are not finite.  As integers
// the magnitudes compare as they do as floats, with those beyond infinity on top, so
// the values are looked at one by one only where there is one.
template <int N>
__device__ __forceinline__ float abs_max(const float* v, bool& bad) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  bad = m >= 0x7f800000u;
  float f = __uint_as_float(m);
  if (bad) {
    f = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) f = fmaxf(f, finite_abs(v[i]));
  }
  return f;
}

// 4 values times 2^-s to e4m3 codes; the scaled values are at most 448 in size
__device__ __forceinline__ uint32_t codes4(const float* v, float inv) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, r, true);
  return static_cast<uint32_t>(r);
}
// 16 of them; `bad` (abs_max): those that are not finite become NaN
__device__ __forceinline__ u32x4 codes16(const float* v, float inv, bool bad) {
  u32x4 c = {codes4(v, inv), codes4(v + 4, inv), codes4(v + 8, inv), codes4(v + 12, inv)};
  if (bad) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((__float_as_uint(v[i]) & 0x7f800000u) == 0x7f800000u) c[i >> 2] |= 0x7fu << (8 * (i & 3));
  }
  return c;
}

// 8 values times 2^-s to e4m3 codes; `bad` (abs_max): those that are not finite become NaN
__device__ __forceinline__ u32x2 codes8(const float* v, float inv, bool bad) {
  u32x2 c = {codes4(v, inv), codes4(v + 4, inv)};
  if (bad) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((__float_as_uint(v[i]) & 0x7f800000u) == 0x7f800000u) c[i >> 2] |= 0x7fu << (8 * (i & 3));
  }
  return c;
}

}  // namespace mapl
