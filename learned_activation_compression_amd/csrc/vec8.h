// Rows of any width and tensors of any offset, 8 consecutive elements at a time.
// The memory system takes 16 bytes at any 4-byte boundary; what rows of other
// widths need beyond that depends on the width and the addresses, so kernels come
// in the first four forms of RowMode and the launch picks one.
#pragma once

#include <initializer_list>
#include <type_traits>

#include "common.h"

namespace mapl {

typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));
typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));
typedef u32x3 u32x3_a4 __attribute__((aligned(4)));

__device__ __forceinline__ u32x4 ld16B(const void* p) { return *reinterpret_cast<const u32x4_a4*>(p); }
__device__ __forceinline__ void st16B(void* p, u32x4 v) { *reinterpret_cast<u32x4_a4*>(p) = v; }

__device__ __forceinline__ bool odd_bf16(const bf16_t* p) { return reinterpret_cast<uintptr_t>(p) & 2; }

__device__ __forceinline__ u32x4 ld8_any(const bf16_t* p) {
  if (!odd_bf16(p)) return ld16B(p);
  const u32x3 m = *reinterpret_cast<const u32x3_a4*>(p + 1);
  return u32x4{static_cast<uint32_t>(p[0]) | (m[0] << 16), (m[0] >> 16) | (m[1] << 16), (m[1] >> 16) | (m[2] << 16),
               (m[2] >> 16) | (static_cast<uint32_t>(p[7]) << 16)};
}
__device__ __forceinline__ void st8_any(bf16_t* p, u32x4 v) {
  if (!odd_bf16(p)) {
    st16B(p, v);
    return;
  }
  p[0] = static_cast<bf16_t>(v[0]);
  *reinterpret_cast<u32x3_a4*>(p + 1) =
      u32x3{(v[0] >> 16) | (v[1] << 16), (v[1] >> 16) | (v[2] << 16), (v[2] >> 16) | (v[3] << 16)};
  p[7] = static_cast<bf16_t>(v[3] >> 16);
}

// the first `left` (1..7; 0 or less: none) of 8, the others zero
__device__ __forceinline__ u32x4 ld_tail(const bf16_t* p, int left) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (left <= 0) return v;
  uint32_t last = 0;
  if (left & 1) last = p[left - 1];
  if (left & 4) {
    const u32x2 q = *reinterpret_cast<const u32x2_a2*>(p);
    v[0] = q[0];
    v[1] = q[1];
    if (left & 2) {
      v[2] = *reinterpret_cast<const u32_a2*>(p + 4);
      v[3] = last;
    } else {
      v[2] = last;
    }
  } else if (left & 2) {
    v[0] = *reinterpret_cast<const u32_a2*>(p);
    v[1] = last;
  } else {
    v[0] = last;
  }
  return v;
}
__device__ __forceinline__ void st_tail(bf16_t* p, u32x4 v, int left) {
  if (left <= 0) return;
  if (left & 4) {
    *reinterpret_cast<u32x2_a2*>(p) = u32x2{v[0], v[1]};
    p += 4;
    v[0] = v[2];
    v[1] = v[3];
  }
  if (left & 2) {
    *reinterpret_cast<u32_a2*>(p) = v[0];
    p += 2;
    v[0] = v[1];
  }
  if (left & 1) *p = static_cast<bf16_t>(v[0]);
}
// 4 elements of fp32 in the same way, left in 1..3
__device__ __forceinline__ u32x4 ld_tail4(const float* p, int left) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (left <= 0) return v;
  uint32_t last = 0;
  if (left & 1) last = __float_as_uint(p[left - 1]);
  if (left & 2) {
    const u32x2 q = *reinterpret_cast<const u32x2_a4*>(p);
    v = u32x4{q[0], q[1], last, 0u};
  } else {
    v[0] = last;
  }
  return v;
}
__device__ __forceinline__ void st_tail4(float* p, u32x4 v, int left) {
  if (left <= 0) return;
  if (left & 2) {
    *reinterpret_cast<u32x2_a4*>(p) = u32x2{v[0], v[1]};
    p += 2;
    v[0] = v[2];
  }
  if (left & 1) *p = __uint_as_float(v[0]);
}

// 8 elements as loaded, widened one by one
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16_t> {
  u32x4 a;
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = a[i >> 1];
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  __device__ __forceinline__ void ones() { a = u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}; }
};
template <>
struct Raw8<float> {
  u32x4 a, b;
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(i < 4 ? a[i & 3] : b[i & 3]); }
  __device__ __forceinline__ void ones() {
    const uint32_t o = 0x3f800000u;
    a = b = u32x4{o, o, o, o};
  }
};

// 1 to 8 elements, any alignment, with branches
__device__ __forceinline__ void load8(Raw8<bf16_t>& r, const bf16_t* p, int left) {
  r.a = left >= 8 ? ld8_any(p) : ld_tail(p, left);
}
__device__ __forceinline__ void load8(Raw8<float>& r, const float* p, int left) {
  r.a = left >= 4 ? ld16B(p) : ld_tail4(p, left);
  r.b = left >= 8 ? ld16B(p + 4) : ld_tail4(p + 4, left - 4);
}
__device__ __forceinline__ void store8(bf16_t* p, const float* v, int left) {
  const u32x4 w = {pack2bf(v[0], v[1]), pack2bf(v[2], v[3]), pack2bf(v[4], v[5]), pack2bf(v[6], v[7])};
  if (left >= 8)
    st8_any(p, w);
  else
    st_tail(p, w, left);
}
__device__ __forceinline__ void store8(float* p, const float* v, int left) {
  const u32x4 a = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  const u32x4 b = {__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
  if (left >= 4)
    st16B(p, a);
  else
    st_tail4(p, a, left);
  if (left >= 8)
    st16B(p + 4, b);
  else
    st_tail4(p + 4, b, left - 4);
}

// How a row of d elements is read:
//  kVec   d a multiple of 8, every tensor 4-byte aligned: vectors are whole or
//         absent;
//  kEven  d >= 8, every row 4-byte aligned: the row's last vector is read where
//         it ends with the row, and shifted;
//  kOdd   d >= 8, bf16 rows at 2-byte boundaries: 12 + 2 + 2 bytes, likewise;
//  kTiny  d < 8.
// The first three load without a branch, so that loads can stay in flight over
// the arithmetic of an earlier row; Fetch keeps what was loaded until value().
// Every address lies within the row.
//  kAny   d >= 8, one row that all others share (a weight beside odd rows), at any
//         address: 16 bytes in one access, which the compiler and the memory system
//         take at 2-byte boundaries too, at a price.  From a 4-byte boundary only
//         the last vector pays it, otherwise each, out of the caches.
enum RowMode { kVec, kEven, kOdd, kTiny, kAny };

template <typename T, RowMode MODE>
struct Fetch;

// dwords of 8 elements moved down by `s` elements (0..8), zeros behind them
__device__ __forceinline__ u32x4 shift_down(u32x4 v, int s) {
  if (s & 8) v = u32x4{0u, 0u, 0u, 0u};
  v = (s & 4) ? u32x4{v[2], v[3], 0u, 0u} : v;
  v = (s & 2) ? u32x4{v[1], v[2], v[3], 0u} : v;
  return (s & 1) ? u32x4{(v[0] >> 16) | (v[1] << 16), (v[1] >> 16) | (v[2] << 16), (v[2] >> 16) | (v[3] << 16), v[3] >> 16}
                 : v;
}

template <>
struct Fetch<bf16_t, kVec> {
  u32x4 a;
  __device__ __forceinline__ void issue(const bf16_t* row, int64_t c, int64_t d) { a = ld16B(row + (c < d ? c : 0)); }
  __device__ __forceinline__ Raw8<bf16_t> value(int64_t c, int64_t d, bool in) const {
    return {in && c < d ? a : u32x4{0u, 0u, 0u, 0u}};
  }
};
template <>
struct Fetch<bf16_t, kEven> {
  u32x4 a;
  __device__ __forceinline__ void issue(const bf16_t* row, int64_t c, int64_t d) { a = ld16B(row + (c + 8 <= d ? c : d - 8)); }
  __device__ __forceinline__ Raw8<bf16_t> value(int64_t c, int64_t d, bool in) const {
    return {shift_down(a, in ? static_cast<int>(min(max(c + 8 - d, int64_t(0)), int64_t(8))) : 8)};
  }
};
template <>
struct Fetch<bf16_t, kOdd> {
  u32x3 m;
  uint32_t x, y, odd;
  __device__ __forceinline__ void issue(const bf16_t* row, int64_t c, int64_t d) {
    const bf16_t* p = row + (c + 8 <= d ? c : d - 8);
    odd = odd_bf16(p);
    m = *reinterpret_cast<const u32x3_a4*>(p + odd);  // elements 1..6 of an odd vector, 0..5 of an even one
    x = p[odd ? 0 : 6];
    y = p[7];
  }
  __device__ __forceinline__ Raw8<bf16_t> value(int64_t c, int64_t d, bool in) const {
    const u32x4 e = {m[0], m[1], m[2], x | (y << 16)};
    const u32x4 o = {x | (m[0] << 16), (m[0] >> 16) | (m[1] << 16), (m[1] >> 16) | (m[2] << 16), (m[2] >> 16) | (y << 16)};
    return {shift_down(odd ? o : e, in ? static_cast<int>(min(max(c + 8 - d, int64_t(0)), int64_t(8))) : 8)};
  }
};
template <>
struct Fetch<bf16_t, kAny> {
  u32x4 a;
  __device__ __forceinline__ void issue(const bf16_t* row, int64_t c, int64_t d) {
    a = *reinterpret_cast<const u32x4_a2*>(row + (c + 8 <= d ? c : d - 8));
  }
  __device__ __forceinline__ Raw8<bf16_t> value(int64_t c, int64_t d, bool in) const {
    return {shift_down(a, in ? static_cast<int>(min(max(c + 8 - d, int64_t(0)), int64_t(8))) : 8)};
  }
};
template <>
struct Fetch<float, kVec> {
  u32x4 a, b;
  __device__ __forceinline__ void issue(const float* row, int64_t c, int64_t d) {
    const float* p = row + (c < d ? c : 0);
    a = ld16B(p);
    b = ld16B(p + 4);
  }
  __device__ __forceinline__ Raw8<float> value(int64_t c, int64_t d, bool in) const {
    const bool k = in && c < d;
    return {k ? a : u32x4{0u, 0u, 0u, 0u}, k ? b : u32x4{0u, 0u, 0u, 0u}};
  }
};
template <>
struct Fetch<float, kEven> {
  u32x4 a, b;
  __device__ __forceinline__ void issue(const float* row, int64_t c, int64_t d) {
    const float* p = row + (c + 8 <= d ? c : d - 8);
    a = ld16B(p);
    b = ld16B(p + 4);
  }
  __device__ __forceinline__ Raw8<float> value(int64_t c, int64_t d, bool in) const {
    const int s = in ? static_cast<int>(min(max(c + 8 - d, int64_t(0)), int64_t(8))) : 8;
    u32x4 u = a, v = b;
    const u32x4 z = {0u, 0u, 0u, 0u};
    u = (s & 8) ? z : (s & 4) ? v : u;
    v = (s & 12) ? z : v;
    if (s & 2) {
      u = u32x4{u[2], u[3], v[0], v[1]};
      v = u32x4{v[2], v[3], 0u, 0u};
    }
    if (s & 1) {
      u = u32x4{u[1], u[2], u[3], v[0]};
      v = u32x4{v[1], v[2], v[3], 0u};
    }
    return {u, v};
  }
};
template <typename T>
struct Fetch<T, kTiny> {  // d < 8: only the vector at column 0 holds anything
  Raw8<T> r;
  __device__ __forceinline__ void issue(const T* row, int64_t c, int64_t d) {
    load8(r, row, c == 0 ? static_cast<int>(d) : 0);
  }
  __device__ __forceinline__ Raw8<T> value(int64_t, int64_t, bool in) const {
    Raw8<T> v = r;
    if (!in) load8(v, static_cast<const T*>(nullptr), 0);
    return v;
  }
};

// the columns c .. c + 7 of a row, as many as there are
template <RowMode MODE, typename T>
__device__ __forceinline__ void put_row(T* row, int64_t c, int64_t d, bool in, const float* v) {
  if (!in || c >= d) return;
  if constexpr (MODE == kVec) {
    if constexpr (sizeof(T) == 2)
      st16B(row + c, u32x4{pack2bf(v[0], v[1]), pack2bf(v[2], v[3]), pack2bf(v[4], v[5]), pack2bf(v[6], v[7])});
    else
      store8(row + c, v, 8);
  } else {
    store8(row + c, v, static_cast<int>(min(d - c, int64_t(8))));
  }
}

// Host side: the mode of rows of d elements at addresses whose bits are or-ed in `at`
inline RowMode row_mode(int64_t d, int elem_bytes, uintptr_t at) {
  if (d < 8) return kTiny;
  const bool aligned = at % 4 == 0;
  if (aligned && d % 8 == 0) return kVec;
  return elem_bytes == 4 || (aligned && d % 2 == 0) ? kEven : kOdd;
}

// f(mode of the rows as a constant); TINY: widths below 8 occur
template <typename T, bool TINY, typename F>
void by_row_mode(int64_t d, std::initializer_list<const void*> ps, F f) {
  uintptr_t at = 0;
  for (const void* p : ps) at |= reinterpret_cast<uintptr_t>(p);
  const RowMode m = row_mode(d, sizeof(T), at);
  if (m == kVec) return f(std::integral_constant<RowMode, kVec>{});
  if (m == kEven) return f(std::integral_constant<RowMode, kEven>{});
  if constexpr (TINY) {
    if (m == kTiny) return f(std::integral_constant<RowMode, kTiny>{});
  }
  if constexpr (sizeof(T) == 2) f(std::integral_constant<RowMode, kOdd>{});
}

}  // namespace mapl
