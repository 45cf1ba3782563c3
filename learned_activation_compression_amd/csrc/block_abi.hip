// C ABI of the operators between a stage's boundary and its loss: host-side
// validation, then launches.  The operations are documented in include/mapl_block.h.
#include "../../include/mapl_block.h"

#include <cmath>
#include <initializer_list>

#include "internal.h"

using namespace mapl;

namespace {

bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) & (to - 1); }

bool elem_misaligned(mapl_dtype dt, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (misaligned(p, dt == MAPL_BF16 ? 2 : 4)) return true;
  return false;
}

int check_attn_shape(int64_t N, int64_t Hq, int64_t Hkv, int64_t D) {
  if (N < 0 || Hkv < 1 || Hq < 1 || Hq > 65536 || Hkv > Hq || Hq % Hkv != 0 || D < 1 || D > 128) return MAPL_ERR_SHAPE;
  return N > (int64_t(1) << 30) / Hq ? MAPL_ERR_SHAPE : MAPL_OK;
}

// rows of `heads` heads: leading dimensions
bool short_rows(int64_t heads, int64_t D, std::initializer_list<int64_t> lds) {
  for (int64_t ld : lds)
    if (ld < heads * D || ld > INT32_MAX) return true;
  return false;
}

}  // namespace

extern "C" {

int stage_attn(const void* Q, const void* K, const void* V, const int32_t* cu, void* O, float* lse, float scale,
               int64_t S, int64_t N, int64_t Hq, int64_t Hkv, int64_t D, int64_t ldq, int64_t ldk, int64_t ldv,
               int64_t ldo, mapl_dtype dt, hipStream_t stream) {
  if (!dtype_ok(dt)) return MAPL_ERR_DTYPE;
  if (int st = check_attn_shape(N, Hq, Hkv, D)) return st;
  if (S < 0 || S >= INT32_MAX || short_rows(Hq, D, {ldq, ldo}) || short_rows(Hkv, D, {ldk, ldv})) return MAPL_ERR_SHAPE;
  if (!(scale > 0.f) || !std::isfinite(scale)) return MAPL_ERR_ARG;
  if (N == 0 || S == 0) return MAPL_OK;
  if (!Q || !K || !V || !cu || !O || !lse) return MAPL_ERR_NULL;
  if (elem_misaligned(dt, {Q, K, V, O}) || elem_misaligned(MAPL_F32, {cu, lse})) return MAPL_ERR_ARG;
  LaunchScope ls;
  if (!ls.ready()) return MAPL_ERR_HIP;
  Attn a{};
  a.Q = Q, a.K = K, a.V = V, a.out = O, a.cu = cu, a.lse = lse;
  a.ldq = ldq, a.ldk = ldk, a.ldv = ldv, a.ldo = ldo;
  a.scale = scale, a.S = S, a.N = N, a.Hq = Hq, a.Hkv = Hkv, a.D = D;
  launch_attn(a, dt == MAPL_BF16, stream);
  return ls.done();
}

size_t stage_attn_bwd_workspace_bytes(int64_t N, int64_t Hq, int64_t Hkv, int64_t D) {
  return check_attn_shape(N, Hq, Hkv, D) ? 0 : attn_bwd_ws_bytes(N, Hq, Hkv, D);
}

int stage_attn_bwd(const void* gO, const void* Q, const void* K, const void* V, const void* O, const float* lse,
                   const int32_t* cu, void* gQ, void* gK, void* gV, float scale, int64_t S, int64_t N, int64_t Hq,
                   int64_t Hkv, int64_t D, int64_t ldgo, int64_t ldq, int64_t ldk, int64_t ldv, int64_t ldo,
                   int64_t ldgq, int64_t ldgk, int64_t ldgv, mapl_dtype dt, void* ws, size_t ws_bytes,
                   hipStream_t stream) {
  if (!dtype_ok(dt)) return MAPL_ERR_DTYPE;
  if (int st = check_attn_shape(N, Hq, Hkv, D)) return st;
  if (S < 0 || S >= INT32_MAX || short_rows(Hq, D, {ldgo, ldq, ldo, ldgq}) || short_rows(Hkv, D, {ldk, ldv, ldgk, ldgv}))
    return MAPL_ERR_SHAPE;
  if (!(scale > 0.f) || !std::isfinite(scale)) return MAPL_ERR_ARG;
  if (N == 0 || S == 0) return MAPL_OK;
  if (!gO || !Q || !K || !V || !O || !lse || !cu || !gQ || !gK || !gV || !ws) return MAPL_ERR_NULL;
  if (elem_misaligned(dt, {gO, Q, K, V, O, gQ, gK, gV}) || elem_misaligned(MAPL_F32, {cu, lse}) || misaligned(ws, 16))
    return MAPL_ERR_ARG;
  if (ws_bytes < attn_bwd_ws_bytes(N, Hq, Hkv, D)) return MAPL_ERR_WORKSPACE;
  LaunchScope ls;
  if (!ls.ready()) return MAPL_ERR_HIP;
  Attn a{};
  a.Q = Q, a.K = K, a.V = V, a.O = O, a.gO = gO, a.gQ = gQ, a.gK = gK, a.gV = gV, a.cu = cu;
  a.lse = const_cast<float*>(lse), a.rows = static_cast<float*>(ws);
  a.ldq = ldq, a.ldk = ldk, a.ldv = ldv, a.ldo = ldo, a.ldgo = ldgo, a.ldgq = ldgq, a.ldgk = ldgk, a.ldgv = ldgv;
  a.scale = scale, a.S = S, a.N = N, a.Hq = Hq, a.Hkv = Hkv, a.D = D;
  launch_attn_bwd(a, dt == MAPL_BF16, stream);
  return ls.done();
}

}  // extern "C"
