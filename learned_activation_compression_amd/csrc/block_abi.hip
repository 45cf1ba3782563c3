// C ABI of the operators between a stage's boundary and its loss: host-side
// validation, then launches.  The operations are documented in include/mapl_block.h.
#include "../../include/mapl_block.h"

#include "abi_check.h"
#include "internal.h"

using namespace mapl;

namespace {

int check_attn_shape(int64_t N, int64_t Hq, int64_t Hkv, int64_t D) {
  if (N < 0 || Hkv < 1 || Hq < 1 || Hq > 65536 || Hkv > Hq || Hq % Hkv != 0 || D < 1 || D > 128) return MAPL_ERR_SHAPE;
  return N > (int64_t(1) << 28) || N > (int64_t(1) << 30) / Hq ? MAPL_ERR_SHAPE : MAPL_OK;
}

// rows of `heads` heads: leading dimensions
bool short_rows(int64_t heads, int64_t D, std::initializer_list<int64_t> lds) {
  for (int64_t ld : lds)
    if (ld < heads * D || ld > (int64_t(1) << 22)) return true;  // a tile's 128 rows at most: 2^31 bytes
  return false;
}

int check_distill(int64_t N, int64_t V, int64_t K, float temperature, float w_ce, float w_kd) {
  // a block a row at least: a grid has fewer than 2^32 threads
  if (N < 0 || N > (int64_t(1) << 23) || V < 1 || V > (int64_t(1) << 27) || K < 0 || K > 1024) return MAPL_ERR_SHAPE;
  if (N > kMaxElems / V) return MAPL_ERR_SHAPE;
  if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(1.f / temperature)) return MAPL_ERR_ARG;
  return std::isfinite(w_ce) && std::isfinite(w_kd) ? MAPL_OK : MAPL_ERR_ARG;
}

}  // namespace

extern "C" {

int stage_norm_pack(const void* X, const void* Y, const void* w_post, const void* gate, const void* w_pre, void* X_out,
                    void* H, void* pkH, size_t pkH_bytes, float res_scale, float eps, double p, uint64_t seed,
                    uint64_t offset, int64_t N, int64_t d, int64_t gate_rows, mapl_dtype dt, hipStream_t stream) {
  if (!dtype_ok(dt)) return MAPL_ERR_DTYPE;
  if (int st = check_norm_shape(N, d, gate_rows)) return st;
  if (int st = check_fp8_shape(N, d)) return st;
  if (int st = check_norm_scalars(res_scale, eps, p)) return st;
  if ((gate == nullptr) != (gate_rows == 0)) return MAPL_ERR_ARG;
  if (N == 0) return MAPL_OK;  // the tensors without rows may be NULL
  if (Y == nullptr && (w_post || gate || p != 0.0)) return MAPL_ERR_ARG;
  if (!X || !w_pre || !pkH) return MAPL_ERR_NULL;
  if (elem_misaligned(dt, {X, Y, w_post, gate, w_pre, X_out, H}) || misaligned(pkH, 16)) return MAPL_ERR_ARG;
  if (pkH_bytes < fp8_bytes(N, d)) return MAPL_ERR_WORKSPACE;
  LaunchScope ls;
  if (!ls.ready()) return MAPL_ERR_HIP;
  launch_stage_norm_pack({X, Y, w_post, gate, w_pre, X_out, H, res_scale, eps, p, seed, offset, N, d, gate_rows},
                         static_cast<uint8_t*>(pkH), dt == MAPL_BF16, stream);
  return ls.done();
}

int stage_attn(const void* Q, const void* K, const void* V, const int32_t* cu, void* O, float* lse, float scale,
               int64_t S, int64_t N, int64_t Hq, int64_t Hkv, int64_t D, int64_t ldq, int64_t ldk, int64_t ldv,
               int64_t ldo, mapl_dtype dt, hipStream_t stream) {
  if (!dtype_ok(dt)) return MAPL_ERR_DTYPE;
  if (int st = check_attn_shape(N, Hq, Hkv, D)) return st;
  if (S < 0 || S >= INT32_MAX || short_rows(Hq, D, {ldq, ldo}) || short_rows(Hkv, D, {ldk, ldv})) return MAPL_ERR_SHAPE;
  if (!(scale >= 0x1p-64f && scale <= 0x1p64f)) return MAPL_ERR_ARG;  // its reciprocal and products stay normal
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
  if (!(scale >= 0x1p-64f && scale <= 0x1p64f)) return MAPL_ERR_ARG;  // its reciprocal and products stay normal
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

size_t stage_distill_workspace_bytes(int64_t N, int64_t V) {
  return check_distill(N, V, 0, 1.f, 0.f, 0.f) || N == 0 ? 0 : distill_ws_bytes(N, V);
}

int stage_distill(const void* Z, const int32_t* labels, const int32_t* t_ids, const float* t_logits, float* loss,
                  float* stats, float temperature, float w_ce, float w_kd, int64_t N, int64_t V, int64_t K,
                  mapl_dtype dt, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!dtype_ok(dt)) return MAPL_ERR_DTYPE;
  if (int st = check_distill(N, V, K, temperature, w_ce, w_kd)) return st;
  if (N == 0) return MAPL_OK;
  if (!Z || !loss || !stats || (K > 0 && (!t_ids || !t_logits))) return MAPL_ERR_NULL;
  if (elem_misaligned(dt, {Z}) || elem_misaligned(MAPL_F32, {labels, t_ids, t_logits, loss, stats})) return MAPL_ERR_ARG;
  if (const size_t need = distill_ws_bytes(N, V)) {
    if (!ws) return MAPL_ERR_NULL;
    if (misaligned(ws, 16)) return MAPL_ERR_ARG;
    if (ws_bytes < need) return MAPL_ERR_WORKSPACE;
  }
  LaunchScope lsc;
  if (!lsc.ready()) return MAPL_ERR_HIP;
  launch_distill({Z, labels, t_ids, t_logits, nullptr, loss, stats, nullptr, temperature, w_ce, w_kd, N, V, K},
                 dt == MAPL_BF16, static_cast<float*>(ws), stream);
  return lsc.done();
}

int stage_distill_bwd(const float* gloss, const void* Z, const float* stats, const int32_t* labels,
                      const int32_t* t_ids, const float* t_logits, void* gZ, float temperature, float w_ce, float w_kd,
                      int64_t N, int64_t V, int64_t K, mapl_dtype dt, hipStream_t stream) {
  if (!dtype_ok(dt)) return MAPL_ERR_DTYPE;
  if (int st = check_distill(N, V, K, temperature, w_ce, w_kd)) return st;
  if (N == 0) return MAPL_OK;
  if (!gloss || !Z || !stats || !gZ || (K > 0 && (!t_ids || !t_logits))) return MAPL_ERR_NULL;
  if (elem_misaligned(dt, {Z, gZ}) || elem_misaligned(MAPL_F32, {gloss, stats, labels, t_ids, t_logits}))
    return MAPL_ERR_ARG;
  LaunchScope ls;
  if (!ls.ready()) return MAPL_ERR_HIP;
  launch_distill_bwd({Z, labels, t_ids, t_logits, gloss, nullptr, const_cast<float*>(stats), gZ, temperature, w_ce, w_kd,
                      N, V, K}, dt == MAPL_BF16, stream);
  return ls.done();
}

}  // extern "C"
