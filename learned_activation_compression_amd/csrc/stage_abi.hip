// C ABI of the pipeline-stage operators: host-side validation, then launches.
// The operations are documented in include/mapl_stage.h.
#include "../../include/mapl_stage.h"

#include "abi_check.h"
#include "internal.h"

using namespace mapl;

namespace {

int check_fp8_pack(const void* pk, size_t bytes, int64_t rows, int64_t cols) {
  if (misaligned(pk, 16)) return MAPL_ERR_ARG;
  return bytes < fp8_bytes(rows, cols) ? MAPL_ERR_WORKSPACE : MAPL_OK;
}

}  // namespace

extern "C" {

int stage_dropout(const void* X, void* Y, double p, uint64_t seed, uint64_t offset, int64_t N, int64_t d,
                  mapl_dtype dt, hipStream_t stream) {
  if (!dtype_ok(dt)) return MAPL_ERR_DTYPE;
  if (N < 0 || N > INT32_MAX || d < 1 || d > INT32_MAX - 7 || N > kMaxElems / d) return MAPL_ERR_SHAPE;
  if (!(p >= 0.0 && p <= 1.0)) return MAPL_ERR_ARG;
  if (N == 0) return MAPL_OK;
  if (!X || !Y) return MAPL_ERR_NULL;
  if (elem_misaligned(dt, {X, Y})) return MAPL_ERR_ARG;
  LaunchScope ls;
  if (!ls.ready()) return MAPL_ERR_HIP;
  launch_dropout(X, Y, p, seed, offset, N, d, dt == MAPL_BF16, stream);
  return ls.done();
}

int stage_norm(const void* X, const void* Y, const void* w_post, const void* gate, const void* w_pre, void* X_out,
               void* H, float res_scale, float eps, double p, uint64_t seed, uint64_t offset, int64_t N, int64_t d,
               int64_t gate_rows, mapl_dtype dt, hipStream_t stream) {
  if (!dtype_ok(dt)) return MAPL_ERR_DTYPE;
  int st = check_norm_shape(N, d, gate_rows);
  if (st) return st;
  if ((st = check_norm_scalars(res_scale, eps, p))) return st;
  if ((gate == nullptr) != (gate_rows == 0)) return MAPL_ERR_ARG;
  if (N == 0) return MAPL_OK;  // the tensors without rows may be NULL
  if (Y == nullptr && (w_post || gate || p != 0.0)) return MAPL_ERR_ARG;
  if (!X || (!X_out && !H) || (H && !w_pre)) return MAPL_ERR_NULL;
  if (w_pre && !H) return MAPL_ERR_ARG;
  if (elem_misaligned(dt, {X, Y, w_post, gate, w_pre, X_out, H})) return MAPL_ERR_ARG;
  LaunchScope ls;
  if (!ls.ready()) return MAPL_ERR_HIP;
  launch_stage_norm({X, Y, w_post, gate, w_pre, X_out, H, res_scale, eps, p, seed, offset, N, d, gate_rows},
                    dt == MAPL_BF16, stream);
  return ls.done();
}

size_t stage_norm_bwd_workspace_bytes(int64_t N, int64_t d, int64_t gate_rows) {
  if (check_norm_shape(N, d, gate_rows) || N == 0) return 0;
  return stage_norm_bwd_ws_bytes(N, d, gate_rows);
}

int stage_norm_bwd(const void* gX_out, const void* gH, const void* X_out, const void* Y, const void* w_post,
                   const void* gate, const void* w_pre, void* gX, void* gY, float* g_w_post, float* g_gate,
                   float* g_w_pre, int accumulate, float res_scale, float eps, double p, uint64_t seed,
                   uint64_t offset, int64_t N, int64_t d, int64_t gate_rows, mapl_dtype dt, void* ws,
                   size_t ws_bytes, hipStream_t stream) {
  if (!dtype_ok(dt)) return MAPL_ERR_DTYPE;
  int st = check_norm_shape(N, d, gate_rows);
  if (st) return st;
  if ((st = check_norm_scalars(res_scale, eps, p))) return st;
  if (accumulate != 0 && accumulate != 1) return MAPL_ERR_ARG;
  if ((gate == nullptr) != (gate_rows == 0)) return MAPL_ERR_ARG;
  if (elem_misaligned(MAPL_F32, {g_w_post, g_gate, g_w_pre})) return MAPL_ERR_ARG;
  if ((w_post && !g_w_post) || (gate && !g_gate)) return MAPL_ERR_NULL;
  if (N == 0) {  // the tensors without rows may be NULL; each given gradient is zero (unchanged when accumulating)
    if (accumulate || !(g_w_post || g_gate || g_w_pre)) return MAPL_OK;
    LaunchScope ls0;
    if (!ls0.ready()) return MAPL_ERR_HIP;
    if (g_w_post) launch_fill_f32(g_w_post, d, 0.f, stream);
    if (g_gate) launch_fill_f32(g_gate, gate_rows * d, 0.f, stream);
    if (g_w_pre) launch_fill_f32(g_w_pre, d, 0.f, stream);
    return ls0.done();
  }
  if (Y == nullptr && (w_post || gate || p != 0.0)) return MAPL_ERR_ARG;
  if (gH && (!w_pre || !g_w_pre)) return MAPL_ERR_NULL;
  if ((!gX_out && !gH) || (gH && !X_out) || !gX || (Y && !gY)) return MAPL_ERR_NULL;
  if (elem_misaligned(dt, {gX_out, gH, X_out, Y, w_post, gate, w_pre, gX, gY})) return MAPL_ERR_ARG;
  if (w_post || gate || gH) {
    if (!ws) return MAPL_ERR_NULL;
    if (misaligned(ws, 16)) return MAPL_ERR_ARG;
    if (ws_bytes < stage_norm_bwd_ws_bytes(N, d, gate_rows)) return MAPL_ERR_WORKSPACE;
  }
  LaunchScope ls;
  if (!ls.ready()) return MAPL_ERR_HIP;
  const StageNorm c{nullptr, Y,   w_post, gate,   w_pre, const_cast<void*>(X_out), nullptr, res_scale,
                    eps,     p,   seed,   offset, N,     d,                        gate_rows};
  launch_stage_norm_bwd(c, {gX_out, gH, gX, gY, g_w_post, g_gate, g_w_pre, accumulate, static_cast<float*>(ws)},
                        dt == MAPL_BF16, stream);
  return ls.done();
}

size_t fp8_pack_bytes(int64_t rows, int64_t cols) { return check_fp8_shape(rows, cols) ? 0 : fp8_bytes(rows, cols); }

int fp8_pack(const void* X, void* pk, size_t pk_bytes, void* pkT, size_t pkT_bytes, int square, int64_t R, int64_t C,
             mapl_dtype dt, hipStream_t stream) {
  if (!dtype_ok(dt)) return MAPL_ERR_DTYPE;
  int st = check_fp8_shape(R, C);
  if (st) return st;
  if (square != 0 && square != 1) return MAPL_ERR_ARG;
  if (R == 0 || C == 0) return MAPL_OK;  // no element and no block
  if (!X || (!pk && !pkT)) return MAPL_ERR_NULL;
  if (pk && (st = check_fp8_pack(pk, pk_bytes, R, C))) return st;
  if (pkT && (st = check_fp8_pack(pkT, pkT_bytes, C, R))) return st;
  if (elem_misaligned(dt, {X})) return MAPL_ERR_ARG;
  LaunchScope ls;
  if (!ls.ready()) return MAPL_ERR_HIP;
  launch_fp8_pack(X, static_cast<uint8_t*>(pk), static_cast<uint8_t*>(pkT), square, R, C, dt == MAPL_BF16, stream);
  return ls.done();
}

int fp8_unpack(const void* pk, size_t pk_bytes, void* X, int64_t rows, int64_t cols, mapl_dtype dt,
               hipStream_t stream) {
  if (!dtype_ok(dt)) return MAPL_ERR_DTYPE;
  int st = check_fp8_shape(rows, cols);
  if (st) return st;
  if (rows == 0 || cols == 0) return MAPL_OK;
  if (!pk || !X) return MAPL_ERR_NULL;
  if ((st = check_fp8_pack(pk, pk_bytes, rows, cols))) return st;
  if (elem_misaligned(dt, {X})) return MAPL_ERR_ARG;
  LaunchScope ls;
  if (!ls.ready()) return MAPL_ERR_HIP;
  launch_fp8_unpack(static_cast<const uint8_t*>(pk), X, rows, cols, dt == MAPL_BF16, stream);
  return ls.done();
}

size_t fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (check_fp8_shape(M, N) || check_fp8_shape(M, K) || check_fp8_shape(N, K)) return 0;
  if (M == 0 || N == 0 || K == 0) return 0;
  return fp8_gemm_ws_bytes(M, N, K);
}

int fp8_gemm(const void* pkA, size_t pkA_bytes, const void* pkB, size_t pkB_bytes, void* C, int accumulate, int64_t M,
             int64_t N, int64_t K, mapl_dtype dt, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!dtype_ok(dt)) return MAPL_ERR_DTYPE;
  int st;
  if ((st = check_fp8_shape(M, N)) || (st = check_fp8_shape(M, K)) || (st = check_fp8_shape(N, K))) return st;
  if ((accumulate != 0 && accumulate != 1) || (accumulate && dt != MAPL_F32)) return MAPL_ERR_ARG;
  if (M == 0 || N == 0) return MAPL_OK;
  if (!C || (K > 0 && (!pkA || !pkB))) return MAPL_ERR_NULL;
  if (elem_misaligned(dt, {C})) return MAPL_ERR_ARG;
  if (K > 0) {
    if ((st = check_fp8_pack(pkA, pkA_bytes, M, K)) || (st = check_fp8_pack(pkB, pkB_bytes, N, K))) return st;
    const size_t need = fp8_gemm_ws_bytes(M, N, K);
    if (need > 0 && !ws) return MAPL_ERR_NULL;
    if (need > 0 && misaligned(ws, 16)) return MAPL_ERR_ARG;
    if (ws_bytes < need) return MAPL_ERR_WORKSPACE;
  }
  LaunchScope ls;
  if (!ls.ready()) return MAPL_ERR_HIP;
  launch_fp8_gemm(static_cast<const uint8_t*>(pkA), static_cast<const uint8_t*>(pkB), C, accumulate, M, N, K,
                  dt == MAPL_BF16, static_cast<float*>(ws), stream);
  return ls.done();
}

}  // extern "C"
