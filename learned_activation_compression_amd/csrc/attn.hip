// Causal attention over packed sequences: the fp32 kernels and the launches.  The bf16
// kernels are compiled apart (attn_bf16.hip), so that the two build side by side.
#include "attn_kernels.h"

namespace mapl {

size_t attn_bwd_ws_bytes(int64_t N, int64_t Hq, int64_t Hkv, int64_t D) {
  if (N == 0) return 0;
  const int64_t q = dq_splits(N, Hq), k = dkv_splits(N, Hkv);
  const int64_t part = std::max(q > 1 ? q * Hq : 0, k > 1 ? 2 * k * Hkv : 0) * N * D;
  return size_t(attn_rows_floats(N, Hq) + part) * sizeof(float);
}
void launch_attn_bf16(const Attn& c, hipStream_t s);
void launch_attn_bwd_bf16(const Attn& c, hipStream_t s);
void launch_attn(const Attn& c, int bf16, hipStream_t s) { (bf16 ? launch_attn_bf16 : attn_t<float, false>)(c, s); }
void launch_attn_bwd(const Attn& c, int bf16, hipStream_t s) { (bf16 ? launch_attn_bwd_bf16 : attn_t<float, true>)(c, s); }

}  // namespace mapl
