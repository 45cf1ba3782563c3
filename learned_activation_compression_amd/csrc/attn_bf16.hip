// The bf16 kernels of causal attention over packed sequences.
#include "attn_kernels.h"

namespace mapl {

void launch_attn_bf16(const Attn& c, hipStream_t s) { attn_t<bf16_t, false>(c, s); }
void launch_attn_bwd_bf16(const Attn& c, hipStream_t s) { attn_t<bf16_t, true>(c, s); }

}  // namespace mapl
