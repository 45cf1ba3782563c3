// Host-side exercise of include/mapl_block.h for a build of the library's host
// code with AddressSanitizer and UndefinedBehaviorSanitizer: extreme sizes (the
// size arithmetic must not overflow), invalid arguments (the documented status
// before memory is touched) and valid shapes (which stop at the device set-up when
// there is no device).  No pointer is dereferenced on the host.
#include <cstdint>
#include <cstdio>
#include <limits>

#include "mapl_block.h"

static int failures = 0;

static void expect(int got, int a, int b, const char* what) {
  if (got != a && got != b) {
    std::fprintf(stderr, "FAIL %s: got %d want %d or %d\n", what, got, a, b);
    ++failures;
  }
}

int main() {
  void* F = reinterpret_cast<void*>(uintptr_t(0x100000));  // never dereferenced
  float* Ff = static_cast<float*>(F);
  int32_t* Fi = static_cast<int32_t*>(F);
  const int64_t big = std::numeric_limits<int64_t>::max(), small = std::numeric_limits<int64_t>::min();
  const size_t huge = ~size_t(0);

  const int64_t xs[] = {0, 1, 7, 128, 129, 1024, 1 << 22, 1 << 28, (1 << 28) + 1, int64_t(1) << 31, big, small, -1};
  for (int64_t a : xs)
    for (int64_t b : xs)
      for (int64_t c : xs) {
        (void)stage_attn_bwd_workspace_bytes(a, b, c, 64);
        (void)stage_attn_bwd_workspace_bytes(a, 8, b, c);
        (void)stage_distill_workspace_bytes(a, b);
        for (mapl_dtype dt : {MAPL_F32, MAPL_BF16}) {
          (void)stage_norm_pack(F, F, F, c ? F : nullptr, F, F, F, F, huge, 1.f, 1e-5f, 0.5, 1, 2, a, b, c, dt, nullptr);
          (void)stage_attn(F, F, F, Fi, F, Ff, 0.1f, c, a, b, 1, 64, c, c, c, c, dt, nullptr);
          (void)stage_attn(F, F, F, Fi, F, Ff, 0.1f, 3, a, b, c, 64, 1 << 20, 1 << 20, 1 << 20, 1 << 20, dt, nullptr);
          (void)stage_attn_bwd(F, F, F, F, F, Ff, Fi, F, F, F, 0.1f, 3, a, b, c, 64, 1 << 20, 1 << 20, 1 << 20, 1 << 20,
                               1 << 20, 1 << 20, 1 << 20, 1 << 20, dt, F, huge, nullptr);
          (void)stage_distill(F, Fi, Fi, Ff, Ff, Ff, 2.f, 1.f, 1.f, a, b, c, dt, F, huge, nullptr);
          (void)stage_distill_bwd(Ff, F, Ff, Fi, Fi, Ff, F, 2.f, 1.f, 1.f, a, b, c, dt, nullptr);
        }
      }

  expect(stage_norm_pack(F, F, F, F, F, F, F, F, 10, 1.f, 1e-5f, 0.5, 1, 0, 4, 64, 1, MAPL_BF16, nullptr),
         MAPL_ERR_WORKSPACE, MAPL_ERR_WORKSPACE, "norm_pack small pack");
  expect(stage_attn(F, F, F, Fi, F, Ff, 0.f, 1, 4, 4, 2, 64, 256, 128, 128, 256, MAPL_BF16, nullptr), MAPL_ERR_ARG,
         MAPL_ERR_ARG, "attn scale = 0");
  expect(stage_attn(F, F, F, Fi, F, Ff, 1.f, 1, big, 4, 2, 64, 256, 128, 128, 256, MAPL_BF16, nullptr), MAPL_ERR_SHAPE,
         MAPL_ERR_SHAPE, "attn huge");
  expect(stage_attn_bwd(F, F, F, F, F, Ff, Fi, F, F, F, 1.f, 1, 4, 4, 2, 64, 256, 256, 128, 128, 256, 256, 128, 128,
                        MAPL_BF16, F, 0, nullptr),
         MAPL_ERR_WORKSPACE, MAPL_ERR_WORKSPACE, "attn_bwd without workspace");
  expect(stage_distill(F, Fi, Fi, Ff, Ff, Ff, 0.f, 1.f, 1.f, 4, 100, 5, MAPL_F32, F, huge, nullptr), MAPL_ERR_ARG,
         MAPL_ERR_ARG, "distill temperature 0");
  // valid: the device set-up's error, or a launch
  expect(stage_norm_pack(F, F, F, F, F, F, F, F, huge, 1.f, 1e-5f, 0.5, 1, 0, 4, 64, 1, MAPL_BF16, nullptr), MAPL_ERR_HIP,
         MAPL_OK, "norm_pack valid");
  expect(stage_attn(F, F, F, Fi, F, Ff, 1.f, 1, 4, 4, 2, 64, 256, 128, 128, 256, MAPL_F32, nullptr), MAPL_ERR_HIP, MAPL_OK,
         "attn valid");
  expect(stage_attn_bwd(F, F, F, F, F, Ff, Fi, F, F, F, 1.f, 1, 4, 4, 2, 64, 256, 256, 128, 128, 256, 256, 128, 128,
                        MAPL_BF16, F, huge, nullptr),
         MAPL_ERR_HIP, MAPL_OK, "attn_bwd valid");
  expect(stage_distill(F, Fi, Fi, Ff, Ff, Ff, 2.f, 1.f, 1.f, 4, 100, 5, MAPL_F32, F, huge, nullptr), MAPL_ERR_HIP, MAPL_OK,
         "distill valid");
  expect(stage_distill_bwd(Ff, F, Ff, Fi, Fi, Ff, F, 2.f, 1.f, 1.f, 4, 100, 5, MAPL_BF16, nullptr), MAPL_ERR_HIP, MAPL_OK,
         "distill_bwd valid");

  if (failures) std::fprintf(stderr, "%d failure(s)\n", failures);
  else std::printf("block driver: all expectations held\n");
  return failures ? 1 : 0;
}
