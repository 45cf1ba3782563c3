// Host-side exercise of include/mapl_stage.h for a build of the library's host
// code with AddressSanitizer and UndefinedBehaviorSanitizer: extreme sizes (the
// size arithmetic must not overflow), invalid arguments (the documented status
// before memory is touched) and valid shapes (which stop at the device set-up when
// there is no device).  No pointer is dereferenced on the host.
#include <cstdint>
#include <cstdio>
#include <limits>

#include "mapl_stage.h"

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
  const int64_t big = std::numeric_limits<int64_t>::max(), small = std::numeric_limits<int64_t>::min();
  const uint64_t all = ~uint64_t(0);
  const size_t huge = ~size_t(0);

  const int64_t xs[] = {0, 1, 7, 128, 129, 8192, 1 << 27, (1 << 27) + 1, int64_t(1) << 31, big, small, -1};
  for (int64_t a : xs)
    for (int64_t b : xs)
      for (int64_t c : xs) {
        (void)stage_norm_bwd_workspace_bytes(a, b, c);
        (void)fp8_gemm_workspace_bytes(a, b, c);
        (void)fp8_pack_bytes(a, b);
        for (mapl_dtype dt : {MAPL_F32, MAPL_BF16}) {
          (void)stage_dropout(F, F, 0.5, all, all, a, b, dt, nullptr);
          (void)stage_norm(F, F, F, c ? F : nullptr, F, F, F, 1.f, 1e-5f, 0.5, all, all, a, b, c, dt, nullptr);
          (void)stage_norm_bwd(F, F, F, F, F, c ? F : nullptr, F, F, F, Ff, Ff, Ff, 1, 1.f, 1e-5f, 0.5, all, all, a, b,
                               c, dt, F, huge, nullptr);
          (void)fp8_pack(F, F, huge, F, huge, 1, a, b, dt, nullptr);
          (void)fp8_unpack(F, huge, F, a, b, dt, nullptr);
          (void)fp8_gemm(F, huge, F, huge, F, 0, a, b, c, dt, F, huge, nullptr);
        }
      }

  expect(stage_dropout(F, F, 0.5, 1, 0, big, big, MAPL_BF16, nullptr), MAPL_ERR_SHAPE, MAPL_ERR_SHAPE, "dropout huge");
  expect(stage_norm(F, F, F, F, F, F, F, 1.f, 0.f, 0.5, 1, 0, 4, 64, 1, MAPL_BF16, nullptr), MAPL_ERR_ARG, MAPL_ERR_ARG,
         "norm eps = 0");
  expect(stage_norm_bwd(F, F, F, F, F, F, F, F, F, Ff, Ff, Ff, 0, 1.f, 1e-5f, 0.5, 1, 0, 4, 64, 1, MAPL_BF16, F, 0,
                        nullptr),
         MAPL_ERR_WORKSPACE, MAPL_ERR_WORKSPACE, "norm_bwd without workspace");
  expect(fp8_pack(F, F, 1, nullptr, 0, 0, 4, 4, MAPL_F32, nullptr), MAPL_ERR_WORKSPACE, MAPL_ERR_WORKSPACE, "small pack");
  expect(fp8_gemm(F, huge, F, huge, F, 1, 4, 4, 4, MAPL_BF16, nullptr, 0, nullptr), MAPL_ERR_ARG, MAPL_ERR_ARG,
         "bf16 accumulate");
  // valid: the device set-up's error, or a launch
  expect(stage_dropout(F, F, 0.5, 1, 0, 4, 64, MAPL_BF16, nullptr), MAPL_ERR_HIP, MAPL_OK, "dropout valid");
  expect(fp8_pack(F, F, huge, nullptr, 0, 0, 4, 4, MAPL_F32, nullptr), MAPL_ERR_HIP, MAPL_OK, "pack valid");
  expect(fp8_gemm(F, huge, F, huge, F, 0, 4, 4, 4, MAPL_F32, nullptr, 0, nullptr), MAPL_ERR_HIP, MAPL_OK, "gemm valid");

  if (failures) std::fprintf(stderr, "%d failure(s)\n", failures);
  else std::printf("stage driver: all expectations held\n");
  return failures ? 1 : 0;
}
