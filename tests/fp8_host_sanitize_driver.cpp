// Host-only driver for the sanitizer build of the 8-bit path's validation and
// planning (hxq_fp8_api.cpp): workspace queries over sizes up to the 2^31
// limit, and calls that are refused before anything would be queued.  Built
// with host AddressSanitizer and UndefinedBehaviorSanitizer (no recovery).
// Prints "fp8 host sanitize: N checks ok" and exits 0 on success.

#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "hxq.h"

int main() {
  int checks = 0, fails = 0;
  auto expect = [&](bool ok, const char* what) {
    ++checks;
    if (!ok) {
      ++fails;
      printf("FAIL %s\n", what);
    }
  };
  const int64_t top = (int64_t)INT32_MAX - 65536;
  const int64_t dims[] = {0, 1, 2, 15, 16, 17, 63, 64, 100, 128, 255, 256, 1000, 2048, 8512, 11008, 22016, 65537,
                          (int64_t)1 << 20, (int64_t)1 << 24, ((int64_t)1 << 30) + 1, top, top + 1, -1, INT64_MAX, INT64_MIN};
  const int64_t experts[] = {1, 2, 64, 65535};
  for (int dt = -1; dt <= 3; ++dt)
    for (int64_t M : dims)
      for (int64_t N : dims)
        for (int64_t K : dims) {
          const bool bad = M < 0 || N < 0 || K < 0 || M > top || N > top || K > top || dt < 0 || dt > 2;
          const int64_t w = hxq_linear_fwd_fp8_workspace(dt, M, N, K);
          expect(bad ? w < 0 : w >= 0 || w == HXQ_ERR_SHAPE, "workspace");
          if (dt == HXQ_E4M3 && !bad) {
            for (int64_t E : experts) {
              const int64_t e = hxq_linear_fwd_fp8_experts_workspace(HXQ_BF16, M, N, E, K, 2048);
              expect(e >= 0 || e == HXQ_ERR_SHAPE, "experts workspace");
              expect(hxq_linear_fwd_fp8_experts_workspace(dt, 7, M, E, N, K) >= HXQ_ERR_SHAPE, "experts workspace");
            }
          }
          // a workspace that is too small, or sizes that are refused
          const uintptr_t F = 0x100000;
          if (w != 0) {
            const int st = hxq_linear_fwd_fp8((const void*)F, dt, (const uint8_t*)F, (const uint8_t*)F, (const uint8_t*)F,
                                              nullptr, (void*)F, HXQ_F32, M, N, K, (void*)F, w > 0 ? w - 1 : 0, nullptr);
            expect(w > 0 ? st == HXQ_ERR_UNSUPPORTED : st == (int)w, "fwd");
          }
        }
  for (int64_t M : dims)
    for (int64_t K : dims) {
      const int64_t w = hxq_rms_norm_bwd_workspace(M, K);
      expect(M < 0 || K < 0 || M > top || K > top ? w == HXQ_ERR_SHAPE : w >= 0, "norm workspace");
    }
  for (int64_t E : {(int64_t)0, (int64_t)-1, (int64_t)65536, INT64_MAX})
    expect(hxq_linear_fwd_fp8_experts_workspace(HXQ_F32, 1, 1, E, 1, 1) == HXQ_ERR_SHAPE, "experts");
  if (fails == 0) printf("fp8 host sanitize: %d checks ok\n", checks);
  return fails != 0;
}
