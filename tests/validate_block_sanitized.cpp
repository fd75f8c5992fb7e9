// The routed block's host-side validation (csrc/validate.hpp) under the
// sanitizers: every validator over a grid of extreme sizes must return a
// status in range without overflow, workspace sizes are 0 exactly for the
// shapes that are rejected, and no region wraps.
#include <math.h>
#include <stdio.h>

#include <limits>
#include <vector>

#include "validate.hpp"

static int failures = 0;
static void check(bool ok, const char* what) {
  if (!ok) {
    fprintf(stderr, "%s\n", what);
    ++failures;
  }
}
static bool in_range(int st) { return st >= 0 && st <= 9; }

int main() {
  using namespace swg;
  const int64_t big = std::numeric_limits<int64_t>::max(), small = std::numeric_limits<int64_t>::min();
  const std::vector<int64_t> dims = {small, -8, -1, 0, 1, 2, 8, 16, 17, 64, 65, 1024, 1025, 16384, 16385, int64_t(1) << 20,
                                     (int64_t(1) << 20) + 8, (int64_t(1) << 31) - 1, int64_t(1) << 31, int64_t(1) << 40, big};
  const std::vector<int64_t> few = {small, -1, 0, 1, 2, 16, 17, 64, 65, big};
  void* const A = reinterpret_cast<void*>(0x10000);
  long calls = 0;
  for (int64_t T : dims)
    for (int64_t E : dims)
      for (int64_t k : few)
        for (int dt : {-1, 0, 1, 2}) {
          const int st = validate_route(1, dt, T, E, k, A, 1.0f, A, A, A, true);
          check(in_range(st), "route status");
          if (st == SWIGLU_OK) check(T >= 0 && E >= 1 && E <= 1024 && k >= 1 && k <= 16 && k <= E, "route accepts");
          ++calls;
        }
  for (int64_t N : dims)
    for (int64_t K : dims)
      for (int64_t T : few)
        for (int64_t k : few) {
          const size_t total = moe_workspace_total(T, N, K, k);
          if (moe_shape_status(T, N, K, k) != SWIGLU_OK) {
            check(total == 0, "moe workspace of a rejected shape");
          } else {
            const MoeLayout L = moe_layout(T, N, K, k);
            check(L.total == total && L.off_part <= L.total && L.off_part >= (size_t)T * k * N * 4 &&
                      L.total - L.off_part >= (moe_parts(K, 32) > 1 ? (size_t)moe_parts(K, 32) * T * K * 4 : 0) &&
                      moe_parts(K, 16) <= moe_parts(K, 32),
                  "moe regions");
          }
          for (int64_t stride : {small, int64_t(-8), int64_t(0), int64_t(8), int64_t(1) << 40, int64_t(1) << 49, big})
            for (int64_t E : few) {
              check(in_range(validate_moe(T, E, k, N, K, A, A, A, A, stride, A, stride, A, stride, A, A, total)), "moe status");
              ++calls;
            }
        }
  for (int64_t rows : dims)
    for (int64_t cols : dims)
      for (int64_t groups : dims) {
        const size_t total = norm_bwd_workspace_total(rows, cols, groups);
        if (norm_shape_status(rows, cols, groups) != SWIGLU_OK) check(total == 0, "norm workspace of a rejected shape");
        else if (rows > 0) check(total >= (size_t)8 * cols, "norm workspace");
        for (float eps : {0.0f, 1e-6f, NAN, INFINITY}) {
          check(in_range(validate_norm_fwd(1, rows, cols, groups, A, A, A, groups ? A : nullptr, A, 1, 1, 0, eps, A, A)),
                "norm status");
          check(in_range(validate_norm_bwd(0, rows, cols, groups, A, A, A, groups ? A : nullptr, A, A, A, 1, 1, 0, eps, A, A, A,
                                           groups ? A : nullptr, A, A, total)),
                "norm backward status");
          calls += 2;
        }
      }
  if (failures) return 1;
  printf("block: ok (%ld calls)\n", calls);
  return 0;
}
