// The launch rules of the routed block that lie in csrc/validate.hpp, under
// the sanitizers.
#include <stdio.h>

#include "validate.hpp"

static int failures = 0;
static void check(bool ok, const char* what) {
  if (!ok) {
    fprintf(stderr, "%s\n", what);
    ++failures;
  }
}

// The workgroups that a CU is taken to hold fit its registers' waves and its
// 160 KiB of LDS, and one more would not.
static void resident() {
  using swg::moe_resident;
  const size_t cu_lds = 160 * 1024;
  for (int waves = 1; waves <= 16; ++waves)
    for (int cu_waves = waves; cu_waves <= 16; ++cu_waves)
      for (size_t lds = 1; lds <= cu_lds; lds += 1021) {
        const int n = moe_resident(waves, cu_waves, lds);
        check(n >= 1 && n * waves <= cu_waves && n * lds <= cu_lds, "resident workgroups fit");
        check((n + 1) * waves > cu_waves || (n + 1) * lds > cu_lds, "no more would fit");
      }
  // The first product's, with a token mask of 8 KiB beside 8 KiB a wave: 4 of 4 waves, 2 of 8; with the pairs' ids and
  // weights beside it 3 of 4 waves would fit.
  check(moe_resident(4, 16, 4 * 8192 + 8192) == 4 && moe_resident(8, 16, 8 * 8192 + 8192) == 2 &&
            moe_resident(4, 16, 4 * 8192 + 16384) == 3 && moe_resident(1, 16, 8192 + 8192) == 10,
        "first product");
}

// The backward's parts: no more than the workspace has room for, and every
// row in one part's turn, for both element sizes and every launch shape.
static void parts() {
  using namespace swg;
  const int64_t cols[] = {1, 7, 8, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1024, 1864, 2048, 2051, 4096, 4097,
                          6001, 8192, 8193, 8201, 12288, 12289, 16383, 16384};
  const int64_t per_group[] = {1, 2, 3, 7, 16, 33, 170, 171, 511, 512, 513, 1024, 1537, 2048, 5000, 16385, 65536};
  for (int64_t c : cols)
    for (int64_t g : {0, 1, 2, 3, 5, 16, 17, 511, 512, 513, 2048, 2100, 1 << 20})
      for (int64_t n : per_group) {
        const int64_t rows = n * (g > 0 ? g : 1), groups = g > 0 ? g : 1;
        if (norm_shape_status(rows, c, g) != SWIGLU_OK) continue;
        const size_t total = norm_bwd_workspace_total(rows, c, g);
        check(total == (size_t)(2 * groups * norm_most_parts(rows, c, g) * c * 4 + 255) / 256 * 256, "norm workspace");
        for (int elem : {2, 4}) {
          const int64_t nch = (c * elem + 15) / 16, per = norm_bwd_parts(elem, rows, c, g);
          check(per >= 1 && per <= n && (size_t)(2 * groups * per * c * 4) <= total, "norm parts fit the workspace");
          check(norm_lanes(nch) || norm_wide_threads(nch, norm_chunks(nch)) <= 1024, "norm threads");
        }
      }
  check(norm_bwd_parts(2, 0, 64, 3) == 0 && norm_bwd_workspace_total(0, 64, 3) == 0, "no rows");
}

int main() {
  resident();
  parts();
  if (failures) return 1;
  printf("block rules: ok\n");
  return 0;
}
