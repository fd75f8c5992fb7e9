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

int main() {
  resident();
  if (failures) return 1;
  printf("block rules: ok\n");
  return 0;
}
