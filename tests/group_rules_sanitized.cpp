// The rules of rows in order of expert that lie in csrc/validate.hpp, under
// the sanitizers: the plan's shares, and which gradients may be clipped
// together, against a check of every pair of bytes.
#include <stdio.h>

#include <random>

#include "validate.hpp"

static int failures = 0;
static void check(bool ok, const char* what) {
  if (!ok) {
    fprintf(stderr, "%s\n", what);
    ++failures;
  }
}

// Every pair falls to one wave's run of whole 64s, and the workspace holds
// every block's counts.
static void plan() {
  using namespace swg;
  for (int64_t n : {int64_t(0), int64_t(1), int64_t(1023), int64_t(1024), int64_t(8192), int64_t(8193), int64_t(131072),
                    int64_t(131073), int64_t(262144), int64_t(1) << 24, (int64_t(1) << 31) - 1}) {
    const int64_t per = plan_per_block(n), blocks = plan_blocks(n);
    check(per % kPlanThreads == 0 && blocks >= 1 && blocks <= kPlanBlocks, "plan: shares");
    check(blocks * per >= n && (blocks - 1) * per < (n < 1 ? 1 : n), "plan: every pair once");
    check(n > kPlanOne || blocks == 1, "plan: one workgroup");
  }
  check(plan_workspace_total(8193, 1, 1024) >= (size_t)plan_blocks(8193) * 1025 * 4, "plan: room");
}

static bool overlap_by_bytes(int64_t count, const int* dt, void* const* g, const int64_t* n, void* const* o) {
  auto len = [&](int64_t i) { return (uintptr_t)(n[i] * swg::elem_size(dt[i])); };
  auto cross = [](uintptr_t a, uintptr_t la, uintptr_t b, uintptr_t lb) { return a < b + lb && b < a + la; };
  auto u = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  for (int64_t i = 0; i < count; ++i)
    for (int64_t j = 0; j < count; ++j) {
      if (n[i] == 0 || n[j] == 0) continue;
      void* const wi = o ? o[i] : g[i];
      void* const wj = o ? o[j] : g[j];
      if (i != j && cross(u(wi), len(i), u(wj), len(j))) return true;
      // What i writes against what j reads.
      if (o && !(i == j && o[i] == g[i]) && cross(u(wi), len(i), u(g[j]), len(j))) return true;
    }
  return false;
}

static void overlaps() {
  std::mt19937 r(7);
  int found = 0;
  for (int round = 0; round < 20000; ++round) {
    const int64_t count = 1 + r() % 5;
    int dt[5];
    int64_t n[5];
    void *g[5], *o[5];
    for (int i = 0; i < count; ++i) {
      dt[i] = r() % 2;
      n[i] = r() % 7;
      g[i] = reinterpret_cast<void*>(uintptr_t(0x1000 + 4 * (r() % 60)));
      o[i] = r() % 3 == 0 ? g[i] : reinterpret_cast<void*>(uintptr_t(0x1000 + 4 * (r() % 90)));
    }
    for (void* const* outs : {(void* const*)nullptr, (void* const*)o}) {
      const bool want = overlap_by_bytes(count, dt, g, n, outs);
      found += want;
      check((swg::check_disjoint(count, dt, g, n, outs) == SWIGLU_ERR_ARG) == want, "overlap");
    }
  }
  check(found > 1000, "overlaps were tried");
}

static void sizes() {
  using namespace swg;
  for (int dt : {SWIGLU_F32, SWIGLU_BF16})
    for (int64_t R : {1, 3, 35, 64, 65, 130, 500, 4001, 100000})
      for (int64_t n : {8, 248, 256, 264, 3824, 8192})
        for (int64_t r : {0, 8, 512, 1024, 13448, 131072})
          for (int halves : {1, 2})
            for (int64_t E : {1, 2, 39, 1024}) {
              const int parts = split_parts(dt, R, E, n, r, halves);
              const SplitTile t = dt == SWIGLU_BF16 ? kSplitBf16 : kSplitF32;
              const int64_t steps = halves * ((r + t.step - 1) / t.step);
              check(parts >= 1 && (parts == 1 || (parts * 8 <= steps && parts <= t.target)), "parts of 8 k-steps at least");
              check(parts == 1 || (size_t)(parts * R * n * 4) <= split_bytes(dt, R, n, r, halves), "the parts' sums fit");
              const int row_parts = split_row_parts(dt, R, E, r, n, halves);
              const SplitTile w = dt == SWIGLU_BF16 ? kSplitRowsBf16 : kSplitRowsF32;
              check(row_parts >= 1 && (row_parts == 1 || row_parts * 8 * E * w.step <= R), "8 k-steps of each expert's rows");
              check(row_parts == 1 || (size_t)(row_parts * E * halves * r * n * 4) <= split_row_bytes(dt, R, r, n, halves),
                    "the rows' parts' sums fit");
              check(split_row_bytes(dt, R, r, n, halves) <= (size_t)w.target * w.bm * w.bn * 4 + 256, "as many as tiles of weights");
              check(split_bytes(dt, R, n, r, halves) <= (size_t)t.target * t.bm * t.bn * 4 + 256, "as many as tiles");
            }
  check(grouped_bwd_workspace_total(SWIGLU_BF16, (int64_t(1) << 30) - 1024, 8, 8, true) > size_t(1) << 34, "rows near 2^30");
  check(grouped_bwd_workspace_total(SWIGLU_BF16, kMaxDim, 8, 8, true) == 0, "more row tiles than a launch has");
  check(grouped_shape_status(SWIGLU_F32, kMaxDim, 1024, kMaxDim, kMaxDim) != SWIGLU_OK, "sizes that overflow");
  check(check_pairs(INT64_MAX, 16) == SWIGLU_ERR_SHAPE && check_pairs(kMaxDim, 1) == SWIGLU_OK, "pairs");
  check(rows_status(SWIGLU_F32, int64_t(1) << 23, 1, kMaxDim / 4 * 4) == SWIGLU_ERR_UNSUPPORTED, "wide rows");
  check(grad_norm_workspace_total(INT64_MAX) == 0, "count");
}

int main() {
  plan();
  overlaps();
  sizes();
  if (failures == 0) printf("group rules: ok\n");
  return failures != 0;
}
