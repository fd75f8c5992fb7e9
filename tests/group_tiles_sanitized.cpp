// The rules of the grouped products' tiles (csrc/validate.hpp) under the
// sanitizers.  Reads lines "form dtype R E n r halves" and prints the tile, the
// parts of the reduction and whether column tiles start apart; then checks
// that every launch of allowed sizes holds its threads.
#include <stdio.h>
#include <string.h>

#include <random>

#include "validate.hpp"

using namespace swg;

static RowForm form_of(const char* name) {
  return !strcmp(name, "gated") ? RowForm::kGated : !strcmp(name, "recompute") ? RowForm::kRecompute
         : !strcmp(name, "nt") ? RowForm::kNT : RowForm::kNN;
}

int main() {
  char form[16];
  int dtype, halves;
  long long R, E, n, r;
  while (scanf("%15s %d %lld %lld %lld %lld %d", form, &dtype, &R, &E, &n, &r, &halves) == 7) {
    const RowForm f = form_of(form);
    const RowTile t = row_tile(dtype, f, R, E, n);
    const bool nn = f == RowForm::kNN;
    printf("%d %d %d %d\n", t.bm, t.bn, nn ? split_parts(dtype, R, E, n, r, halves) : 1, !nn && weights_bound(R, E));
  }
  std::mt19937_64 g(5);
  auto size = [&](int64_t most) {
    return (int64_t)std::exp2(std::uniform_real_distribution<double>(0.0, std::log2((double)most))(g));
  };
  int64_t tried = 0, few = 0;
  for (int i = 0; i < 200000; ++i) {
    const int dt = (int)(g() % 2);
    const int64_t rows = size(kMaxDim), experts = size(SWIGLU_MAX_EXPERTS), c = chunk_elems(dt);
    const int64_t N = size(kMaxLd / 2 / c) * c, K = size(kMaxLd / c) * c;
    if (grouped_shape_status(dt, rows, experts, N, K) != SWIGLU_OK) continue;
    for (RowForm f : {RowForm::kGated, RowForm::kRecompute, RowForm::kNT, RowForm::kNN}) {
      const int64_t cols = f == RowForm::kNN ? K : N;
      const RowTile t = row_tile(dt, f, rows, experts, cols);
      const TileRule rule = tile_rule(dt, f);
      ++tried;
      few += t == rule.few;
      if (!(t == rule.large || t == rule.few) || row_column_tiles(t, rows, experts, cols) * t.threads >= (int64_t(1) << 32)) {
        fprintf(stderr, "tile of %lld rows, %lld experts, %lld columns\n", (long long)rows, (long long)experts, (long long)cols);
        return 1;
      }
    }
  }
  if (tried < 100000 || few < 1000 || few > tried - 1000) return 2;
  printf("group tiles: ok\n");
  return 0;
}
