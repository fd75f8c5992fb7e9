"""Sizes at which the products of rows in order of expert take their large tiles over many k-steps.

A case: the product's form, its type, the rows of each expert (2 rows of no expert in front of them, 3 behind), N, K, the
tile that it takes (rows, columns), and whether its column tiles start at different places of the reduction.  The
reductions are 13 k-steps of 32 bf16 and a remainder (fp32: 13 of 32 too, so that sums are folded within them).
"""
THREE, TWO = [300, 0, 400], [250, 350]       # at most 256 rows per expert on average, and more

# The gate/up stage and its recompute: n = N columns, reduction K.
GATED = [("bf16", THREE, 4552, 424, (256, 128), True), ("bf16", TWO, 5720, 424, (256, 128), False),
         ("f32", THREE, 2084, 424, (128, 64), True), ("f32", TWO, 2788, 424, (128, 64), False)]
# y = x W^T: n = N columns, reduction K; dx = dy W with N and K exchanged: n = K columns, reduction N, not split.
SINGLE = [("bf16", THREE, 9144, 424, (256, 256), True), ("bf16", TWO, 11480, 424, (256, 256), False),
          ("f32", THREE, 4196, 424, (128, 128), True), ("f32", TWO, 5604, 424, (128, 128), False)]


def rows_of(counts):
    return 2 + sum(counts) + 3


def queries():
    """(form, type, rows, experts, columns of the output, reduction, halves, tile, apart) of all cases."""
    for dt, counts, N, K, tile, apart in GATED:
        for form in ("gated", "recompute"):
            yield form, dt, rows_of(counts), len(counts), N, K, 1, tile, apart
    for dt, counts, N, K, tile, apart in SINGLE:
        yield "nt", dt, rows_of(counts), len(counts), N, K, 1, tile, apart
        for halves in (1, 2):
            yield "nn", dt, rows_of(counts), len(counts), N, K, halves, tile, False
