"""Products that between them take every kernel and ring of moe_fp8_gemm and
moe_fp8_gemm_grouped on 148 SMs: (rows or counts of the groups, N, K, plan)."""

DENSE = [
    (3, 1000, 400, (16, 32, 7)),
    (32, 300, 2064, (16, 32, 7)),
    (4, 4001, 1040, (32, 32, 5)),
    (1, 8190, 528, (64, 32, 3)),
    (4, 8192, 2048, (64, 32, 3)),
    (30, 16391, 272, (128, 32, 4)),
    (32, 16384, 1936, (128, 32, 4)),
    (100, 2041, 400, (16, 128, 5)),
    (33, 4100, 1936, (32, 128, 4)),
    (97, 8200, 272, (64, 128, 4)),
    (128, 16400, 1040, (128, 128, 3)),
    (130, 32768, 272, (256, 128, 4)),
    (2500, 4095, 400, (256, 128, 4)),
]


def _spread(groups, rows):
    """`rows` one-row groups among `groups`, unevenly."""
    at = sorted({(i * i * 7 + 3 * i) % groups for i in range(rows)})
    return [1 if g in at else 0 for g in range(groups)]


# 31, 32, 33 rows, and a second row tile of one 32-row piece: a whole 32-row piece may be
# stored at once only where it does not reach into the next group
MIXED = [31, 32, 33, 100, 160, 0, 1, 129, 64, 0]

GROUPED = [
    (_spread(512, 20), 2048, 272, (128, 32, 4)),
    (_spread(100, 14), 2050, 528, (128, 32, 4)),
    ([3, 0, 20], 264, 2064, (16, 32, 7)),
    ([9, 0, 0, 11, 5], 1600, 272, (64, 32, 3)),
    ([5, 17], 2048, 400, (32, 32, 5)),
    (MIXED, 264, 400, (32, 128, 4)),
    (MIXED, 410, 400, (64, 128, 4)),
    ([40, 0, 33], 200, 400, (16, 128, 5)),
    (MIXED * 2, 600, 528, (128, 128, 3)),
    (MIXED * 10, 1000, 400, (256, 128, 4)),
    (MIXED * 10, 1001, 272, (256, 128, 4)),
    (MIXED * 30, 1000, 272, (256, 128, 3)),
    (MIXED * 30, 513, 400, (256, 128, 3)),
    (MIXED * 30, 257, 400, (128, 128, 3)),
    (MIXED * 30, 999, 272, (256, 128, 3)),
]
