"""Calls that, between them, launch every kernel build of the training step's
operators.

tests/test_gpu_training_builds.py runs them on the GPU against 64 bits;
tests/test_training_coverage.py checks on the host that they reach every
cross entropy build that a sweep over sizes, types and alignment reaches
(plan_linear_cross_entropy), and every class of row width of layer norm and
the embedding.
"""

# Cross entropy, (rows, cols, vocabulary, dtypes).
ALL = ("bf16", "fp16", "fp32")
HALF = ("bf16", "fp16")
XENT_CASES = [
    # A few rows, which take whole rows of W: one to eight of them, whole
    # vectors, a partial last one, less than one.
    *[(n, d, 333, ALL) for n in (1, 2, 3, 7) for d in (72, 77, 3)],
    (4, 64, 500, ALL),
    # Short, wide tiles; the small edge, a block's join per row and per 16.
    (100, 200, 700, ALL),
    (150, 128, 400, ALL),
    (1100, 72, 300, ALL),
    # Either edge with work-groups that take several tiles, each of more
    # k-tiles than the three LDS stages hold, in dz and in both gradients.
    # Rows that need staging copies (264, 200, 136, ...) and rows that do not.
    (1000, 264, 20000, HALF),
    (385, 264, 50001, HALF),
    (1153, 600, 20000, HALF),
    (1000, 1408, 32003, HALF),
    (70, 136, 9001, ("fp32",)),
    (193, 200, 32003, ("fp32",)),
    (70, 1408, 25001, ("fp32",)),
    (577, 768, 5000, ("fp32",)),
    # Several pieces of the vocabulary, whose dH adds up: the large edge, and
    # the small one.
    (9000, 200, 32003, HALF),
    (1500, 200, 16001, ("fp32",)),
    (20000, 64, 15000, ALL),
]
XENT_RUNS = [(n, d, v, t) for n, d, v, types in XENT_CASES for t in types]

# Layer norm: the widest row of each build, in vectors of 16 bytes, whole and
# with a partial vector at the end, and the narrowest of the next.
NORM_VECTORS = (1, 32, 33, 64, 65, 96, 97, 128, 129, 192, 193, 256, 257, 512, 513, 1024, 1025, 2048)


def norm_widths(element_size):
    v = 16 // element_size
    widths = {n * v - off for n in NORM_VECTORS for off in (0, 1)} | {1, v - 1, v + 1}
    if element_size == 4:
        # fp32 rows in registers go on to 4096 vectors.
        widths |= {2049 * v, 2049 * v - 1, 4096 * v, 4096 * v - 1}
    return sorted(widths | {16384 + v, 16385})


# Embedding: one, two and four vectors a lane, several slices of columns;
# whole vectors, a partial last one, less than one.
def embed_widths(element_size):
    v = 16 // element_size
    wave = 64 * v
    return sorted({v - 1, 1} | {n - off for n in (wave, 2 * wave, 4 * wave, 9 * wave) for off in (0, 1)})
