"""Calls that, between them, launch every kernel build of the gated
feed-forward block.

tests/test_gpu_gated_mlp.py runs them on the GPU against 64 bits;
tests/test_block_host.py checks on the host that they reach every build that
a sweep over sizes, types and alignment reaches (plan_gated_mlp).
"""

ALL = ("bf16", "fp16", "fp32")
HALF = ("bf16", "fp16")
# (rows, cols, inner, dtypes).
MLP_CASES = [
    # A few rows, which take whole rows of the weights: whole vectors, a
    # partial last one, less than one.
    *[(n, d, f, ALL) for n in (1, 2, 3, 4, 7) for d, f in ((72, 40), (77, 203), (3, 2), (2, 65))],
    # Tiles: one, ragged ones, one row and one column more than a tile.
    (9, 64, 64, ALL), (40, 72, 136, ALL), (129, 129, 65, ALL), (128, 128, 128, ALL), (10, 1, 1, ALL), (193, 7, 500, ALL),
    (70, 300, 5, ALL), (48, 256, 3000, ALL), (300, 1000, 731, ALL),
    # The larger tiles, work-groups with several of them, each of more k-tiles
    # than the three LDS stages hold.
    (1003, 520, 1407, ALL), (1500, 264, 3001, HALF), (5000, 776, 264, HALF), (5000, 1000, 2800, ("bf16",)),
    (4000, 200, 3001, ("fp32",)), (4000, 776, 264, ("fp32",)), (1500, 64, 3001, ("fp32",)),
    # Copies in a launch of their own, as the tiles leave too few compute
    # units to them.
    (513, 1, 14336, HALF), (1, 1000, 14336, HALF), (513, 1, 2048, HALF), (1003, 1, 14336, ("fp16",)), (8192, 1, 1407, ("fp32",)),
]
MLP_RUNS = [(n, d, f, t) for n, d, f, types in MLP_CASES for t in types]
