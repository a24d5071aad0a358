"""Row widths that, between them, launch every kernel build of the residual
norms.

tests/test_gpu_residual_norm.py and tests/test_gpu_residual_norm_builds.py run
them on the GPU against 64 bits; tests/test_block_builds_host.py checks on the
host that they reach every build.
"""

# Beside test_gpu_residual_norm.py's: partial last vectors where a half-wave or
# a wave holds two vectors of fp32 each.
MORE_WIDTHS = [130, 255, 385, 511]


def build_of(cols, io, pt):
    """(vectors a thread, threads a row, whole vectors or not) for a row of
    `cols` elements of `io` bytes with parameters of `pt` bytes; None where a
    row goes element by element."""
    v = 16 // io
    if cols < v or cols > 8192:
        return None
    n = -(-cols // v)
    if n <= 256:
        form = next(f for most, f in ((32, (1, 32)), (64, (2, 32)), (96, (3, 32)), (128, (2, 64)), (256, (1, 256))) if n <= most)
    elif io == 4:
        form = (2, 256) if n <= 512 else (2, 512) if n <= 1024 else (2, 1024)
    elif n <= 512:
        form = (2, 256) if pt == 2 else (1, 512)
    else:
        form = (1, 1024)
    return (*form, cols % v == 0)
