"""The waits of the gated feed-forward block's products, read from the
assembly that the compiler makes of them (host only; see
test_training_waits.py)."""

import re
import subprocess

import pytest

from newton_schulz_matrix_amd import build as nsbuild
from test_training_waits import HIPCC, _steps

# And the vector stores that the streams' waits count on at a tile's border,
# per 32 x 32 block of a wave: of h 2 in 16 bits and 4 in fp32 (for half the
# blocks, beside twice as many of a and b, which are not counted on).  dh's
# tiles are no stream (4 of da and db in rows, 12 of the transposed results, which
# in its large 16-bit tile leave 32 columns of 64 rows at a time).  Barriers and
# copies: at least three steps' (two for dh).
KERNELS = [("k_mlp_up<__bf16, 128, 256>(MlpUpArgs)", 4 * (2 + 4), 7, 36),
           ("k_mlp_up<_Float16, 64, 128>(MlpUpArgs)", 2 + 4, 7, 18),
           ("k_mlp_up<float, 64, 128>(MlpUpArgs)", 4 + 8, 7, 18),
           ("k_mlp_dz<_Float16, 128, 128>(MlpDzArgs)", 4 * 4 + 2 * 12, 5, 24), ("k_mlp_dz<__bf16, 64, 128>(MlpDzArgs)", 2 * 16, 4, 18),
           ("k_mlp_dz<float, 64, 64>(MlpDzArgs)", 20, 4, 12),
           ("k_mlp_products<__bf16, 192, 192>(MlpGradArgs)", 0, 7, 36), ("k_mlp_products<__bf16, 64, 128>(MlpGradArgs)", 0, 7, 18)]


@pytest.mark.skipif(HIPCC is None, reason="hipcc not found")
@pytest.mark.parametrize("kernel,stores,barriers,copies", KERNELS)
def test_every_barrier_behind_copies_has_a_wait_that_waits(kernel, stores, barriers, copies, tmp_path):
    src = tmp_path / "one.hip"
    src.write_text(f'#include "mlp.hpp"\nnamespace nsk {{ template __global__ void {kernel}; }}\n')
    got = subprocess.run([HIPCC, *nsbuild.HIP_FLAGS, "-I", nsbuild.CSRC, "-I", nsbuild.INCLUDE, "-S", "--cuda-device-only",
                          str(src), "-o", "-"], capture_output=True, text=True, timeout=600)
    assert got.returncode == 0, got.stderr[-2000:]
    # None of the stores is merged with another or left out.
    assert len(re.findall(r"^\s*global_store_dwordx[24]\b", got.stdout, re.M)) >= stores
    steps = _steps(got.stdout)
    assert sum(k == "barrier" for k, _ in steps) >= barriers and sum(k == "copy" for k, _ in steps) >= copies
    waited, seen = True, 0
    for kind, count in steps:
        if kind == "copy":
            waited = False
        elif kind == "wait":
            waited |= count is not None and count < 63
        else:
            assert waited, f"barrier {seen} follows copies without a wait"
            seen += 1
