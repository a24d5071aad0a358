"""The waits of the streamed products, read from the assembly that the
compiler makes of them (host only).

A work-group's stages are handed over by a wait for the copies that filled
them and a barrier.  The wait is a number of younger memory operations that
may still be in flight; the counter has six bits, and at its maximum, 63, the
instruction does not wait at all.
"""

import os
import re
import subprocess

import pytest

from newton_schulz_matrix_amd import build as nsbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

try:
    HIPCC = nsbuild.hipcc()
except RuntimeError:
    HIPCC = None

# And the vector stores that their waits count on at a tile's border: per
# 32 x 32 block of a wave, of dz 6 in 16 bits and 8 in fp32, of dH's sums 4
# (beside dW's own 2, which its waits do not count).
KERNELS = [("k_xent_dz<__bf16, 192, 192>(XentArgs)", 9 * 6), ("k_xent_dz<float, 64, 64>(XentArgs)", 8),
           ("k_xent_fwd<__bf16, 192, 192>(XentArgs)", 0),
           ("k_xent_grads<__bf16, 192, 192>(XentDwArgs, XentDhArgs)", 9 * (4 + 2))]


def _steps(text):
    """Copies, waits (with their vmcnt, None without one) and barriers, in the
    order of the text."""
    out = []
    for line in text.splitlines():
        s = line.strip()
        if s.startswith("buffer_load") and s.split(";")[0].rstrip().endswith("lds"):
            out.append(("copy", None))
        elif s.startswith("s_waitcnt"):
            m = re.search(r"vmcnt\((\d+)\)", s)
            out.append(("wait", int(m[1]) if m else None))
        elif s.startswith("s_barrier"):
            out.append(("barrier", None))
    return out


@pytest.mark.skipif(HIPCC is None, reason="hipcc not found")
@pytest.mark.parametrize("kernel,stores", KERNELS)
def test_every_barrier_behind_copies_has_a_wait_that_waits(kernel, stores, tmp_path):
    src = tmp_path / "one.hip"
    src.write_text(f'#include "xent.hpp"\nnamespace nsk {{ template __global__ void {kernel}; }}\n')
    got = subprocess.run([HIPCC, *nsbuild.HIP_FLAGS, "-I", nsbuild.CSRC, "-I", nsbuild.INCLUDE, "-S", "--cuda-device-only",
                          str(src), "-o", "-"], capture_output=True, text=True, timeout=600)
    assert got.returncode == 0, got.stderr[-2000:]
    # None of the stores is merged with another or left out.
    assert len(re.findall(r"^\s*global_store_dwordx[24]\b", got.stdout, re.M)) >= stores
    steps = _steps(got.stdout)
    assert sum(k == "barrier" for k, _ in steps) >= 7 and sum(k == "copy" for k, _ in steps) >= 36
    waited, seen = True, 0
    for kind, count in steps:
        if kind == "copy":
            waited = False
        elif kind == "wait":
            waited |= count is not None and count < 63
        else:
            assert waited, f"barrier {seen} follows copies without a wait"
            seen += 1
