"""The waits of the fp16 second launches of the gated feed-forward block, read
from the assembly as in test_block_waits.py (host only): the same stores and
copies as the first, and at least as many barriers."""

import pytest

from test_block_waits import HIPCC, test_every_barrier_behind_copies_has_a_wait_that_waits as check

KERNELS = [("k_mlp_up<_Float16, 128, 256, true>(MlpUpArgs)", 4 * 2, 7, 36), ("k_mlp_up<_Float16, 128, 128, true>(MlpUpArgs)", 2 * 2, 7, 24),
           ("k_mlp_up<_Float16, 64, 128, true>(MlpUpArgs)", 2, 7, 18), ("k_mlp_dz<_Float16, 128, 128, true>(MlpDzArgs)", 4 * 4 + 2 * 12, 5, 24),
           ("k_mlp_dz<_Float16, 64, 128, true>(MlpDzArgs)", 2 * 16, 4, 18)]


@pytest.mark.skipif(HIPCC is None, reason="hipcc not found")
@pytest.mark.parametrize("kernel,stores,barriers,copies", KERNELS)
def test_the_second_launches_wait_as_the_first(kernel, stores, barriers, copies, tmp_path):
    check(kernel, stores, barriers, copies, tmp_path)
