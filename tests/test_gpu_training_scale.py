"""The cross entropy's gradients where the losses' gradients or the operands
are far from 1: dz is held in units of the largest of them, and neither that
unit nor the sums on the way may cost a result that the type can hold.
"""

import pytest
import torch

import newton_schulz_matrix_amd as nsa
from newton_schulz_matrix_amd import _binding as B

from test_gpu_training import DTYPES, _check_xent, _dev, _word, _xent_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [1e-30, 1e-34, 3e-35, 1e-36])
def test_cross_entropy_gradients_of_tiny_coefficients_bf16(size):
    # bf16 holds gradients of this size: they are checked as any others (the
    # bound's absolute part, half a step of dz times the operands, is some
    # hundred times bf16's smallest step, 2^-133).
    dev = _dev()
    n, d, v = 200, 128, 300
    print(f"coefficients near {size}", flush=True)
    h, w, t, dloss = _xent_inputs(n, d, v, "bf16", dev, seed=8)
    _check_xent(n, d, v, "bf16", dev, h, w, t, size * (0.5 + n * dloss))
