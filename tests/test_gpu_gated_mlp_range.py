"""The gated feed-forward block far from one: activations of the largest
numbers."""

import numpy as np
import pytest
import torch

import newton_schulz_matrix_amd as nsa
from test_gpu_gated_mlp import ACTS, DTYPES, HALF_STEP, U32, _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_activations_of_any_finite_number(act, dtype):
    # One column of a gate for each size.  Both value and slope end at 0 on the
    # left and at a and 1 on the right, exactly from |a| = 128 on, where exp(-|a|)
    # is below fp32's smallest number.
    dev = _dev()
    print(f"activation {act} {dtype}", flush=True)
    sizes = np.array([128, 1e3, 1e6, 1e12, 1.1e13, 1.3e13, 1e14, 1e18, 1e19, 2e19, 1e25, 1e30, 1e38, 3.3e38])
    a = torch.tensor(np.concatenate([-sizes, sizes])).to(DTYPES[dtype]).to(dev)
    n, d, f = 130, 72, a.numel()
    x = torch.zeros(n, d, dtype=DTYPES[dtype], device=dev)
    x[:, 0], x[:, 1] = 1.0, 2.0 ** -100
    wg, wu = torch.zeros(f, d, dtype=x.dtype, device=dev), torch.zeros(f, d, dtype=x.dtype, device=dev)
    wg[:, 0], wu[:, 1] = a, 1.0
    wd = torch.zeros(d, f, dtype=x.dtype, device=dev)
    wd[:f] = torch.eye(f, device=dev, dtype=x.dtype)
    dy = torch.ones(n, d, dtype=x.dtype, device=dev)
    right = (a > 0).to(x.dtype)
    for rows in (2, n):
        y, gate, up = nsa.gated_mlp(x[:rows], wg, wu, wd, activation=act)
        assert torch.equal(gate[0], a.float()) and bool((up == 2.0 ** -100).all())
        # h = 2^-100 act(a): exact, and its sum has one term.
        assert torch.equal(y[:, :f].float(), (a * right * 2.0 ** -100).float().expand(rows, f))
    up = torch.full_like(gate, 0.5)
    dx, dwg, dwu, dwd = nsa.gated_mlp_backward(dy, x, wg, wu, wd, gate, up, activation=act, need_dx=False)
    # da = b slope, db = value: sums of n equal terms, of powers of two times
    # the values' digits, in fp32 (a sum of 130 terms is off by 131 u32).
    big = a.double() * right.double() * (n * 2.0 ** -100)
    assert torch.equal(dwg[:, 0].double(), right.double() * 0.5 * n)
    u = HALF_STEP[dtype]
    assert ((dwu[:, 1].double() - big).abs() <= (u + 132 * U32) * big).all()
