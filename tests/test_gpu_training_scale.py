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


@pytest.mark.parametrize("n,d,v", [(300, 72, 40), (5000, 64, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_cross_entropy_weight_gradient_near_the_largest_number(n, d, v, dtype):
    # W = 0: every logit is 0 and p = 1 / v.  All targets are v - 1, so
    # dw[v - 1] = -g n (1 - 1 / v) h and dw[j] = g n h / v elsewhere: half the
    # type's largest number at most, from rows of h of that size and g of
    # about 1 / n, as the mean of the losses has.
    dev = _dev()
    print(f"large dw n={n} d={d} v={v} {dtype}", flush=True)
    top = float(torch.finfo(DTYPES[dtype]).max)
    w = torch.zeros(v, d, dtype=DTYPES[dtype], device=dev)
    t = torch.full((n,), v - 1, dtype=torch.int64, device=dev)
    h = torch.zeros(n, d, dtype=DTYPES[dtype], device=dev)
    big = 2.0 ** (126 if dtype != "fp16" else 14)
    h[:, d - 1] = big
    g = 0.5 * top / (big * n * (1 - 1 / v))
    lse = nsa.linear_cross_entropy(h, w, t)[1]
    dh, dw = nsa.linear_cross_entropy_backward(h, w, t, lse, g)
    assert torch.count_nonzero(dh) == 0 and torch.count_nonzero(dw[:, :d - 1]) == 0
    # Rounding to the type: dz, the result; g, lse, exp, the sum of n terms in
    # fp32.
    u = torch.finfo(DTYPES[dtype]).eps / 2
    rel = 2 * u + (n + 20) * 2.0 ** -24
    assert abs(float(dw[v - 1, d - 1]) / (-0.5 * top) - 1) <= rel
    off = dw[:v - 1, d - 1].double() / (0.5 * top / (v - 1)) - 1
    assert float(off.abs().max()) <= rel


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_cross_entropy_hidden_gradient_near_the_largest_number(dtype):
    # H = 0: every logit is 0.  W is a, but -a in the target's row:
    # dh = g (sum_j p_j w_j - w_t) = 2 g a (1 - 1 / v), in reach of the type
    # only with its g.
    dev = _dev()
    n, d, v = 130, 96, 500
    a = (1.5 * 2.0 ** 127) if dtype != "fp16" else 49152.0
    g = 0.125
    w = torch.full((v, d), a, dtype=DTYPES[dtype], device=dev)
    w[7] = -a
    h = torch.zeros(n, d, dtype=DTYPES[dtype], device=dev)
    t = torch.full((n,), 7, dtype=torch.int64, device=dev)
    lse = nsa.linear_cross_entropy(h, w, t)[1]
    dh, dw = nsa.linear_cross_entropy_backward(h, w, t, lse, g)
    assert torch.count_nonzero(dw) == 0
    # dz's entries are off by u and a few u32 each, and add up to 2 g in
    # magnitude; the sum of v terms in fp32.
    u = torch.finfo(DTYPES[dtype]).eps / 2
    rel = 2 * u + (v + 20) * 2.0 ** -24
    off = dh.double() / (2 * g * a * (1 - 1 / v)) - 1
    assert float(off.abs().max()) <= rel


@pytest.mark.parametrize("size", [2.0 ** 90, 2.0 ** 120])
def test_cross_entropy_gradients_of_huge_coefficients_bf16(size):
    dev = _dev()
    n, d, v = 200, 128, 300
    print(f"coefficients near {size}", flush=True)
    h, w, t, dloss = _xent_inputs(n, d, v, "bf16", dev, seed=9)
    _check_xent(n, d, v, "bf16", dev, h, w, t, size * (0.5 + n * dloss))
