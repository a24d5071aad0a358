"""The residual norms' kernel builds that test_gpu_residual_norm.py's widths
leave out, and column sums over millions of narrow rows."""

import pytest
import torch

import newton_schulz_matrix_amd as nsa
from resnorm_cases import MORE_WIDTHS
from test_gpu_residual_norm import TYPES, U32, _check, _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", MORE_WIDTHS)
@pytest.mark.parametrize("dtype,pdtype", TYPES)
@pytest.mark.parametrize("rows", [1, 40, 1100])
def test_matches_the_oracle_at_more_widths(rows, cols, dtype, pdtype):
    _check(rows, cols, dtype, pdtype, 2 if rows > 1 else 1, seed=cols + rows)


@pytest.mark.parametrize("cols", [1, 3])
@pytest.mark.parametrize("groups", [1, 4, 1 << 22])
def test_sums_over_millions_of_narrow_rows(cols, groups):
    # Terms of one sign and size: a thread's running sum rounds each of them
    # the same way.  A sum is made of runs of 256 terms, their totals (512 blocks,
    # with a gate row for 4 rows 4 rows at a time: 32), two joins of 32 and of
    # 16 + 32, and the roundings of each term's product.
    dev = _dev()
    rows, term = 1 << 24, 1 + 1.5 * 2.0 ** -12
    print(f"residual norm {rows} x {cols}, {groups} gate rows", flush=True)
    ones = torch.ones(rows, cols, device=dev)
    stat, w = torch.ones(rows, device=dev), torch.ones(cols, device=dev)
    grad = torch.full((rows, cols), term, device=dev)
    bound = (256 + 32 + 32 + 48 + 8) * U32
    if groups == 1:
        dw = nsa.residual_norm_backward(None, grad, ones, rstd=stat, weight=w)[4]
        assert ((dw.double() / (rows * term) - 1).abs() <= bound).all()
    gate = torch.ones(groups, cols, device=dev)
    _, _, dgate, dwb, _ = nsa.residual_norm_backward(grad, None, ones, ones, stat, gate=gate, branch_weight=w)
    for got, count in ((dwb, rows), (dgate, rows // groups)):
        off = float((got.double() / (count * term) - 1).abs().max())
        print(f"off {off / U32:.1f} half steps", flush=True)
        assert off <= bound
