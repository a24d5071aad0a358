"""The status word of the training step's operators: every result that is not
finite is reported, wherever it is written, and nothing else is.

The inputs are made so that exactly one of a call's results overflows.
"""

import pytest
import torch

import newton_schulz_matrix_amd as nsa
from newton_schulz_matrix_amd import _binding as B

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BAD = B.NS_ERR_NONFINITE | B.STATUS_AT_OUTPUT


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _word(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


# ---------------------------------------------------------------------------
# Cross entropy: the weights' gradient.
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n,d,v", [(1, 64, 40), (300, 72, 40), (150, 200, 700), (1000, 64, 5000)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("need_dh", [False, True])
def test_cross_entropy_reports_an_overflowing_weight_gradient(n, d, v, dtype, need_dh):
    # W = 0: all logits are 0, p = 1 / v, dh = 0.  Every row's target is
    # v - 1, so dw[v - 1] = -n (1 - 1 / v) g h and dw[j] = n g h / v elsewhere.
    dev = _dev()
    print(f"dw overflow n={n} d={d} v={v} {dtype} need_dh={need_dh}", flush=True)
    top = float(torch.finfo(DTYPES[dtype]).max)
    w = torch.zeros(v, d, dtype=DTYPES[dtype], device=dev)
    t = torch.full((n,), v - 1, dtype=torch.int64, device=dev)
    for factor, overflows in ((0.5, False), (1.5, True)):
        # |dw[v - 1]| is factor times the largest number in the last column,
        # 0 in the others.
        h = torch.zeros(n, d, dtype=DTYPES[dtype], device=dev)
        h[:, d - 1] = 2.0 ** (126 if dtype != "fp16" else 14)
        g = factor * top / (float(h[0, d - 1]) * n * (1 - 1 / v))
        lse = nsa.linear_cross_entropy(h, w, t)[1]
        st = _word(dev)
        dh, dw = nsa.linear_cross_entropy_backward(h, w, t, lse, g, need_dh=need_dh, status=st)
        assert torch.isinf(dw[v - 1, d - 1]) == overflows
        assert torch.isfinite(dw[:v - 1]).all() and torch.count_nonzero(dw[:, :d - 1]) == 0
        assert not need_dh or torch.count_nonzero(dh) == 0
        assert int(st.item()) == (BAD if overflows else 0)
