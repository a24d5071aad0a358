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


# ---------------------------------------------------------------------------
# Layer norm: the parameters' gradients.
# ---------------------------------------------------------------------------

# Rows that share a wave, rows of a block, rows in registers of 1024 threads,
# rows that are taken element by element, and less than a vector.
@pytest.mark.parametrize("rows,cols", [(10000, 768), (10000, 97), (6000, 4096), (4000, 9000), (2000, 20001), (10000, 4)])
@pytest.mark.parametrize("which", ["dbias", "dweight"])
def test_layer_norm_reports_overflowing_parameter_gradients(rows, cols, which):
    # Every other row of x is turned round, so that one of the two sums
    # cancels and the other grows to 80000 times a number of about 1: past
    # fp16, well inside the dx that the same call writes, and inside fp32.
    dev = _dev()
    print(f"norm sums {rows}x{cols} {which}", flush=True)
    g = torch.Generator().manual_seed(cols)
    sign = (1 - 2 * (torch.arange(rows) % 2)).float()[:, None].to(dev)
    base = torch.where(torch.arange(cols) % 2 == 0, 1.0, -1.0) * (1 + 0.25 * torch.rand(cols, generator=g))
    base = (base - base.mean()).half().to(dev)
    x = base * sign.half()
    size = 80000.0 / rows
    dy = torch.full((rows, cols), size, device=dev).half() if which == "dbias" else (size * sign).half().expand(rows, cols).contiguous()
    for pdtype, overflows in ((torch.float16, True), (torch.float32, False)):
        w = torch.ones(cols, dtype=pdtype, device=dev)
        _, mean, rstd = nsa.layer_norm(x, w)
        st = _word(dev)
        dx, dw, db = nsa.layer_norm_backward(dy, x, mean, rstd, w, status=st)
        assert torch.isfinite(dx).all()
        grown, cancelled = (db, dw) if which == "dbias" else (dw, db)
        assert torch.isfinite(cancelled).all() and torch.isinf(grown).any() == overflows
        assert not torch.isnan(grown).any()
        assert int(st.item()) == (BAD if overflows else 0)
        # Without the parameters' gradients there is nothing to report.
        st.zero_()
        nsa.layer_norm_backward(dy, x, mean, rstd, w, params=False, status=st)
        assert int(st.item()) == 0


# ---------------------------------------------------------------------------
# Cross entropy: the loss.
# ---------------------------------------------------------------------------

# One row by whole rows of W; tiles with a block's join per row; short, wide
# tiles; many rows' join.
@pytest.mark.parametrize("n,d,v", [(1, 64, 100), (6, 100, 300), (40, 64, 300), (500, 72, 400), (1500, 64, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_cross_entropy_reports_an_infinite_loss(n, d, v, dtype):
    # A weight row of -inf against positive hidden states: that logit is
    # -inf, lse finite, and the loss +inf for the row whose target it is.
    dev = _dev()
    print(f"infinite loss n={n} d={d} v={v} {dtype}", flush=True)
    g = torch.Generator().manual_seed(n)
    h = (0.1 + torch.rand(n, d, generator=g)).to(DTYPES[dtype]).to(dev)
    w = (torch.randn(v, d, generator=g) / d).to(DTYPES[dtype]).to(dev)
    w[5] = -float("inf")
    t = torch.full((n,), 9, dtype=torch.int64, device=dev)
    st = _word(dev)
    loss, lse = nsa.linear_cross_entropy(h, w, t, status=st)
    assert torch.isfinite(loss).all() and torch.isfinite(lse).all() and int(st.item()) == 0
    t[n - 1] = 5
    loss, lse = nsa.linear_cross_entropy(h, w, t, status=st)
    assert torch.isfinite(lse).all() and torch.isfinite(loss[:n - 1]).all()
    assert float(loss[n - 1]) == float("inf") and int(st.item()) == BAD
    # An ignored row's loss is 0 whatever its logits, a bad target's NaN is
    # reported by its own bit alone.
    st.zero_()
    loss, lse = nsa.linear_cross_entropy(h, w, t, ignore_index=5, status=st)
    assert float(loss[n - 1]) == 0 and int(st.item()) == 0
    t[n - 1] = v
    loss, lse = nsa.linear_cross_entropy(h, w, t, status=st)
    assert torch.isnan(loss[n - 1]) and int(st.item()) == B.STATUS_BAD_INDEX


# ---------------------------------------------------------------------------
# Layer norm: a variance that fp32 does not hold.
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(3, 64), (5, 768), (4, 1001), (3, 4096), (2, 9000), (2, 20001), (2, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_layer_norm_reports_an_infinite_variance(rows, cols, dtype):
    # Deviations past 2^64 have infinite squares in fp32: rstd comes out as 0
    # and y as 0 (or the bias), finite and wrong, which the word says.
    dev = _dev()
    print(f"infinite variance {rows}x{cols} {dtype}", flush=True)
    x = torch.where(torch.arange(cols, device=dev) % 2 == 0, 1.0, -1.0).expand(rows, cols).contiguous()
    st = _word(dev)
    for size, reported in ((2.0 ** 55, False), (2.0 ** 66, True)):
        scaled = x.clone()
        scaled[rows - 1] *= size
        y, mean, rstd = nsa.layer_norm(scaled.to(DTYPES[dtype]), status=st)
        assert torch.isfinite(y).all() and torch.isfinite(rstd).all()
        assert (float(rstd[rows - 1]) == 0) == reported
        assert int(st.item()) == (BAD if reported else 0)
        st.zero_()
