"""Every kernel build of the training step's operators, run on the GPU and
checked against 64 bits (tests/training_cases.py; the host checks that the
cases reach all of them).  The bounds are those of test_gpu_training.py,
worked out element by element; the larger ones on the device.
"""

import pytest
import torch

import newton_schulz_matrix_amd as nsa

import test_gpu_training as base
from training_cases import XENT_RUNS, embed_widths, norm_widths

pytestmark = pytest.mark.gpu

U32 = base.U32


def _within(got, want, bound, what):
    worst = float(((got.double() - want).abs() / bound.clamp(min=1e-300)).max()) if got.numel() else 0.0
    print(f"{what}: worst error {worst:.3f} of the bound", flush=True)
    # NaN is no pass.
    assert worst <= 1, (what, worst)


def _check_on_device(h, w, t, dloss, dtype):
    """test_gpu_training._check_xent in torch's 64 bits (see there for each term)."""
    (n, d), v, dev = h.shape, w.shape[0], h.device
    st = base._word(dev)
    loss, lse = nsa.linear_cross_entropy(h, w, t, status=st)
    dh, dw = nsa.linear_cross_entropy_backward(h, w, t, lse, dloss, status=st, out_dh=base._poisoned(h.shape, h.dtype, dev),
                                               out_dw=base._poisoned(w.shape, w.dtype, dev))
    h64, w64, g = h.double(), w.double(), dloss.double().abs()
    u, tiny = base.HALF_STEP[dtype], base.TINY[dtype]
    z = h64 @ w64.t().contiguous()
    ez = (d + 1) * U32 * (h64.abs() @ w64.abs().t().contiguous())
    lse64 = torch.logsumexp(z, 1)
    elz = ez.amax(1) + U32 * (96 + v / 96 / 16 + 40 + 4 * z.abs().amax(1) + 2 * lse64.abs())
    _within(lse, lse64, elz, "lse")
    rows = torch.nonzero(t >= 0)[:, 0]
    loss64 = torch.zeros_like(lse64)
    loss64[rows] = (lse64 - z.gather(1, t.clamp(min=0)[:, None])[:, 0])[rows]
    _within(loss, loss64, (elz + ez.amax(1) + U32 * loss64.abs()) * (t >= 0), "loss")
    p = torch.exp(z - lse64[:, None])
    g = g * (t >= 0)
    # |dz| and its error, the target's entries apart.
    edz = p * (ez + (elz + 8 * U32)[:, None])
    edz[rows, t[rows]] += 2 * U32
    p[rows, t[rows]] -= 1
    edz += u * p.abs()
    if dtype == "fp16":
        edz += float(g.max()) * 2.0 ** -40 / g.clamp(min=1e-300)[:, None]
    edz *= g[:, None]
    p *= (dloss.double() * (t >= 0))[:, None]
    dh64, dw64 = p @ w64, p.t().contiguous() @ h64
    adz = p.abs() + edz
    eh = 1.05 * ((edz + U32 * (v + 20) * adz) @ w64.abs())
    ew = 1.05 * ((edz + U32 * (n + 20) * adz).t().contiguous() @ h64.abs())
    _within(dh, dh64, u * dh64.abs() + tiny + eh, "dh")
    _within(dw, dw64, u * dw64.abs() + tiny + ew, "dw")
    assert int(st.item()) == 0
    return loss, lse, dh, dw


@pytest.mark.parametrize("n,d,v,dtype", XENT_RUNS, ids=lambda x: str(x))
def test_every_cross_entropy_build(n, d, v, dtype):
    dev = base._dev()
    print(f"cross entropy n={n} d={d} v={v} {dtype}", flush=True)
    print("  ", *nsa.plan_linear_cross_entropy(n, d, v, base.DTYPES[dtype]),
          *nsa.plan_linear_cross_entropy(n, d, v, base.DTYPES[dtype], backward=True), flush=True)
    h, w, t, dloss = base._xent_inputs(n, d, v, dtype, dev, seed=n + d + v)
    first = _check_on_device(h, w, t, dloss, dtype)
    # Again: the same bits.
    loss, lse = nsa.linear_cross_entropy(h, w, t)
    for a, b in zip(first, (loss, lse) + nsa.linear_cross_entropy_backward(h, w, t, lse, dloss)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_cross_entropy_gradients_without_rows(dtype):
    dev = base._dev()
    for d in (64, 77, 1):
        w = torch.ones(500, d, dtype=base.DTYPES[dtype], device=dev)
        h, t = w[:0], torch.zeros(0, dtype=torch.int64, device=dev)
        lse = torch.zeros(0, device=dev)
        dh, dw = nsa.linear_cross_entropy_backward(h, w, t, lse, lse, out_dw=base._poisoned(w.shape, w.dtype, dev))
        assert dh.shape == (0, d) and torch.equal(dw, torch.zeros_like(w))


@pytest.mark.parametrize("dtype,pdtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"),
                                          ("fp32", "fp32")])
def test_every_layer_norm_width(dtype, pdtype):
    # Nine rows: more than one block, the last one not full, where rows share a block.
    for cols in norm_widths(base.DTYPES[dtype].itemsize):
        base.test_layer_norm_matches_the_oracle(9, cols, dtype, pdtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_every_embedding_width(dtype):
    for i, cols in enumerate(embed_widths(base.DTYPES[dtype].itemsize)):
        base.test_embedding_and_its_gradient(200, 70, cols, dtype, bool(i % 2))
