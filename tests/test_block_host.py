"""AdamW, residual norms and the gated feed-forward block without a device:
the oracle's pins, the workspace queries and every refusal of the C entry
points (made on the host before anything is enqueued; no device pointer is
dereferenced)."""

import ctypes
import os

import numpy as np
import pytest
import torch

import oracle
import newton_schulz_matrix_amd as nsa
from newton_schulz_matrix_amd import _binding as B
from newton_schulz_matrix_amd import _block

built = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libnsortho.so not built")

INV, DT, WSP = 1, 2, 3
PTR = 1 << 20  # stands for a device pointer


# ---------------------------------------------------------------------------
# AdamW.
# ---------------------------------------------------------------------------

def test_oracle_adamw_against_closed_forms():
    g, p = np.array([0.5, -2.0, 0.0]), np.array([1.0, 1.0, 1.0])
    m = v = np.zeros(3)
    q = p
    for t in range(1, 6):
        before = q
        q, m, v = oracle.adamw(q, g, m, v, 0.01, t, (0.9, 0.99), 1e-30, 0.0)
        # A constant gradient: the corrected moments are g and g^2.
        assert np.allclose(m, (1 - 0.9 ** t) * g) and np.allclose(v, (1 - 0.99 ** t) * g * g)
        assert np.allclose(q, before - 0.01 * np.sign(g))
    q, _, _ = oracle.adamw(p, 0 * g, 0 * p, 0 * p, 0.01, 1, weight_decay=0.5)
    assert np.allclose(q, p * (1 - 0.005))
    q, m, v = oracle.adamw(p, 4 * g, 0 * p, 0 * p, 0.01, 1, grad_scale=0.25)
    assert np.allclose(m, 0.1 * g) and np.allclose(v, 0.05 * g * g)


def _adamw(beta1=0.9, beta2=0.95, eps=1e-8, step=1, d_step=None, count=1, table=True, **kw):
    e = dict(param=PTR, grad=PTR, m=PTR, v=PTR, scales=0, copy=0, numel=10, lr=1e-3, wd=0.1, pt=0, gt=0, ct=0, zero=0)
    e.update(kw)
    raw = bytearray(_block._TENSOR.pack(*(e[k] or 0 for k in ("param", "grad", "m", "v", "scales", "copy", "numel", "lr",
                                                              "wd", "pt", "gt", "ct", "zero"))))
    arr = (ctypes.c_char * len(raw)).from_buffer(raw) if table else None
    return B.lib().ns_adamw_step(arr, count, beta1, beta2, eps, step, d_step, None, None, None, None)


@built
def test_adamw_refusals():
    for name in ("param", "grad", "m", "v"):
        assert _adamw(**{name: None}) == INV, name
    for kw in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=-1e-9),
               dict(eps=float("inf")), dict(step=0), dict(step=-3), dict(count=-1), dict(table=False), dict(numel=-1),
               dict(numel=(1 << 40) + 1), dict(lr=float("nan")), dict(wd=float("inf")), dict(zero=1)):
        assert _adamw(**kw) == INV, kw
    assert _adamw(pt=3) == DT and _adamw(gt=7) == DT and _adamw(copy=PTR, ct=3) == DT
    # Nothing to do: no launch.
    assert _adamw(count=0, table=False) == 0
    assert _adamw(numel=0, param=None, grad=None, m=None, v=None) == 0


@built
def test_adamw_table_entry_has_the_headers_layout():
    text = open(os.path.join(os.path.dirname(B.PKG), "include", "nsortho.h")).read()
    body = text[text.index("typedef struct ns_adamw_tensor {"):text.index("} ns_adamw_tensor;")]
    names = [line.split()[-1].rstrip(";").lstrip("*") for line in body.splitlines()[1:] if line.strip()]
    assert names == ["param", "grad", "exp_avg", "exp_avg_sq", "scales", "copy", "numel", "lr", "weight_decay",
                     "param_dtype", "grad_dtype", "copy_dtype", "reserved"]
    assert _block._TENSOR.size == 6 * 8 + 8 + 2 * 4 + 4 * 4


def test_adamw_states_and_host_tensors():
    p = [torch.zeros(3, 100), torch.zeros(0), torch.zeros(1)]
    m, v, scales = nsa.adamw_states(p)
    assert scales is None and all(t.dtype == torch.float32 and t.shape == q.shape for t, q in zip(m + v, p + p))
    m, v, scales = nsa.adamw_states(p, bits=8)
    assert [tuple(s.shape) for s in scales] == [(2, 2), (2, 0), (2, 1)]
    assert all(t.dtype == torch.float8_e4m3fn for t in m + v)
    with pytest.raises(ValueError, match="device tensor"):
        nsa.adamw_step(p, p, m, v, lr=1e-3, step=1, scales=scales)


# ---------------------------------------------------------------------------
# Norms before and after a block.
# ---------------------------------------------------------------------------

def _slope(f, x, direction, step=1e-5):
    return (f(x + step * direction) - f(x - step * direction)) / (2 * step)


@pytest.mark.parametrize("norm_branch", [True, False])
@pytest.mark.parametrize("groups", [None, 1, 3, 6])
def test_oracle_residual_norm_gradients_against_differences(norm_branch, groups):
    rng = np.random.default_rng(5)
    x, z = rng.normal(size=(6, 9)), rng.normal(size=(6, 9))
    gate = None if groups is None else rng.normal(size=(groups, 9))
    wb, w = rng.normal(size=9), rng.normal(size=9)
    ds, dy = rng.normal(size=(6, 9)), rng.normal(size=(6, 9))
    s, y, rb, rs = oracle.residual_norm(x, z, eps=0.0)
    assert np.allclose((y * y).mean(1), 1) and np.allclose(((z * rb[:, None]) ** 2).mean(1), 1)

    def value(x=x, z=z, gate=gate, wb=wb, w=w):
        s, y, _, _ = oracle.residual_norm(x, z, gate, 0.7, wb, w, norm_branch)
        return (ds * s).sum() + (dy * y).sum()

    s, y, rb, rs = oracle.residual_norm(x, z, gate, 0.7, wb, w, norm_branch)
    o = oracle.residual_norm_backward(ds, dy, s, z, rb if norm_branch else None, rs, gate, 0.7, wb, w)
    for name, at, grad in (("x", x, o["dx"]), ("z", z, o["dz"]), ("wb", wb, o["dwb"]), ("w", w, o["dw"])):
        d = rng.normal(size=at.shape)
        assert _slope(lambda v: value(**{name: v}), at, d) == pytest.approx((grad * d).sum(), rel=1e-6), name
    if groups is not None:
        d = rng.normal(size=gate.shape)
        dgate = o["dgate"].reshape(groups, -1, 9).sum(1)
        assert _slope(lambda v: value(gate=v), gate, d) == pytest.approx((dgate * d).sum(), rel=1e-6)


def test_oracle_residual_norm_without_a_branch():
    rng = np.random.default_rng(6)
    x, w, dy = rng.normal(size=(4, 5)), rng.normal(size=5), rng.normal(size=(4, 5))
    s, y, _, rs = oracle.residual_norm(x, None, weight=w)
    o = oracle.residual_norm_backward(None, dy, s, None, None, rs, weight=w)
    d = rng.normal(size=x.shape)
    slope = _slope(lambda v: (dy * oracle.residual_norm(v, None, weight=w)[1]).sum(), x, d)
    assert slope == pytest.approx((o["dx"] * d).sum(), rel=1e-6)


def _norm(X=PTR, ldx=8, Z=PTR, ldz=8, rows=4, cols=8, dtype=B.NS_BF16, gate=PTR, groups=2, wb=PTR, w=PTR, pt=B.NS_FP32,
          scale=1.0, nb=1, eps=1e-6, S=PTR, lds=8, Y=PTR, ldy=8):
    return B.lib().ns_residual_norm(X, ldx, Z, ldz, rows, cols, dtype, gate, groups, wb, w, pt, scale, nb, eps, S, lds,
                                    Y, ldy, None, None, None, None)


@built
def test_residual_norm_refusals():
    for kw in (dict(X=None), dict(S=None), dict(ldx=7), dict(ldz=7), dict(lds=7), dict(ldy=7), dict(rows=-1),
               dict(rows=1 << 31, groups=1), dict(cols=0), dict(cols=(1 << 24) + 1, ldx=1 << 25, ldz=1 << 25, lds=1 << 25, ldy=1 << 25),
               dict(groups=0), dict(groups=3), dict(groups=8), dict(groups=-1), dict(scale=float("nan")), dict(nb=2),
               dict(eps=-1.0), dict(eps=float("inf")), dict(Z=None), dict(Z=None, gate=None, wb=None),
               dict(Z=None, gate=None, wb=None, S=None, scale=0.5), dict(Z=None, gate=None, wb=None, S=None, Y=None)):
        assert _norm(**kw) == INV, kw
    assert _norm(dtype=5) == DT and _norm(pt=B.NS_FP16) == DT
    assert _norm(rows=0, X=None, Z=PTR, S=None, Y=None) == 0


def _norm_back(dS=PTR, ldds=8, dY=PTR, lddy=8, S=PTR, lds=8, Z=PTR, ldz=8, rows=4, cols=8, dtype=B.NS_BF16, rb=PTR,
               rs=PTR, gate=PTR, groups=2, wb=PTR, w=PTR, pt=B.NS_FP32, scale=1.0, dX=PTR, lddx=8, dZ=PTR, lddz=8,
               dg=PTR, dwb=PTR, dw=PTR, ws=256, n=1 << 30):
    return B.lib().ns_residual_norm_backward(dS, ldds, dY, lddy, S, lds, Z, ldz, rows, cols, dtype, rb, rs, gate, groups,
                                             wb, w, pt, scale, dX, lddx, dZ, lddz, dg, dwb, dw, None, ws, n, None)


@built
def test_residual_norm_backward_refusals():
    for kw in (dict(dS=None, dY=None), dict(S=None), dict(rs=None), dict(dZ=None), dict(dY=None), dict(dY=None, w=None),
               dict(ldds=7), dict(lddy=7), dict(lds=7), dict(ldz=7), dict(lddx=7), dict(lddz=7), dict(groups=0),
               dict(groups=3), dict(gate=None, groups=0), dict(rows=-1), dict(cols=0), dict(scale=float("inf")),
               dict(Z=None), dict(Z=None, gate=None, dg=None, wb=None, dwb=None),
               dict(Z=None, gate=None, dg=None, wb=None, dwb=None, dZ=None, scale=0.5),
               dict(Z=None, gate=None, dg=None, wb=None, dwb=None, dZ=None, dX=None),
               dict(rows=0, groups=1 << 40)):
        assert _norm_back(**kw) == INV, kw
    assert _norm_back(dtype=5) == DT and _norm_back(pt=B.NS_FP16) == DT
    assert _norm_back(ws=None) == WSP and _norm_back(ws=100) == WSP and _norm_back(n=100) == WSP
    assert nsa.residual_norm_workspace_size(0, 8) >= 256 and nsa.residual_norm_workspace_size(-1, 8) == 0
    assert nsa.residual_norm_workspace_size(4, 0) == 0
    # No rows and nothing wanted.
    assert _norm_back(rows=0, dg=None, dwb=None, dw=None) == 0
