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
