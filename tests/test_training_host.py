"""Embedding, layer norm and cross entropy without a device: the oracle's
pins, the workspace queries and every refusal of the C entry points (made on
the host before anything is enqueued; no pointer is dereferenced)."""

import ctypes
import os

import numpy as np
import pytest
import torch

import oracle
import newton_schulz_matrix_amd as nsa
from newton_schulz_matrix_amd import _binding as B

built = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libnsortho.so not built")

INV, DT, WSP = 1, 2, 3
PTR = 1 << 20  # stands for a device pointer


# ---------------------------------------------------------------------------
# The oracle.
# ---------------------------------------------------------------------------

def _slope(f, x, direction, step=1e-5):
    return (f(x + step * direction) - f(x - step * direction)) / (2 * step)


def test_oracle_layer_norm_gradients_against_differences():
    rng = np.random.default_rng(0)
    x, w, b = rng.normal(size=(5, 7)), rng.normal(size=7), rng.normal(size=7)
    dy = rng.normal(size=(5, 7))
    y, mean, rstd = oracle.layer_norm(x, eps=0.0)
    assert np.allclose(y.mean(1), 0) and np.allclose((y * y).mean(1), 1)
    _, mean, rstd = oracle.layer_norm(x, w, b)
    dx, dw, db = oracle.layer_norm_backward(dy, x, mean, rstd, w)
    for _ in range(3):
        d = rng.normal(size=x.shape)
        assert _slope(lambda v: (dy * oracle.layer_norm(v, w, b)[0]).sum(), x, d) == pytest.approx((dx * d).sum(), rel=1e-6)
        d = rng.normal(size=7)
        assert _slope(lambda v: (dy * oracle.layer_norm(x, v, b)[0]).sum(), w, d) == pytest.approx((dw * d).sum(), rel=1e-6)
        assert _slope(lambda v: (dy * oracle.layer_norm(x, w, v)[0]).sum(), b, d) == pytest.approx((db * d).sum(), rel=1e-6)


def test_oracle_embedding_gradient_against_differences():
    rng = np.random.default_rng(1)
    ids = np.array([3, 0, 3, 9, -1, 3, 4])
    table, dy = rng.normal(size=(6, 4)), rng.normal(size=(7, 4))
    onehot = np.array([[1.0 if i == v else 0.0 for v in range(6)] for i in ids])
    assert np.allclose(oracle.embedding(ids, table, 1.5), 1.5 * onehot @ table)
    dt = oracle.embedding_backward(ids, dy, 6, 1.5)
    d = rng.normal(size=table.shape)
    assert _slope(lambda v: (dy * oracle.embedding(ids, v, 1.5)).sum(), table, d) == pytest.approx((dt * d).sum(), rel=1e-6)


def test_oracle_cross_entropy_gradients_against_differences():
    rng = np.random.default_rng(2)
    h, w = rng.normal(size=(6, 5)), rng.normal(size=(9, 5))
    t, g = np.array([0, 8, -100, 4, 4, 2]), rng.normal(size=6)
    loss, lse = oracle.linear_cross_entropy(h, w, t)
    assert np.allclose(lse, np.log(np.exp(h @ w.T).sum(1)))
    assert loss[2] == 0 and np.allclose(loss[[0, 1]], lse[[0, 1]] - (h @ w.T)[[0, 1], [0, 8]])
    assert np.isnan(oracle.linear_cross_entropy(h, w, np.full(6, 9))[0]).all()
    dh, dw = oracle.linear_cross_entropy_backward(h, w, t, g)
    for _ in range(3):
        d = rng.normal(size=h.shape)
        assert _slope(lambda v: (g * oracle.linear_cross_entropy(v, w, t)[0]).sum(), h, d) == pytest.approx((dh * d).sum(), rel=1e-6)
        d = rng.normal(size=w.shape)
        assert _slope(lambda v: (g * oracle.linear_cross_entropy(h, v, t)[0]).sum(), w, d) == pytest.approx((dw * d).sum(), rel=1e-6)


# ---------------------------------------------------------------------------
# Workspace queries.
# ---------------------------------------------------------------------------

@built
def test_workspace_sizes():
    # Refused shapes.
    assert nsa.layer_norm_workspace_size(-1, 8) == 0
    assert nsa.layer_norm_workspace_size(8, 0) == 0
    assert nsa.layer_norm_workspace_size(1 << 31, 8) == 0
    assert nsa.embedding_workspace_size(-1, 8, 8) == 0
    assert nsa.embedding_workspace_size(8, 0, 8) == 0
    assert nsa.embedding_workspace_size((1 << 30) + 1, 8, 8) == 0
    assert nsa.embedding_workspace_size(1 << 30, 8, 8) > 0
    # The sort reads all ids once per 512 table rows.
    assert nsa.embedding_workspace_size(1 << 30, 1 << 16, 8) > 0
    assert nsa.embedding_workspace_size(1 << 30, (1 << 16) + 1, 8) == 0
    assert nsa.linear_cross_entropy_workspace_size(1 << 22, 8, 1 << 21) == 0
    assert nsa.linear_cross_entropy_workspace_size(8, 8, 0) == 0
    assert nsa.linear_cross_entropy_workspace_size((1 << 23) + 1, 8, 8) == 0
    assert nsa.linear_cross_entropy_workspace_size(8, (1 << 20) + 1, 8) == 0
    assert B.lib().ns_linear_cross_entropy_workspace_size(8, 8, 8, 7, 1, 0) == 0
    # Empty inputs still have one (not 0, which means refused).
    assert nsa.layer_norm_workspace_size(0, 5) > 0
    assert nsa.embedding_workspace_size(0, 5, 5) > 0
    for backward in (False, True):
        assert nsa.linear_cross_entropy_workspace_size(0, 64, 100, backward=backward) > 0
    # Layer norm: at most 512 partial rows, whatever the number of rows.
    assert nsa.layer_norm_workspace_size(1 << 20, 4096) == 512 * 2 * 4096 * 4
    # The logits are not kept: forward needs a few bytes per row and 192
    # columns, backward holds one piece of at most 2^28 elements in two
    # orientations plus H^T, one piece of W^T and dH in fp32.
    logits = 8192 * 128000 * 2
    assert nsa.linear_cross_entropy_workspace_size(8192, 4096, 128000) < logits / 15
    for n in (8192, 65536):
        back = nsa.linear_cross_entropy_workspace_size(n, 4096, 128000, backward=True)
        h = (n + 192) * 4224
        assert back < 2 * 2 ** 28 * 2 + 128000 * 4224 * 2 + h * 2 + 8 * h * 4
    # Operands that are not aligned, or rows that are not whole k-tiles, are copied.
    plain = nsa.linear_cross_entropy_workspace_size(300, 1024, 5000)
    copied = nsa.linear_cross_entropy_workspace_size(300, 1024, 5000, aligned=False)
    assert copied - plain == pytest.approx((300 + 5000) * 1024 * 2, abs=1024)
    assert nsa.linear_cross_entropy_workspace_size(300, 1000, 5000) == copied


# ---------------------------------------------------------------------------
# Refusals.
# ---------------------------------------------------------------------------

def _norm(X=PTR, rows=4, cols=8, ldx=8, dtype=B.NS_BF16, W=PTR, Bi=PTR, pdt=B.NS_BF16, eps=1e-5, Y=PTR, ldy=8):
    return B.lib().ns_layer_norm(X, rows, cols, ldx, dtype, W, Bi, pdt, eps, Y, ldy, None, None, None, None)


@built
def test_layer_norm_refusals():
    assert _norm(X=None) == INV and _norm(Y=None) == INV
    assert _norm(rows=-1) == INV and _norm(cols=0) == INV and _norm(cols=(1 << 24) + 1, ldx=1 << 25, ldy=1 << 25) == INV
    assert _norm(rows=1 << 31) == INV
    assert _norm(ldx=7) == INV and _norm(ldy=7) == INV
    assert _norm(eps=-1.0) == INV and _norm(eps=float("nan")) == INV and _norm(eps=float("inf")) == INV
    assert _norm(dtype=3) == DT
    assert _norm(pdt=B.NS_FP16) == DT                       # neither the data's type nor fp32
    assert _norm(dtype=B.NS_FP32, pdt=B.NS_BF16) == DT
    assert _norm(rows=0, X=None, Y=None) == 0               # nothing to do


def _norm_back(dY=PTR, lddy=8, X=PTR, ldx=8, rows=4, cols=8, dtype=B.NS_BF16, mean=PTR, rstd=PTR, pdt=B.NS_BF16,
               dX=PTR, lddx=8, dw=PTR, db=PTR, ws=256, n=1 << 30):
    return B.lib().ns_layer_norm_backward(dY, lddy, X, ldx, rows, cols, dtype, mean, rstd, None, pdt, dX, lddx, dw, db,
                                          None, ws, n, None)


@built
def test_layer_norm_backward_refusals():
    for name in ("dY", "X", "mean", "rstd", "dX"):
        assert _norm_back(**{name: None}) == INV, name
    for name in ("lddy", "ldx", "lddx"):
        assert _norm_back(**{name: 7}) == INV, name
    assert _norm_back(dtype=4) == DT and _norm_back(pdt=B.NS_FP16) == DT
    assert _norm_back(ws=None) == WSP and _norm_back(ws=128) == WSP and _norm_back(n=8) == WSP
    # No rows and no parameter gradients: nothing to do, no workspace needed.
    assert _norm_back(rows=0, dw=None, db=None, ws=None, n=0) == 0


def _embed(ids=PTR, ids64=1, n=4, T=PTR, vocab=10, cols=8, ldt=8, dtype=B.NS_BF16, scale=1.0, out=PTR, ldo=8):
    return B.lib().ns_embedding(ids, ids64, n, T, vocab, cols, ldt, dtype, scale, out, ldo, None, None)


@built
def test_embedding_refusals():
    assert _embed(ids=None) == INV and _embed(T=None) == INV and _embed(out=None) == INV
    assert _embed(ids64=2) == INV and _embed(n=-1) == INV and _embed(vocab=0) == INV and _embed(cols=0) == INV
    assert _embed(cols=(1 << 23) + 1, ldt=1 << 24, ldo=1 << 24) == INV
    assert _embed(vocab=(1 << 28) + 1) == INV and _embed(n=(1 << 30) + 1) == INV
    assert _embed(ldt=7) == INV and _embed(ldo=7) == INV
    assert _embed(scale=float("nan")) == INV and _embed(scale=float("inf")) == INV
    assert _embed(dtype=9) == DT
    assert _embed(n=0, ids=None, T=None, out=None) == 0


def _embed_back(ids=PTR, ids64=1, n=4, dY=PTR, lddy=8, vocab=10, cols=8, dtype=B.NS_BF16, scale=1.0, dT=PTR, ldt=8,
                acc=0, ws=256, nb=1 << 30):
    return B.lib().ns_embedding_backward(ids, ids64, n, dY, lddy, vocab, cols, dtype, scale, dT, ldt, acc, None, ws, nb,
                                         None)


@built
def test_embedding_backward_refusals():
    assert _embed_back(ids=None) == INV and _embed_back(dY=None) == INV and _embed_back(dT=None) == INV
    assert _embed_back(ids64=-1) == INV and _embed_back(acc=2) == INV
    assert _embed_back(lddy=7) == INV and _embed_back(ldt=7) == INV and _embed_back(scale=float("nan")) == INV
    assert _embed_back(dtype=9) == DT
    assert _embed_back(ws=None) == WSP and _embed_back(ws=100) == WSP and _embed_back(nb=16) == WSP


def _xent(H=PTR, ldh=64, W=PTR, ldw=64, t=PTR, t64=1, rows=4, cols=64, vocab=10, dtype=B.NS_BF16, loss=PTR, lse=PTR,
          ws=256, nb=1 << 40):
    return B.lib().ns_linear_cross_entropy(H, ldh, W, ldw, t, t64, rows, cols, vocab, dtype, -100, loss, lse, None, ws,
                                           nb, None)


@built
def test_cross_entropy_refusals():
    for name in ("H", "W", "t", "loss", "lse"):
        assert _xent(**{name: None}) == INV, name
    assert _xent(ldh=63) == INV and _xent(ldw=63) == INV and _xent(ldw=(1 << 23) + 1) == INV
    assert _xent(t64=3) == INV and _xent(rows=-1) == INV and _xent(cols=0) == INV and _xent(vocab=0) == INV
    assert _xent(vocab=(1 << 23) + 1) == INV and _xent(dtype=5) == DT
    assert _xent(ws=None) == WSP and _xent(ws=64) == WSP and _xent(nb=16) == WSP
    # A misaligned operand needs the copies' workspace too.
    need = nsa.linear_cross_entropy_workspace_size(40, 64, 10, aligned=True)
    assert _xent(rows=40, H=PTR + 2, nb=need) == WSP
    assert _xent(rows=0, H=None, W=None, t=None, loss=None, lse=None, ws=None, nb=0) == 0


def _xent_back(H=PTR, ldh=64, W=PTR, ldw=64, t=PTR, t64=1, rows=4, cols=64, vocab=10, dtype=B.NS_BF16, lse=PTR, g=PTR,
               dH=PTR, lddh=64, dW=PTR, lddw=64, ws=256, nb=1 << 40):
    return B.lib().ns_linear_cross_entropy_backward(H, ldh, W, ldw, t, t64, rows, cols, vocab, dtype, -100, lse, g, dH,
                                                    lddh, dW, lddw, None, ws, nb, None)


@built
def test_cross_entropy_backward_refusals():
    for name in ("H", "W", "t", "lse", "g"):
        assert _xent_back(**{name: None}) == INV, name
    for name in ("ldh", "ldw", "lddh", "lddw"):
        assert _xent_back(**{name: 63}) == INV, name
    assert _xent_back(t64=3) == INV and _xent_back(dtype=5) == DT and _xent_back(cols=(1 << 20) + 1, ldh=1 << 21, ldw=1 << 21) == INV
    assert _xent_back(ws=None) == WSP and _xent_back(ws=64) == WSP and _xent_back(nb=16) == WSP
    # Nothing wanted, nothing enqueued.
    assert _xent_back(dH=None, dW=None) == 0
    assert _xent_back(rows=0, dW=None, H=None, lse=None, ws=None, nb=0) == 0


@built
def test_python_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 8)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: nsa.layer_norm(x), lambda: nsa.layer_norm_backward(x, x, x[:, 0], x[:, 0]),
                 lambda: nsa.embedding(ids, x), lambda: nsa.embedding_backward(ids, x, 5),
                 lambda: nsa.linear_cross_entropy(x, x, ids),
                 lambda: nsa.linear_cross_entropy_backward(x, x, ids, x[:, 0], 1.0)):
        with pytest.raises(ValueError, match="device tensor"):
            call()


@built
def test_bad_index_bit_is_outside_the_code_and_the_other_bits():
    text = open(os.path.join(os.path.dirname(B.PKG), "include", "nsortho.h")).read()
    assert "#define NS_STATUS_BAD_INDEX (1 << 13)" in text and B.STATUS_BAD_INDEX == 1 << 13
    assert nsa.status_code(B.STATUS_BAD_INDEX) == 0
    others = (B.STATUS_AT_INPUT, B.STATUS_AT_STATE, B.STATUS_AT_ITERATE, B.STATUS_AT_OUTPUT, B.STATUS_AT_SPLIT,
              B.STATUS_GUARD_RESTART)
    assert all(B.STATUS_BAD_INDEX & o == 0 for o in others)
