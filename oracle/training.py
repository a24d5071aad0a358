"""The two ends of a training step in fp64: embedding, layer norm, cross entropy.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The formulas are the definitions; gradients are written out by hand and
pinned against finite differences of the forward functions.
"""

from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) over the last axis."""
    x = _f64(x)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(np.mean((x - mean[..., None]) ** 2, -1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    if weight is not None:
        y = y * _f64(weight)
    if bias is not None:
        y = y + _f64(bias)
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None):
    """(dx, dweight, dbias) of 2-D x, given its statistics."""
    dy, x, mean, rstd = _f64(dy), _f64(x), _f64(mean)[:, None], _f64(rstd)[:, None]
    xhat = (x - mean) * rstd
    a = dy if weight is None else dy * _f64(weight)
    dx = rstd * (a - a.mean(1, keepdims=True) - xhat * (a * xhat).mean(1, keepdims=True))
    return dx, (dy * xhat).sum(0), dy.sum(0)


def embedding(ids, table, scale=1.0):
    """scale * table[ids]; ids outside the table give zeros."""
    ids, table = np.asarray(ids), _f64(table)
    ok = (ids >= 0) & (ids < table.shape[0])
    return np.where(ok[..., None], scale * table[np.where(ok, ids, 0)], 0.0)


def embedding_backward(ids, dy, vocab, scale=1.0):
    """The table's gradient: scale times dy's rows summed by id."""
    ids, dy = np.asarray(ids).reshape(-1), _f64(dy)
    dy = dy.reshape(ids.size, -1)
    ok = (ids >= 0) & (ids < vocab)
    out = np.zeros((vocab, dy.shape[1]))
    np.add.at(out, ids[ok], dy[ok])
    return scale * out


def linear_cross_entropy(h, w, targets, ignore_index=-100):
    """(loss, lse) per row of softmax cross entropy on the logits h w^T."""
    z, t = _f64(h) @ _f64(w).T, np.asarray(targets).reshape(-1)
    top = z.max(1)
    top = np.where(np.isfinite(top), top, 0.0)
    with np.errstate(divide="ignore"):
        lse = top + np.log(np.exp(z - top[:, None]).sum(1))
    ok = (t >= 0) & (t < z.shape[1]) & (t != ignore_index)
    loss = np.where(ok, lse - z[np.arange(len(t)), np.where(ok, t, 0)],
                    np.where(t == ignore_index, 0.0, np.nan))
    return loss, lse


def linear_cross_entropy_dz(h, w, targets, dloss, ignore_index=-100):
    """dloss_i (softmax(z)_ij - [j == targets_i]); rows without a target are 0."""
    z, t = _f64(h) @ _f64(w).T, np.asarray(targets).reshape(-1)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    ok = (t >= 0) & (t < z.shape[1]) & (t != ignore_index)
    p[np.nonzero(ok)[0], t[ok]] -= 1.0
    return p * np.where(ok, _f64(dloss), 0.0)[:, None]


def linear_cross_entropy_backward(h, w, targets, dloss, ignore_index=-100):
    """(dh, dw)."""
    dz = linear_cross_entropy_dz(h, w, targets, dloss, ignore_index)
    return dz @ _f64(w), dz.T @ _f64(h)
