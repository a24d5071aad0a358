"""The rest of a block's training step in fp64: AdamW, norms, feed-forward.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The formulas are the definitions; gradients are written out by hand and
pinned against finite differences of the forward functions.
"""

from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def adamw(p, g, m, v, lr, step, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, grad_scale=1.0):
    """(p, m, v) after one step."""
    p, g = _f64(p), _f64(g) * grad_scale
    m = betas[0] * _f64(m) + (1 - betas[0]) * g
    v = betas[1] * _f64(v) + (1 - betas[1]) * g * g
    root = np.sqrt(v / (1 - betas[1] ** step))
    p = p - lr * weight_decay * p - lr * (m / (1 - betas[0] ** step)) / (root + eps)
    return p, m, v


def state_tops(x, block=256, least=2.0 ** -100):
    """The largest magnitude of each block of an 8-bit moment."""
    x = np.abs(_f64(x).reshape(-1))
    padded = np.pad(x, (0, -x.size % block)).reshape(-1, block)
    return np.maximum(padded.max(1), least)


def _gate_of_rows(gate, rows, cols):
    """The gate's row of every data row (ones without a gate)."""
    if gate is None:
        return np.ones((rows, cols))
    gate = _f64(gate).reshape(-1, cols)
    return np.repeat(gate, rows // gate.shape[0], 0)


def residual_norm(x, z, gate=None, scale=1.0, branch_weight=None, weight=None, norm_branch=True, eps=1e-6):
    """(s, y, rb, rs) for 2-D x and z (z None: the norm of x alone)."""
    x = _f64(x)
    rows, cols = x.shape
    w = np.ones(cols) if weight is None else _f64(weight)
    wb = np.ones(cols) if branch_weight is None else _f64(branch_weight)
    rb = np.ones(rows)
    s = x
    if z is not None:
        z = _f64(z)
        if norm_branch:
            rb = 1.0 / np.sqrt(np.mean(z * z, 1) + eps)
        s = scale * x + _gate_of_rows(gate, rows, cols) * (z * rb[:, None] * wb)
    rs = 1.0 / np.sqrt(np.mean(s * s, 1) + eps)
    return s, s * rs[:, None] * w, rb, rs


def residual_norm_backward(ds, dy, s, z, rb=None, rs=None, gate=None, scale=1.0, branch_weight=None, weight=None):
    """A dict of the gradients and of the G they come from, given the statistics.

    rb None: the branch was not normed.  dgate has one row per row of the data;
    the caller sums over those that share a row of the gate.
    """
    some = ds if ds is not None else dy
    rows, cols = some.shape
    w = np.ones(cols) if weight is None else _f64(weight)
    wb = np.ones(cols) if branch_weight is None else _f64(branch_weight)
    g = np.zeros((rows, cols)) if ds is None else _f64(ds)
    out = {}
    if dy is not None:
        rs = _f64(rs)[:, None]
        shat, u = _f64(s) * rs, _f64(dy) * w
        g = g + rs * (u - shat * np.mean(u * shat, 1, keepdims=True))
        out["dw"] = (_f64(dy) * shat).sum(0)
    out.update(g=g, dx=scale * g)
    if z is not None:
        r = np.ones((rows, 1)) if rb is None else _f64(rb)[:, None]
        bhat = _f64(z) * r
        q = _gate_of_rows(gate, rows, cols) * g
        a = wb * q
        out["dz"] = a if rb is None else r * (a - bhat * np.mean(a * bhat, 1, keepdims=True))
        out["dgate"] = g * bhat * wb
        out["dwb"] = (q * bhat).sum(0)
    return out


_C, _K = np.sqrt(2.0 / np.pi), 0.044715


def activation(a, name):
    """(value, slope) of an activation."""
    from math import erf

    a = _f64(a)
    if name == "relu":
        return np.maximum(a, 0.0), (a > 0) * 1.0
    if name == "gelu":
        phi = 0.5 * (1.0 + np.vectorize(erf, otypes=[float])(a / np.sqrt(2.0)))
        return a * phi, phi + a * np.exp(-0.5 * a * a) / np.sqrt(2.0 * np.pi)
    if name == "gelu_tanh":
        t = np.tanh(_C * (a + _K * a ** 3))
        return 0.5 * a * (1 + t), 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * _C * (1 + 3 * _K * a * a)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-a))
    return a * s, s * (1.0 + a * (1.0 - s))


def gated_mlp(x, w_gate, w_up, w_down, act="silu"):
    """(y, a, b, h) of a gated feed-forward block."""
    x = _f64(x)
    a, b = x @ _f64(w_gate).T, x @ _f64(w_up).T
    h = activation(a, act)[0] * b
    return h @ _f64(w_down).T, a, b, h


def gated_mlp_backward(dy, x, w_gate, w_up, w_down, a, b, act="silu"):
    """A dict of the gradients (dx, dwg, dwu, dwd) and of what they are made of (dh, da, db, h), given a and b."""
    dy, x, a, b = _f64(dy), _f64(x), _f64(a), _f64(b)
    value, slope = activation(a, act)
    dh = dy @ _f64(w_down)
    da, db, h = dh * b * slope, dh * value, value * b
    return {"dx": da @ _f64(w_gate) + db @ _f64(w_up), "dwg": da.T @ x, "dwu": db.T @ x, "dwd": dy.T @ h,
            "dh": dh, "da": da, "db": db, "h": h}
