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
