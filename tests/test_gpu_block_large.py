"""AdamW, residual norms and the gated feed-forward block on tensors of more
than 2^31 elements: what lies past 32-bit offsets is as right as the rest.
"""

import numpy as np
import pytest
import torch

import oracle
import newton_schulz_matrix_amd as nsa

import test_gpu_gated_mlp as mlp
from test_gpu_training_large import CHUNK, COLS, ROWS, _chunks, _random

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
HALF = 2.0 ** -8


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_past_32_bits(bits):
    dev = mlp._dev()
    p, g = _random(ROWS, COLS, dev, 1), _random(ROWS, COLS, dev, 2)
    m, v, s = nsa.adamw_states([p], bits)
    kw = dict(lr=1e-2, weight_decay=0.1)
    start = [p[c].clone() for c in (slice(0, CHUNK), slice(ROWS - CHUNK, ROWS))]
    nsa.adamw_step([p], [g], m, v, step=1, scales=s, **kw)
    # An element's result (8-bit: a block's) does not depend on the rest.
    for c, q in zip((slice(0, CHUNK), slice(ROWS - CHUNK, ROWS)), start):
        cm, cv, cs = nsa.adamw_states([q], bits)
        nsa.adamw_step([q], [g[c]], cm, cv, step=1, scales=cs, **kw)
        assert torch.equal(p[c], q)
        assert torch.equal(m[0][c].view(torch.uint8), cm[0].view(torch.uint8))
        assert torch.equal(v[0][c].view(torch.uint8), cv[0].view(torch.uint8))
        if bits == 8:
            blocks = slice(c.start * COLS // 256, c.stop * COLS // 256)
            assert torch.equal(s[0][:, blocks], cs[0])


def test_residual_norm_past_32_bits():
    dev = mlp._dev()
    x, z, ds, dy = (_random(ROWS, COLS, dev, i) for i in range(1, 5))
    w, wb, gate = (_random(1, COLS, dev, i) for i in (5, 6, 7))
    w, wb = w[0], wb[0]
    s, y, rb, rs = nsa.residual_norm(x, z, gate=gate, scale=0.5, branch_weight=wb, weight=w)
    dx, dz, dgate, dwb, dw = nsa.residual_norm_backward(ds, dy, s, z, rb, rs, gate=gate, scale=0.5, branch_weight=wb, weight=w)
    sums, mags = torch.zeros(3, COLS, dtype=torch.float64, device=dev), torch.zeros(3, COLS, dtype=torch.float64, device=dev)
    for c in _chunks(ROWS):
        # A row's result does not depend on the rows beside it.
        part = nsa.residual_norm(x[c], z[c], gate=gate, scale=0.5, branch_weight=wb, weight=w)
        assert all(torch.equal(a[c], b) for a, b in zip((s, y, rb, rs), part))
        back = nsa.residual_norm_backward(ds[c], dy[c], s[c], z[c], rb[c], rs[c], gate=gate, scale=0.5, branch_weight=wb,
                                          weight=w, params=False)
        assert torch.equal(dx[c], back[0]) and torch.equal(dz[c], back[1])
        g = dy[c].double()
        shat = s[c].double() * rs[c].double()[:, None]
        u = w.double() * g
        top = ds[c].double() + rs[c].double()[:, None] * (u - shat * (u * shat).mean(1, keepdim=True))
        bhat = z[c].double() * rb[c].double()[:, None]
        sums[0] += (top * bhat).sum(0)
        mags[0] += (top * bhat).abs().sum(0)
        sums[1] += (g * shat).sum(0)
        mags[1] += (g * shat).abs().sum(0)
    # Each of 512 parts of at most 1036 rows is summed in order, then the
    # parts; top is formed to about COLS + 12 steps of its terms.
    depth = 1036 + 512 + 8
    top_depth = COLS // 64 + 24  # lanes of 64, then their sums
    err = (depth + 4 * top_depth) * U32 * mags
    for got, want, e in ((dgate[0], wb.double() * sums[0], wb.double().abs() * err[0]),
                         (dwb, gate[0].double() * sums[0], gate[0].double().abs() * err[0]), (dw, sums[1], err[1])):
        assert bool(((got.double() - want).abs() <= HALF * want.abs() + 1.05 * e).all())


def test_gated_mlp_with_projections_past_32_bits():
    # 530 rows over and over; rows are independent forward.  Backward all but
    # the last 530 rows have no gradient, so the weights' gradients are those
    # of 530 rows.
    dev = mlp._dev()
    n, d, f, times = 530, 64, 4096, 1000
    t = mlp._inputs(n, d, f, "bf16", dev, 3)
    m = {k: mlp._np(v) for k, v in t.items()}
    x = t["x"].repeat(times, 1)
    w = (t["wg"], t["wu"], t["wd"])
    y, gate, up = nsa.gated_mlp(x, *w)
    assert gate.numel() > 2 ** 31
    y64, a64, b64, _ = oracle.gated_mlp(m["x"], m["wg"], m["wu"], m["wd"], "silu")
    ba, bb, by = mlp._forward_bounds(m["x"], m["wg"], m["wu"], m["wd"], a64, b64, "silu", "bf16", y64, "fp32")
    last = slice((times - 1) * n, times * n)
    mlp._close(gate[last], a64, ba, "gate")
    mlp._close(up[last], b64, bb, "up")
    mlp._close(y[last], y64, by, "y")
    for i in range(0, times, 50):
        for full in (y, gate, up):
            part = full[i * n:(i + 50) * n].view(50, n, -1)
            assert bool((part == full[last]).all())
    dy = torch.zeros_like(x)
    dy[last] = t["dy"]
    dx, *dw = nsa.gated_mlp_backward(dy, x, *w, gate, up)
    a, b = mlp._np(gate[last]), mlp._np(up[last])
    o = oracle.gated_mlp_backward(m["dy"], m["x"], m["wg"], m["wu"], m["wd"], a, b, "silu")
    bounds = mlp._backward_bounds(o, m["dy"], m["x"], m["wg"], m["wu"], m["wd"], a, b, "silu", "bf16")
    mlp._close(dx[last], o["dx"], bounds["dx"], "dx")
    assert not bool(dx[:last.start].any())
    for g, name in zip(dw, ("dwg", "dwu", "dwd")):
        mlp._close(g, o[name], bounds[name], name)


@pytest.mark.parametrize("n", [2, 40])
def test_gated_mlp_with_weights_past_32_bits(n):
    dev = mlp._dev()
    d, f, step = 8192, 270_000, 15_000
    g = torch.Generator(device=dev).manual_seed(n)

    def make(rows, cols, scale):
        out = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
        for i in range(0, rows, 16384):
            part = out[i:i + 16384]
            part.copy_(torch.randn(part.shape, device=dev, generator=g).mul_(scale))
        return out

    x, dy = make(n, d, 1.0), make(n, d, 1.0)
    wg, wu, wd = make(f, d, d ** -0.5), make(f, d, d ** -0.5), make(d, f, f ** -0.5)
    assert wg.numel() > 2 ** 31
    y, gate, up = nsa.gated_mlp(x, wg, wu, wd)
    dx, dwg, dwu, dwd = nsa.gated_mlp_backward(dy, x, wg, wu, wd, gate, up)
    x64, dy64 = x.double(), dy.double()
    y64, ey, mag, dx64, edx, mdx = (torch.zeros(n, d, dtype=torch.float64, device=dev) for _ in range(6))

    def within(got, want, err):
        assert bool(((got.double() - want).abs() <= HALF * want.abs() + (1 + HALF) * err).all())

    # The bounds of test_gpu_gated_mlp, a slice of inner units at a time.
    for i in range(0, f, step):
        c = slice(i, i + step)
        g64, u64, d64 = wg[c].double(), wu[c].double(), wd[:, c].double()
        a, b = x64 @ g64.t(), x64 @ u64.t()
        ea, eb = ((d + 2) * U32 * (x64.abs() @ v.abs().t()) for v in (g64, u64))
        assert bool(((gate[:, c].double() - a).abs() <= ea).all()) and bool(((up[:, c].double() - b).abs() <= eb).all())
        a, b = gate[:, c].double(), up[:, c].double()  # from here on the errors of what follows
        sig = torch.sigmoid(a)
        value, slope = a * sig, sig * (1 + a * (1 - sig))
        eh = 8 * U32 * a.abs() * b.abs()
        h = value * b
        eh = eh + HALF * (h.abs() + eh)
        y64 += h @ d64.t()
        ey += (eh + 2 * ea * b.abs()) @ d64.abs().t()
        mag += (h.abs() + eh) @ d64.abs().t()
        dh = dy64 @ d64
        edh = (d + 1) * U32 * (dy64.abs() @ d64.abs())
        da, db = dh * b * slope, dh * value
        eslope = U32 * (8 + 4 * a.abs() + a.abs() ** 3)
        eda = b.abs() * slope.abs() * edh + (dh.abs() + edh) * b.abs() * eslope + 3 * U32 * da.abs()
        edb = value.abs() * edh + (dh.abs() + edh) * 8 * U32 * a.abs() + 2 * U32 * db.abs()
        eda, edb = eda + HALF * (da.abs() + eda), edb + HALF * (db.abs() + edb)
        dx64 += da @ g64 + db @ u64
        edx += eda @ g64.abs() + edb @ u64.abs()
        mdx += (da.abs() + eda) @ g64.abs() + (db.abs() + edb) @ u64.abs()
        for got, v, e in ((dwg[c], da, eda), (dwu[c], db, edb)):
            within(got, v.t() @ x64, e.t() @ x64.abs() + (n + 1) * U32 * ((v.abs() + e).t() @ x64.abs()))
        within(dwd[:, c], dy64.t() @ h, dy64.abs().t() @ eh + (n + 1) * U32 * (dy64.abs().t() @ (h.abs() + eh)))
    within(y, y64, ey + (f + 1) * U32 * mag)
    within(dx, dx64, edx + (2 * f + 2) * U32 * mdx)
