"""The training step's operators on tensors of more than 2^31 elements: what
lies past 32-bit offsets is as right as the rest.
"""

import pytest
import torch

import newton_schulz_matrix_amd as nsa

import test_gpu_training as base

pytestmark = pytest.mark.gpu

U32 = base.U32
HALF = base.HALF_STEP["bf16"]
ROWS, COLS = 530_000, 4096  # 2^31 + 23 million elements
CHUNK = 53_000


def _random(rows, cols, dev, seed, scale=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
    for i in range(0, rows, CHUNK):
        part = out[i:i + CHUNK]
        part.copy_(torch.randn(part.shape, device=dev, generator=g).mul_(scale))
    return out


def _chunks(n):
    return [slice(i, min(i + CHUNK, n)) for i in range(0, n, CHUNK)]


def test_layer_norm_past_32_bits():
    dev = base._dev()
    x, dy = _random(ROWS, COLS, dev, 1), _random(ROWS, COLS, dev, 2)
    w, b = (_random(1, COLS, dev, s)[0] for s in (3, 4))
    y, mean, rstd = nsa.layer_norm(x, w, b)
    dx, dw, db = nsa.layer_norm_backward(dy, x, mean, rstd, w)
    dw64, db64, adw, adb = (torch.zeros(COLS, dtype=torch.float64, device=dev) for _ in range(4))
    for s in _chunks(ROWS):
        # A row's result does not depend on the rows beside it.
        part = nsa.layer_norm(x[s], w, b)
        assert torch.equal(y[s], part[0]) and torch.equal(mean[s], part[1]) and torch.equal(rstd[s], part[2])
        assert torch.equal(dx[s], nsa.layer_norm_backward(dy[s], x[s], mean[s], rstd[s], w, params=False)[0])
        g = dy[s].double()
        xhat = (x[s].double() - mean[s].double()[:, None]) * rstd[s].double()[:, None]
        dw64 += (g * xhat).sum(0)
        db64 += g.sum(0)
        adw += (g * xhat).abs().sum(0)
        adb += g.abs().sum(0)
    depth = ROWS / 512 + 61  # as in test_gpu_training
    assert bool(((dw.double() - dw64).abs() <= HALF * dw64.abs() + 1.05 * depth * U32 * adw).all())
    assert bool(((db.double() - db64).abs() <= HALF * db64.abs() + 1.05 * depth * U32 * adb).all())


def test_embedding_past_32_bits():
    dev = base._dev()
    table = _random(ROWS, COLS, dev, 5)
    ids = torch.randperm(ROWS, device=dev, generator=torch.Generator(device=dev).manual_seed(6))
    out = nsa.embedding(ids, table, scale=0.5)
    for s in _chunks(ROWS):
        assert torch.equal(out[s], table[ids[s]] * 0.5)
    # Every id once: the gradient is the table again, to the bit.
    back = nsa.embedding_backward(ids, out, ROWS, scale=2.0)
    assert torch.equal(back, table)
    # And added to what is there (2 x is exact).
    nsa.embedding_backward(ids, out, ROWS, scale=2.0, out=back, accumulate=True)
    for s in _chunks(ROWS):
        assert torch.equal(back[s], table[s] * 2)


def _bound(got, want, bound, what):
    worst = float(((got.double() - want).abs() / bound.clamp(min=1e-300)).max())
    print(f"{what}: worst error {worst:.3f} of the bound", flush=True)
    assert worst <= 1, what


@pytest.mark.parametrize("n", [2, 9, 200])
def test_cross_entropy_of_a_vocabulary_past_32_bits(n):
    dev = base._dev()
    v, d = ROWS, COLS
    w = _random(v, d, dev, 7, scale=2.0 / 64)
    h = _random(n, d, dev, 8)
    t = torch.linspace(0, v - 1, n, device=dev).long()  # the first and the last row among them
    dloss = torch.full((n,), 1.0 / n, device=dev)
    loss, lse = nsa.linear_cross_entropy(h, w, t)
    dh, dw = nsa.linear_cross_entropy_backward(h, w, t, lse, dloss, out_dw=torch.full_like(w, float("nan")))
    h64 = h.double()
    z = torch.cat([h64 @ w[s].double().t().contiguous() for s in _chunks(v)], 1)
    # The bounds of test_gpu_training._check_xent, a logit's error by the
    # Cauchy-Schwarz inequality.
    wnorm = max(float(w[s].double().norm(dim=1).max()) for s in _chunks(v))
    ez = (d + 1) * U32 * h64.norm(dim=1) * wnorm
    lse64 = torch.logsumexp(z, 1)
    elz = ez + U32 * (96 + v / 96 / 16 + 40 + 4 * z.abs().amax(1) + 2 * lse64.abs())
    _bound(lse, lse64, elz, "lse")
    at = torch.arange(n, device=dev)
    loss64 = lse64 - z[at, t]
    _bound(loss, loss64, elz + ez + U32 * loss64.abs(), "loss")
    p = torch.exp(z - lse64[:, None])
    edz = p * (ez + elz + 8 * U32)[:, None]
    edz[at, t] += 2 * U32
    p[at, t] -= 1
    edz = (edz + HALF * p.abs()) / n
    p /= n
    dh64, eh = torch.zeros(n, d, dtype=torch.float64, device=dev), torch.zeros(n, d, dtype=torch.float64, device=dev)
    ahn = h64.abs()
    for s in _chunks(v):
        w64 = w[s].double()
        dh64 += p[:, s] @ w64
        eh += (edz[:, s] + U32 * (v + 20) * (p[:, s].abs() + edz[:, s])) @ w64.abs()
        dw64 = p[:, s].t().contiguous() @ h64
        ew = (edz[:, s] + U32 * (n + 20) * (p[:, s].abs() + edz[:, s])).t().contiguous() @ ahn
        _bound(dw[s], dw64, HALF * dw64.abs() + 1.05 * ew, f"dw {s.start}")
    _bound(dh, dh64, HALF * dh64.abs() + 1.05 * eh, "dh")


def test_cross_entropy_of_rows_past_32_bits():
    dev = base._dev()
    n, d, v = ROWS, COLS, 150
    h = _random(n, d, dev, 9)
    w = _random(v, d, dev, 10, scale=2.0 / 64)
    t = torch.arange(n, device=dev) % v
    t[::7] = -100
    loss, lse = nsa.linear_cross_entropy(h, w, t)
    g = 1.0 / n
    dh, dw = nsa.linear_cross_entropy_backward(h, w, t, lse, g, out_dh=torch.full_like(h, float("nan")))
    w64 = w.double()
    wt, aw = w64.t().contiguous(), w64.abs()
    dw64, ew = torch.zeros(v, d, dtype=torch.float64, device=dev), torch.zeros(v, d, dtype=torch.float64, device=dev)
    wnorm = float(w64.norm(dim=1).max())
    for s in _chunks(n):
        h64, ts = h[s].double(), t[s]
        z = h64 @ wt
        ez = (d + 1) * U32 * h64.norm(dim=1) * wnorm
        lse64 = torch.logsumexp(z, 1)
        elz = ez + U32 * (96 + v / 96 / 16 + 40 + 4 * z.abs().amax(1) + 2 * lse64.abs())
        valid = ts >= 0
        at = torch.nonzero(valid)[:, 0]
        loss64 = torch.where(valid, lse64 - z.gather(1, ts.clamp(min=0)[:, None])[:, 0], 0.0)
        assert bool(((lse[s].double() - lse64).abs() <= elz).all())
        assert bool(((loss[s].double() - loss64).abs() <= (elz + ez + U32 * loss64.abs()) * valid).all())
        p = torch.exp(z - lse64[:, None])
        edz = p * (ez + elz + 8 * U32)[:, None]
        edz[at, ts[at]] += 2 * U32
        p[at, ts[at]] -= 1
        # The coefficient's own rounding to fp32 (g is no power of two).
        edz = (edz + (HALF + U32) * p.abs()) * g * valid[:, None]
        p *= g * valid[:, None]
        dh64 = p @ w64
        eh = (edz + U32 * (v + 20) * (p.abs() + edz)) @ aw
        assert bool(((dh[s].double() - dh64).abs() <= HALF * dh64.abs() + 1.05 * eh).all()), s
        dw64 += p.t().contiguous() @ h64
        ew += (edz + U32 * (n + 20) * (p.abs() + edz)).t().contiguous() @ h64.abs()
    _bound(dw, dw64, HALF * dw64.abs() + 1.05 * ew, "dw")
