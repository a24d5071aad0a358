"""Embedding, layer norm and cross entropy on the GPU against the fp64 oracle.

Every bound below is a worst case written out from the arithmetic, with
u32 = 2^-24 (half a step of fp32) and u = half a step of the stored type
(bf16 2^-8, fp16 2^-11, fp32 2^-24; torch.finfo(t).eps / 2):

* a value rounded once to the stored type: u |value| (plus half of fp16's
  smallest step where the value may be that small);
* a sum of m terms in fp32 in any order: at most (m - 1) u32 times the sum of
  the terms' magnitudes, or the depth of the sum's tree where that is known.
"""

import math

import numpy as np
import pytest
import torch

import oracle
import newton_schulz_matrix_amd as nsa
from newton_schulz_matrix_amd import _binding as B

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U32 = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, want, bound, what):
    got = _np(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, what
    off = np.abs(got - want)
    worst = float(np.max(off / np.maximum(bound, 1e-300))) if off.size else 0.0
    print(f"{what}: worst error {worst:.3f} of the bound", flush=True)
    assert np.all(off <= bound), (what, worst)


def _word(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


def _poisoned(shape, dtype, dev):
    """NaNs to be overwritten."""
    return torch.full(shape, float("nan"), dtype=dtype, device=dev)


# ---------------------------------------------------------------------------
# Layer norm.
# ---------------------------------------------------------------------------
# Depth of a row sum: up to 32 elements per thread (20 for the longest rows
# here in the looping kernel), six shuffle steps, sixteen waves, one division.
DEPTH = 56


def _norm_inputs(rows, cols, dtype, pdtype, dev, seed=0, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g) + offset).to(DTYPES[dtype]).to(dev)
    w = (1 + 0.1 * torch.randn(cols, generator=g)).to(DTYPES[pdtype]).to(dev)
    b = (0.1 * torch.randn(cols, generator=g)).to(DTYPES[pdtype]).to(dev)
    dy = torch.randn(rows, cols, generator=g).to(DTYPES[dtype]).to(dev)
    return x, w, b, dy


def _norm_y_bound(x, w, b, mean, rstd, y, dtype, eps):
    # mean: off by DEPTH u32 max|x|; rstd: half the relative error of the sum
    # of squares (DEPTH, and 2 per term) and 3 for division and root; then
    # the scale and the shift one each.
    top = np.abs(x).max(1, keepdims=True)
    aw = np.abs(w)[None, :]
    xhat = np.abs((x - mean[:, None]) * rstd[:, None])
    fp32 = U32 * (aw * ((DEPTH + 1) * rstd[:, None] * top + (DEPTH / 2 + 6) * xhat) + np.abs(b)[None, :] + 2 * np.abs(y))
    return HALF_STEP[dtype] * np.abs(y) + TINY[dtype] + 1.05 * fp32


NORM_SHAPES = [(1, 1), (1, 4096), (3, 64), (7, 97), (130, 768), (5, 1000), (9, 1024), (6, 1025), (33, 2048), (4, 4097),
               (3, 8192), (2, 9000), (2, 16384), (2, 20001)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype,pdtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"),
                                          ("fp32", "fp32")])
def test_layer_norm_matches_the_oracle(rows, cols, dtype, pdtype):
    dev = _dev()
    print(f"layer norm {rows}x{cols} {dtype}/{pdtype}", flush=True)
    x, w, b, dy = _norm_inputs(rows, cols, dtype, pdtype, dev, seed=rows * 31 + cols)
    eps = 1e-5
    st = _word(dev)
    y, mean, rstd = nsa.layer_norm(x, w, b, eps=eps, out=_poisoned(x.shape, x.dtype, dev), status=st)
    y64, mean64, rstd64 = oracle.layer_norm(_np(x), _np(w), _np(b), float(np.float32(eps)))
    top = np.abs(_np(x)).max(1)
    _close(mean, mean64, (DEPTH + 1) * U32 * top, "mean")
    # The sum of squares is taken about the rounded mean: the square of the
    # mean's error joins it.
    _close(rstd, rstd64, rstd64 * ((DEPTH / 2 + 6) * U32 + (rstd64 * (DEPTH + 1) * U32 * top) ** 2
                                   + rstd64 * U32 * top), "rstd")
    _close(y, y64, _norm_y_bound(_np(x), _np(w), _np(b), mean64, rstd64, y64, dtype, eps), "y")

    # Backward, from the statistics the forward wrote.
    dx, dw, db = nsa.layer_norm_backward(dy, x, mean, rstd, w, out=_poisoned(x.shape, x.dtype, dev), status=st)
    g64, x64, w64, m64, r64 = _np(dy), _np(x), _np(w), _np(mean)[:, None], _np(rstd)[:, None]
    dx64, dw64, db64 = oracle.layer_norm_backward(g64, x64, _np(mean), _np(rstd), w64)
    # xhat is off by two roundings of its own size, a by one; each mean by the
    # depth of its sum and the terms' roundings, and the difference by one
    # rounding per term.
    xh = np.abs((x64 - m64) * r64)
    a = np.abs(g64 * w64)
    fp32 = U32 * r64 * (4 * a + (DEPTH + 8) * (a.mean(1, keepdims=True) + xh * (a * xh).mean(1, keepdims=True)))
    _close(dx, dx64, HALF_STEP[dtype] * np.abs(dx64) + TINY[dtype] + 1.05 * fp32, "dx")
    # A block adds at most rows / 512 + 1 rows (four of them side by side),
    # the join 16 groups of 32.
    depth = rows / 512 + 1 + 4 + 32 + 16 + 4
    _close(dw, dw64, HALF_STEP[pdtype] * np.abs(dw64) + TINY[pdtype] + 1.05 * depth * U32 * (np.abs(g64) * xh).sum(0), "dweight")
    _close(db, db64, HALF_STEP[pdtype] * np.abs(db64) + TINY[pdtype] + 1.05 * depth * U32 * np.abs(g64).sum(0), "dbias")
    assert int(st.item()) == 0


@pytest.mark.parametrize("cols", [768, 1001, 20001])
def test_layer_norm_many_rows_and_options(cols):
    # More rows than the backward's blocks, no weight, no bias, no statistics.
    dev = _dev()
    rows = 3000 if cols < 2000 else 700
    x, _, _, dy = _norm_inputs(rows, cols, "fp32", "fp32", dev, seed=cols)
    y, mean, rstd = nsa.layer_norm(x)
    y2, none_m, none_r = nsa.layer_norm(x, stats=False)
    assert none_m is None and none_r is None and torch.equal(y, y2)
    one = np.ones(cols)
    y64, mean64, rstd64 = oracle.layer_norm(_np(x), eps=float(np.float32(1e-5)))
    _close(y, y64, _norm_y_bound(_np(x), one, 0 * one, mean64, rstd64, y64, "fp32", 1e-5), "y")
    dx, dw, db = nsa.layer_norm_backward(dy, x, mean, rstd)
    only, no_w, no_b = nsa.layer_norm_backward(dy, x, mean, rstd, params=False)
    assert no_w is None and no_b is None and torch.equal(dx, only)
    _, dw64, db64 = oracle.layer_norm_backward(_np(dy), _np(x), _np(mean), _np(rstd))
    depth = rows / 512 + 61
    g64, xh = np.abs(_np(dy)), np.abs((_np(x) - _np(mean)[:, None]) * _np(rstd)[:, None])
    _close(dw, dw64, U32 * np.abs(dw64) + 1.05 * depth * U32 * 2 * (g64 * xh).sum(0), "dweight")
    _close(db, db64, U32 * np.abs(db64) + 1.05 * depth * U32 * g64.sum(0), "dbias")
    # In place: y over x, dx over dy.
    xi, dyi = x.clone(), dy.clone()
    nsa.layer_norm(xi, out=xi)
    nsa.layer_norm_backward(dyi, x, mean, rstd, out=dyi)
    assert torch.equal(xi, y) and torch.equal(dyi, dx)


def test_layer_norm_strides_alignment_and_rank():
    dev = _dev()
    for cols, lead, off in ((768, 800, 0), (768, 801, 0), (768, 800, 3), (96, 97, 1)):
        big = torch.randn(50, lead + off, device=dev).to(torch.bfloat16)
        x = big[:, off:off + cols]
        want = nsa.layer_norm(x.contiguous())
        out = torch.zeros_like(big)
        got = nsa.layer_norm(x, out=out[:, off:off + cols])
        # Another summation order (vectors against single elements): both are
        # within the bound, so they differ by at most one bf16 step.
        assert (got[0].double() - want[0].double()).abs().max() <= 2.0 ** -7 * want[0].double().abs().max()
        assert torch.count_nonzero(out[:, :off]) == 0 and torch.count_nonzero(out[:, off + cols:]) == 0
        dy = torch.randn_like(x.contiguous())
        dx = nsa.layer_norm_backward(dy, x, want[1], want[2])[0]
        ref = nsa.layer_norm_backward(dy, x.contiguous(), want[1], want[2])[0]
        assert (dx.double() - ref.double()).abs().max() <= 2.0 ** -7 * ref.double().abs().max()
    x = torch.randn(3, 4, 5, 64, device=dev)
    y, mean, rstd = nsa.layer_norm(x)
    flat = nsa.layer_norm(x.view(60, 64))
    assert y.shape == x.shape and mean.shape == (3, 4, 5)
    assert torch.equal(y.view(60, 64), flat[0]) and torch.equal(rstd.view(-1), flat[2])
    assert nsa.layer_norm_backward(x, x, mean, rstd)[0].shape == x.shape


def test_layer_norm_empty_constant_and_nonfinite_rows():
    dev = _dev()
    x = torch.empty(0, 96, device=dev)
    y, mean, rstd = nsa.layer_norm(x)
    assert y.shape == (0, 96) and mean.numel() == 0
    dx, dw, db = nsa.layer_norm_backward(x, x, mean, rstd, torch.ones(96, device=dev))
    assert dx.shape == (0, 96) and torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0
    # A constant row: variance 0, rstd = 1 / sqrt(eps), y = bias.  3 is exact
    # in every sum, so the deviations are exact zeros.
    st = _word(dev)
    c = torch.full((2, 512), 3.0, device=dev, dtype=torch.bfloat16)
    b = torch.linspace(-1, 1, 512, device=dev).to(torch.bfloat16)
    y, mean, rstd = nsa.layer_norm(c, bias=b, status=st)
    assert torch.equal(y, b.expand(2, 512)) and (mean == 3).all()
    assert (rstd.double() * math.sqrt(1e-5) - 1).abs().max() < 4 * U32 and int(st.item()) == 0
    # A large mean against a small spread: the deviations keep their digits.
    g = torch.Generator().manual_seed(3)
    x = (4096 + torch.randint(-8, 9, (4, 1000), generator=g)).float().to(dev)
    y = nsa.layer_norm(x)[0]
    y64, m64, r64 = oracle.layer_norm(_np(x), eps=float(np.float32(1e-5)))
    one = np.ones(1000)
    _close(y, y64, _norm_y_bound(_np(x), one, 0 * one, m64, r64, y64, "fp32", 1e-5), "y about 4096")
    # NaN and infinity stay in their rows and set the status word.
    x = torch.randn(4, 300, device=dev)
    clean = nsa.layer_norm(x)[0]
    x[1, 7], x[2, 8] = float("nan"), float("inf")
    y, mean, rstd = nsa.layer_norm(x, status=st)
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
    assert torch.equal(y[0], clean[0]) and torch.equal(y[3], clean[3])
    assert int(st.item()) == B.NS_ERR_NONFINITE | B.STATUS_AT_OUTPUT


# ---------------------------------------------------------------------------
# Embedding.
# ---------------------------------------------------------------------------

def _skewed_ids(n, vocab, seed, bad=False):
    """A few ids take most positions; some ids take none."""
    rng = np.random.default_rng(seed)
    ids = (vocab * rng.random(n) ** 4).astype(np.int64)
    if n > 40:
        ids[n // 4:n // 2] = vocab - 1  # one long run
    if bad and n > 4:
        ids[1], ids[2], ids[-1] = -1, vocab, 1 << 40
    return torch.from_numpy(ids)


EMBED_SHAPES = [(1, 1, 1), (1, 500, 4096), (5, 7, 64), (63, 64, 97), (300, 65, 512), (1000, 5000, 768), (4099, 33000, 200),
                (5000, 3, 1000), (20000, 700, 130), (70000, 50257, 8)]


@pytest.mark.parametrize("n,vocab,cols", EMBED_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("ids32", [False, True])
def test_embedding_and_its_gradient(n, vocab, cols, dtype, ids32):
    dev = _dev()
    print(f"embedding n={n} vocab={vocab} cols={cols} {dtype} int{32 if ids32 else 64}", flush=True)
    ids = _skewed_ids(n, vocab, n + cols, bad=False)
    ids_d = ids.to(dev).to(torch.int32 if ids32 else torch.int64)
    g = torch.Generator(device=dev).manual_seed(n)
    table = torch.randn(vocab, cols, device=dev, generator=g).to(DTYPES[dtype])
    scale = math.sqrt(cols)
    st = _word(dev)
    out = nsa.embedding(ids_d, table, scale=scale, out=_poisoned((n, cols), table.dtype, dev), status=st)
    # One fp32 product, rounded once: exactly torch's.
    want = (table.cpu()[ids].float() * np.float32(scale)).to(table.dtype)
    assert torch.equal(out.cpu(), want)
    dy = torch.randn(n, cols, device=dev, generator=g).to(table.dtype)
    dt = nsa.embedding_backward(ids_d, dy, vocab, scale=scale, out=_poisoned((vocab, cols), table.dtype, dev), status=st)
    dt64 = oracle.embedding_backward(ids.numpy(), _np(dy), vocab, float(np.float32(scale)))
    mag = oracle.embedding_backward(ids.numpy(), np.abs(_np(dy)), vocab, scale)
    count = np.bincount(ids.numpy(), minlength=vocab)[:, None]
    _close(dt, dt64, HALF_STEP[dtype] * np.abs(dt64) + TINY[dtype] + 1.05 * U32 * (count + 1) * mag, "dtable")
    assert torch.count_nonzero(dt[torch.from_numpy(count[:, 0] == 0).to(dev)]) == 0
    # Again: the same bits.
    assert torch.equal(dt, nsa.embedding_backward(ids_d, dy, vocab, scale=scale))
    # Added to what is there: ids without a position are left alone.
    base = torch.randn(vocab, cols, device=dev, generator=g).to(table.dtype)
    acc = base.clone()
    nsa.embedding_backward(ids_d, dy, vocab, scale=scale, out=acc, accumulate=True, status=st)
    sum64 = _np(base) + dt64
    _close(acc, sum64, HALF_STEP[dtype] * np.abs(sum64) + TINY[dtype]
           + 1.05 * U32 * ((count + 1) * mag + np.abs(sum64) + np.abs(dt64)), "accumulated")
    absent = torch.from_numpy(count[:, 0] == 0).to(dev)
    assert torch.equal(acc[absent], base[absent])
    assert int(st.item()) == 0


def test_embedding_bad_ids_shapes_strides_and_empty():
    dev = _dev()
    vocab, cols, n = 300, 96, 500
    ids = _skewed_ids(n, vocab, 4, bad=True)
    ids_d = ids.to(dev).view(5, 100)
    wide = torch.randn(vocab, cols + 9, device=dev).to(torch.bfloat16)
    table = wide[:, 1:1 + cols]  # rows off every 16-byte boundary
    st = _word(dev)
    out = nsa.embedding(ids_d, table, scale=2.0, status=st)
    assert out.shape == (5, 100, cols) and int(st.item()) == B.STATUS_BAD_INDEX
    assert np.array_equal(_np(out).reshape(n, cols), oracle.embedding(ids.numpy(), _np(table), 2.0))
    dy = torch.randn(5, 100, cols, device=dev).to(torch.bfloat16)
    st.zero_()
    big = torch.zeros(vocab, cols + 9, device=dev, dtype=torch.bfloat16)
    dt = nsa.embedding_backward(ids_d, dy, vocab, out=big[:, 1:1 + cols], status=st)
    assert int(st.item()) == B.STATUS_BAD_INDEX
    assert torch.count_nonzero(big[:, 0]) == 0 and torch.count_nonzero(big[:, 1 + cols:]) == 0
    dt64 = oracle.embedding_backward(ids.numpy(), _np(dy), vocab)
    mag = oracle.embedding_backward(ids.numpy(), np.abs(_np(dy)), vocab)
    _close(dt, dt64, HALF_STEP["bf16"] * np.abs(dt64) + 1.05 * U32 * n * mag, "dtable")
    # NaNs in a bad id's row of dy reach nothing.
    dy.view(n, cols)[1] = float("nan")
    assert torch.equal(nsa.embedding_backward(ids_d, dy, vocab), dt.contiguous())
    # No positions: zeros, or nothing added.
    none = torch.empty(0, dtype=torch.int64, device=dev)
    empty = torch.empty(0, cols, device=dev, dtype=torch.bfloat16)
    assert nsa.embedding(none, table).shape == (0, cols)
    assert torch.count_nonzero(nsa.embedding_backward(none, empty, vocab)) == 0
    keep = dt.contiguous().clone()
    nsa.embedding_backward(none, empty, vocab, out=keep, accumulate=True)
    assert torch.equal(keep, dt)
    # All positions bad, and one id for all positions.
    bad = torch.full((400,), -1, dtype=torch.int64, device=dev)
    dy = torch.randn(400, cols, device=dev)
    assert torch.count_nonzero(nsa.embedding_backward(bad, dy, vocab)) == 0
    one = torch.full((400,), 7, dtype=torch.int64, device=dev)
    got = nsa.embedding_backward(one, dy, vocab)
    _close(got[7], _np(dy).sum(0), 401 * U32 * np.abs(_np(dy)).sum(0), "one id")
    assert torch.count_nonzero(got) == torch.count_nonzero(got[7])


def test_embedding_gradient_long_lists():
    # One id takes nearly all of 200 000 positions: partial sums of chunks.
    dev = _dev()
    n, vocab, cols = 200_000, 900, 64
    ids = torch.full((n,), 17, dtype=torch.int64)
    ids[::1001] = torch.arange(len(ids[::1001])) % vocab
    dy = torch.randn(n, cols, generator=torch.Generator().manual_seed(5))
    got = nsa.embedding_backward(ids.to(dev), dy.to(dev), vocab)
    want = oracle.embedding_backward(ids.numpy(), dy.numpy(), vocab)
    mag = oracle.embedding_backward(ids.numpy(), np.abs(dy.numpy()), vocab)
    # Depth: chunks of at most 128 positions, at most n / 64 of them.
    _close(got, want, (300 + n / 64) * U32 * mag, "dtable")


# ---------------------------------------------------------------------------
# Cross entropy.
# ---------------------------------------------------------------------------

def _xent_inputs(n, d, v, dtype, dev, seed=0, spread=2.0, ignored=0.2):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(n, d, generator=g).to(DTYPES[dtype])
    w = (spread / math.sqrt(d) * torch.randn(v, d, generator=g)).to(DTYPES[dtype])
    t = torch.randint(0, v, (n,), generator=g)
    t[torch.rand(n, generator=g) < ignored] = -100
    dloss = torch.rand(n, generator=g) / max(n, 1)
    return h.to(dev), w.to(dev), t.to(dev), dloss.to(dev)


def _logit_error(h, w, d):
    # Products of 16-bit values are exact in fp32, those of fp32 values off by
    # u32; the sum over d in any order.
    return (d + 1) * U32 * (np.abs(h) @ np.abs(w).T)


def _check_xent(n, d, v, dtype, dev, h, w, t, dloss, ignore_index=-100, dw_rows=None):
    h64, w64, t64, g64 = _np(h), _np(w), t.cpu().numpy(), _np(dloss)
    ez = _logit_error(h64, w64, d)
    st = _word(dev)
    loss, lse = nsa.linear_cross_entropy(h, w, t, ignore_index=ignore_index, status=st)
    loss64, lse64 = oracle.linear_cross_entropy(h64, w64, t64, ignore_index)
    # lse: the logits' errors, and the sum of up to v exponentials (96 in a
    # lane, then the tiles' joins), each off by a few u32 of its argument.
    z64 = h64 @ w64.T
    span = np.abs(z64).max(1)
    elz = ez.max(1) + U32 * (96 + v / 96 / 16 + 40 + 4 * span + 2 * np.abs(lse64))
    _close(lse, lse64, elz, "lse")
    valid = (t64 != ignore_index) & (t64 >= 0) & (t64 < v)
    _close(loss[torch.from_numpy(valid).to(dev)], loss64[valid], (elz + ez.max(1) + U32 * np.abs(loss64))[valid], "loss")
    assert torch.count_nonzero(loss[torch.from_numpy(t64 == ignore_index).to(dev)]) == 0
    dh, dw = nsa.linear_cross_entropy_backward(
        h, w, t, lse, dloss, ignore_index=ignore_index, status=st,
        out_dh=_poisoned(h.shape, h.dtype, dev), out_dw=_poisoned(w.shape, w.dtype, dev))
    dh64, dw64 = oracle.linear_cross_entropy_backward(h64, w64, t64, g64, ignore_index)
    # dz: e^(z - lse) off by the errors of both in relative terms, the
    # difference from 1 by the same amounts, then rounded to the type (for
    # fp16 also half of its smallest step, 2^-25, in units of max g 2^-15).
    p = np.exp(z64 - lse64[:, None])
    g = np.abs(g64) * valid
    hot = np.zeros_like(p)
    hot[np.nonzero(valid)[0], t64[valid]] = 1.0
    dz = np.abs(p - hot) * g[:, None]
    u = HALF_STEP[dtype]
    edz = dz * u + (p * (ez + elz[:, None] + 8 * U32) + 2 * U32 * hot) * g[:, None]
    if dtype == "fp16":
        edz += (g.max(initial=0.0) * 2.0 ** -40) * (g > 0)[:, None]
    adz = dz + edz
    eh = 1.05 * (edz @ np.abs(w64) + U32 * (v + 20) * (adz @ np.abs(w64)))
    ew = 1.05 * (edz.T @ np.abs(h64) + U32 * (n + 20) * (adz.T @ np.abs(h64)))
    _close(dh, dh64, u * np.abs(dh64) + TINY[dtype] + eh, "dh")
    _close(dw, dw64, u * np.abs(dw64) + TINY[dtype] + ew, "dw")
    assert int(st.item()) == 0
    return loss, lse, dh, dw


XENT_SHAPES = [(1, 1, 1), (1, 64, 1000), (1, 4096, 70), (1, 7, 40000), (2, 128, 191), (3, 5, 9), (5, 1001, 77), (8, 96, 1000), (9, 100, 600), (17, 100, 193), (64, 64, 500), (128, 256, 385), (129, 192, 700),
               (200, 1000, 777), (385, 320, 1153), (700, 64, 64),
               # Few rows: dH in many splits of the vocabulary.
               (35, 130, 20011), (1, 72, 30000)]


@pytest.mark.parametrize("n,d,v", XENT_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_linear_cross_entropy_matches_the_oracle(n, d, v, dtype):
    dev = _dev()
    print(f"cross entropy n={n} d={d} v={v} {dtype}", flush=True)
    h, w, t, dloss = _xent_inputs(n, d, v, dtype, dev, seed=n + d + v)
    _check_xent(n, d, v, dtype, dev, h, w, t, dloss)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_linear_cross_entropy_strides_alignment_and_int32(dtype):
    dev = _dev()
    n, d, v = 150, 128, 400
    h, w, t, dloss = _xent_inputs(n, d, v, dtype, dev, seed=9)
    want = _check_xent(n, d, v, dtype, dev, h, w, t, dloss)
    for off, pad in ((0, 8), (1, 3), (8, 8)):
        hw = torch.full((n, d + off + pad), float("nan"), dtype=h.dtype, device=dev)
        ww = torch.full((v, d + off + pad), float("nan"), dtype=h.dtype, device=dev)
        hs, ws = hw[:, off:off + d], ww[:, off:off + d]
        hs.copy_(h)
        ws.copy_(w)
        loss, lse = nsa.linear_cross_entropy(hs, ws, t.to(torch.int32))
        assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])
        out_h, out_w = torch.zeros_like(hw), torch.zeros_like(ww)
        dh, dw = nsa.linear_cross_entropy_backward(hs, ws, t.to(torch.int32), lse, dloss, out_dh=out_h[:, off:off + d],
                                                   out_dw=out_w[:, off:off + d])
        assert torch.equal(dh, want[2]) and torch.equal(dw, want[3])
        for o in (out_h, out_w):
            assert torch.count_nonzero(o[:, :off]) == 0 and torch.count_nonzero(o[:, off + d:]) == 0
    # One gradient at a time, and one number for all rows.
    only_h = nsa.linear_cross_entropy_backward(h, w, t, want[1], dloss, need_dw=False)
    only_w = nsa.linear_cross_entropy_backward(h, w, t, want[1], dloss, need_dh=False)
    assert only_h[1] is None and only_w[0] is None
    assert torch.equal(only_h[0], want[2]) and torch.equal(only_w[1], want[3])
    same = nsa.linear_cross_entropy_backward(h, w, t, want[1], 0.125)
    full = nsa.linear_cross_entropy_backward(h, w, t, want[1], torch.full((n,), 0.125, device=dev))
    assert torch.equal(same[0], full[0]) and torch.equal(same[1], full[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_linear_cross_entropy_several_pieces(dtype):
    # 2^28 elements of dz per piece: 20 000 rows take the vocabulary in
    # several.  The oracle looks at rows of every part of the result.
    dev = _dev()
    n, d, v = 20_000, 64, 15_000
    h, w, t, dloss = _xent_inputs(n, d, v, dtype, dev, seed=2)
    loss, lse = nsa.linear_cross_entropy(h, w, t)
    dh, dw = nsa.linear_cross_entropy_backward(h, w, t, lse, dloss)
    z = h.double() @ w.double().t().contiguous()
    ref = torch.logsumexp(z, 1)
    ez = (d + 1) * U32 * float((h.double().abs().amax(0) * w.double().abs().amax(0)).sum())
    assert (lse.double() - ref).abs().max() <= ez + U32 * 400
    p = torch.exp(z - ref[:, None])
    valid = t >= 0
    p[torch.nonzero(valid)[:, 0], t[valid]] -= 1
    p *= (dloss.double() * valid)[:, None]
    dh64, dw64 = p @ w.double(), p.t().contiguous() @ h.double()
    u = HALF_STEP[dtype]
    e = 2 * ez + 20 * U32
    bh = (u + e + v * U32) * (p.abs() @ w.double().abs()) + e * dloss.double()[:, None] * w.double().abs().amax(0)
    bw = (u + e + n * U32) * (p.abs().t().contiguous() @ h.double().abs()) + e * float(dloss.max()) * n * 0
    hot = torch.zeros(v, d, device=dev, dtype=torch.float64)
    hot.index_add_(0, t[valid], (dloss.double()[:, None] * h.double().abs())[valid])
    bw += e * hot
    if dtype == "fp16":
        sub = float(dloss.max()) * 2.0 ** -40
        bh += sub * w.double().abs().sum(0)
        bw += sub * h.double().abs().sum(0)
    _close(dh, _np(dh64), _np(1.05 * bh + u * dh64.abs()) + TINY[dtype], "dh")
    _close(dw, _np(dw64), _np(1.05 * bw + u * dw64.abs()) + TINY[dtype], "dw")


def test_linear_cross_entropy_targets_outside_and_ignored():
    dev = _dev()
    n, d, v = 70, 64, 300
    h, w, t, dloss = _xent_inputs(n, d, v, "bf16", dev, seed=3, ignored=0.0)
    base = _check_xent(n, d, v, "bf16", dev, h, w, t, dloss)
    st = _word(dev)
    bad = t.clone()
    bad[3], bad[4], bad[5] = v, -1, 1 << 40
    loss, lse = nsa.linear_cross_entropy(h, w, bad, status=st)
    assert torch.isnan(loss[3:6]).all() and torch.equal(lse, base[1])
    assert torch.equal(loss[6:], base[0][6:]) and int(st.item()) == B.STATUS_BAD_INDEX
    st.zero_()
    dh, dw = nsa.linear_cross_entropy_backward(h, w, bad, lse, dloss, status=st)
    assert torch.count_nonzero(dh[3:6]) == 0 and torch.equal(dh[6:], base[2][6:])
    assert int(st.item()) == B.STATUS_BAD_INDEX
    # The same rows ignored instead: the same gradients, no bit.
    st.zero_()
    ign = t.clone()
    ign[3:6] = 299
    keep = torch.nonzero(t == 299)[:, 0]
    loss_i, _ = nsa.linear_cross_entropy(h, w, ign, ignore_index=299, status=st)
    dh_i, dw_i = nsa.linear_cross_entropy_backward(h, w, ign, lse, dloss, ignore_index=299, status=st)
    assert (loss_i[3:6] == 0).all() and (loss_i[keep] == 0).all() and int(st.item()) == 0
    if len(keep) == 0:
        assert torch.equal(dh_i, dh) and torch.equal(dw_i, dw)
    # All rows ignored: zeros everywhere.
    none = torch.full_like(t, -100)
    loss, lse = nsa.linear_cross_entropy(h, w, none)
    dh, dw = nsa.linear_cross_entropy_backward(h, w, none, lse, dloss)
    for x in (loss, dh, dw):
        assert torch.count_nonzero(x) == 0
    # No rows.
    e = torch.empty(0, d, device=dev, dtype=torch.bfloat16)
    nt = torch.empty(0, dtype=torch.int64, device=dev)
    loss, lse = nsa.linear_cross_entropy(e, w, nt)
    dh, dw = nsa.linear_cross_entropy_backward(e, w, nt, lse, lse)
    assert loss.numel() == 0 and dh.shape == (0, d) and torch.count_nonzero(dw) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_linear_cross_entropy_nonfinite_and_extreme_logits(dtype):
    dev = _dev()
    n, d, v = 140, 64, 500
    h, w, t, dloss = _xent_inputs(n, d, v, dtype, dev, seed=6, ignored=0.0)
    loss0, lse0 = nsa.linear_cross_entropy(h, w, t)
    # A NaN row of h stays in its row; ignored or without weight it reaches no gradient.
    hn = h.clone()
    hn[5] = float("nan")
    st = _word(dev)
    loss, lse = nsa.linear_cross_entropy(hn, w, t, status=st)
    assert torch.isnan(loss[5]) and torch.isnan(lse[5]) and int(st.item()) == B.NS_ERR_NONFINITE | B.STATUS_AT_OUTPUT
    mask = torch.arange(n, device=dev) != 5
    assert torch.equal(loss[mask], loss0[mask])
    tn = t.clone()
    tn[5] = -100
    g5 = dloss.clone()
    g5[5] = 0
    dh_a, _ = nsa.linear_cross_entropy_backward(hn, w, tn, lse, dloss, need_dw=False)
    dh_b, _ = nsa.linear_cross_entropy_backward(hn, w, t, lse, g5, need_dw=False)
    assert torch.count_nonzero(dh_a[5]) == 0 and torch.equal(dh_a, dh_b) and torch.isfinite(dh_a).all()
    # Weight rows of -inf against positive columns: logits of -inf, probability 0.
    hp, wi = h.abs() + 0.1, w.clone()
    hp = hp.to(h.dtype)
    wi[v // 2:] = -float("inf")
    tl = t % (v // 2)
    loss, lse = nsa.linear_cross_entropy(hp, wi, tl)
    part = nsa.linear_cross_entropy(hp, wi[:v // 2].contiguous(), tl)
    assert (lse.double() - part[1].double()).abs().max() <= 8 * U32 * lse.abs().max()
    assert torch.isfinite(loss).all()
    # Every logit -inf: lse -inf, no finite loss.
    loss, lse = nsa.linear_cross_entropy(hp[:3], torch.full_like(w, -float("inf")), tl[:3])
    assert (lse == -float("inf")).all() and not torch.isfinite(loss).any()
    # Logits of some thousands: one probability is 1, the others 0.
    big = (300.0 if dtype == "fp16" else 3000.0) * torch.nn.functional.one_hot(torch.arange(n, device=dev) % 60, d).to(h.dtype)
    eye = torch.zeros(v, d, device=dev, dtype=h.dtype)
    eye[torch.arange(60), torch.arange(60)] = 10.0
    loss, lse = nsa.linear_cross_entropy(big, eye, torch.arange(n, device=dev) % 60)
    assert torch.count_nonzero(loss) == 0 and torch.equal(lse, big.float().amax(1) * 10)
    dh, dw = nsa.linear_cross_entropy_backward(big, eye, torch.arange(n, device=dev) % 60, lse, dloss)
    assert torch.count_nonzero(dh) == 0 and torch.count_nonzero(dw) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_linear_cross_entropy_backward_keeps_nonfinite_rows_out(dtype):
    # Rows without a gradient may hold anything in h; a coefficient that is
    # not finite reaches its own row of dh only (and dw).
    dev = _dev()
    n, d, v = 300, 72, 400
    h, w, t, dloss = _xent_inputs(n, d, v, dtype, dev, seed=16, ignored=0.0)
    lse = nsa.linear_cross_entropy(h, w, t)[1]
    t[3], t[150], t[299] = -100, v + 7, -100
    dloss[77] = 0
    rows = [3, 77, 150, 299]
    dh0, dw0 = nsa.linear_cross_entropy_backward(h, w, t, lse, dloss)
    hn, ln = h.clone(), lse.clone()
    hn[3], hn[77], hn[150], hn[299, 5] = float("nan"), float("inf"), -float("inf"), float("nan")
    ln[rows] = float("nan")
    st = _word(dev)
    dh, dw = nsa.linear_cross_entropy_backward(hn, w, t, ln, dloss, status=st)
    assert torch.equal(dh, dh0) and torch.equal(dw, dw0) and torch.count_nonzero(dh[rows]) == 0
    assert int(st.item()) == B.STATUS_BAD_INDEX
    for value in (float("inf"), float("nan")):
        bad = dloss.clone()
        bad[20] = value
        zero = dloss.clone()
        zero[20] = 0
        dh, dw = nsa.linear_cross_entropy_backward(h, w, t, lse, bad)
        base = nsa.linear_cross_entropy_backward(h, w, t, lse, zero)[0]
        others = torch.arange(n, device=dev) != 20
        assert torch.equal(dh[others], base[others]) and not torch.isfinite(dh[20]).all()
        assert not torch.isfinite(dw).all()


def test_linear_cross_entropy_tiny_and_uneven_coefficients_fp16():
    # fp16 holds dz in units of the largest coefficient: a batch of small
    # ones, and rows whose coefficients differ by a factor of 1000.
    dev = _dev()
    n, d, v = 200, 128, 300
    h, w, t, _ = _xent_inputs(n, d, v, "fp16", dev, seed=8)
    for g in (torch.full((n,), 1e-4, device=dev), torch.logspace(-3, 0, n, device=dev), -torch.logspace(-2, 0, n, device=dev)):
        _check_xent(n, d, v, "fp16", dev, h, w, t, g)
    zero = nsa.linear_cross_entropy_backward(h, w, t, torch.zeros(n, device=dev), torch.zeros(n, device=dev))
    assert torch.count_nonzero(zero[0]) == 0 and torch.count_nonzero(zero[1]) == 0
    small = nsa.linear_cross_entropy_backward(h, w, t, nsa.linear_cross_entropy(h, w, t)[1], 1e-42)
    assert torch.count_nonzero(small[0]) == 0 and torch.count_nonzero(small[1]) == 0


# ---------------------------------------------------------------------------
# Refusals of the Python face.
# ---------------------------------------------------------------------------

def test_python_refusals():
    dev = _dev()
    x = torch.randn(8, 64, device=dev)
    ids = torch.zeros(8, dtype=torch.int64, device=dev)
    y, mean, rstd = nsa.layer_norm(x)
    bad_value = [
        lambda: nsa.layer_norm(x.t()),
        lambda: nsa.layer_norm(x.view(2, 4, 64).transpose(0, 1)),
        lambda: nsa.layer_norm(torch.empty(4, 0, device=dev)),
        lambda: nsa.layer_norm(x[:1].expand(8, 64), out=x[:1].expand(8, 64)),
        lambda: nsa.layer_norm(x, weight=torch.ones(63, device=dev)),
        lambda: nsa.layer_norm(x, weight=torch.ones(64)),
        lambda: nsa.layer_norm(x, out=torch.empty(8, 63, device=dev)),
        lambda: nsa.layer_norm_backward(x[:4], x, mean, rstd),
        lambda: nsa.layer_norm_backward(x, x, mean[:4], rstd),
        lambda: nsa.layer_norm_backward(x, x, mean, rstd.cpu()),
        lambda: nsa.layer_norm_backward(x, x, mean, rstd, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
        lambda: nsa.embedding(ids.cpu(), x),
        lambda: nsa.embedding(ids, x.view(2, 4, 64)),
        lambda: nsa.embedding(ids[::2], x),
        lambda: nsa.embedding_backward(ids, x[:4], 5),
        lambda: nsa.embedding_backward(ids, x, 5, accumulate=True),
        lambda: nsa.embedding_backward(ids, x, 5, out=torch.empty(6, 64, device=dev)),
        lambda: nsa.linear_cross_entropy(x, x[:, :32].contiguous(), ids),
        lambda: nsa.linear_cross_entropy(x, x.half(), ids),
        lambda: nsa.linear_cross_entropy(x, x, ids[:4]),
        lambda: nsa.linear_cross_entropy(x, x[:0], ids),
        lambda: nsa.linear_cross_entropy_backward(x, x, ids, mean[:3], 1.0),
        lambda: nsa.linear_cross_entropy_backward(x, x, ids, mean, mean[:3]),
    ]
    for i, call in enumerate(bad_value):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
    bad_type = [
        lambda: nsa.layer_norm(x.double()),
        lambda: nsa.layer_norm(x, weight=torch.ones(64, device=dev).half()),
        lambda: nsa.layer_norm(x, torch.ones(64, device=dev), status=torch.zeros(1, device=dev)),
        lambda: nsa.layer_norm_backward(x, x, mean.double(), rstd),
        lambda: nsa.embedding(ids.float(), x),
        lambda: nsa.linear_cross_entropy(x, x, ids.float()),
        lambda: nsa.linear_cross_entropy_backward(x, x, ids, mean.half(), 1.0),
    ]
    for call in bad_type:
        with pytest.raises(TypeError):
            call()
    with pytest.raises(nsa.NSError):
        nsa.layer_norm(x, eps=-1.0)
    with pytest.raises(nsa.NSError):
        nsa.embedding_backward(ids, x, 0)
    with pytest.raises(nsa.NSError):
        nsa.linear_cross_entropy(x, x, ids, workspace=torch.empty(64, dtype=torch.uint8, device=dev))
    with pytest.raises(nsa.NSError):
        nsa.embedding(ids, x, scale=float("inf"))


# ---------------------------------------------------------------------------
# Streams, graphs and the operators together.
# ---------------------------------------------------------------------------

def _chain(ids, targets, p, ws=None):
    """One training step of a small tied language model: returns the
    gradients of its parameters.  The hidden layer's products are torch's."""
    e = nsa.embedding(ids, p["table"], scale=p["scale"])
    a, m1, r1 = nsa.layer_norm(e, p["w1"], p["b1"])
    hid = torch.mm(a, p["mid"])
    h, m2, r2 = nsa.layer_norm(hid, p["w2"], p["b2"])
    loss, lse = nsa.linear_cross_entropy(h, p["table"], targets)
    dh, dtable = nsa.linear_cross_entropy_backward(h, p["table"], targets, lse, p["g"])
    dhid, dw2, db2 = nsa.layer_norm_backward(dh, hid, m2, r2, p["w2"])
    dmid = torch.mm(a.t().contiguous(), dhid)
    da = torch.mm(dhid, p["mid"].t().contiguous())
    de, dw1, db1 = nsa.layer_norm_backward(da, e, m1, r1, p["w1"])
    nsa.embedding_backward(ids, de, p["table"].shape[0], scale=p["scale"], out=dtable, accumulate=True)
    return {"loss": loss, "dtable": dtable, "dmid": dmid, "dw1": dw1, "db1": db1, "dw2": dw2, "db2": db2}


def _chain_state(n, d, v, dtype, dev, seed=0):
    g = torch.Generator().manual_seed(seed)
    p = {"table": (0.5 * torch.randn(v, d, generator=g)).to(dtype), "mid": (torch.randn(d, d, generator=g) / math.sqrt(d)).to(dtype)}
    for i in ("1", "2"):
        p["w" + i] = 1 + 0.1 * torch.randn(d, generator=g)
        p["b" + i] = 0.1 * torch.randn(d, generator=g)
    ids = torch.randint(0, v, (n,), generator=g)
    targets = torch.randint(0, v, (n,), generator=g)
    targets[::7] = -100
    p["g"] = torch.where(targets >= 0, 1.0 / float((targets >= 0).sum()), 0.0)
    p = {k: t.to(dev) for k, t in p.items()}
    p["scale"] = math.sqrt(d)
    return ids.to(dev), targets.to(dev), p


def test_the_operators_together_against_autograd_in_fp64():
    dev = _dev()
    n, d, v = 96, 64, 130
    ids, targets, p = _chain_state(n, d, v, torch.float32, dev)
    got = _chain(ids, targets, p)
    leaf = {k: t.double().cpu().requires_grad_() for k, t in p.items() if k not in ("scale", "g")}
    F = torch.nn.functional
    x = leaf["table"][ids.cpu()] * p["scale"]
    x = F.layer_norm(x, (d,), leaf["w1"], leaf["b1"], 1e-5) @ leaf["mid"]
    x = F.layer_norm(x, (d,), leaf["w2"], leaf["b2"], 1e-5)
    loss = F.cross_entropy(x @ leaf["table"].t(), targets.cpu(), ignore_index=-100, reduction="none")
    (loss * p["g"].double().cpu()).sum().backward()
    names = {"dtable": "table", "dmid": "mid", "dw1": "w1", "db1": "b1", "dw2": "w2", "db2": "b2"}
    # A chain of six fp32 operators on rows of 64 and sums of up to 130 terms:
    # each adds a few hundred u32 relative to its terms' magnitudes, and the
    # gradients here are sums without large cancellation, so 2^-13 = 2048 u32
    # of each gradient's norm bounds them.
    for name, key in names.items():
        want = leaf[key].grad.numpy()
        err = np.linalg.norm(_np(got[name]) - want) / np.linalg.norm(want)
        print(f"{name}: {err:.2e}", flush=True)
        assert err < 2.0 ** -13, name
    # Against differences: the loss along the whole gradient.
    with torch.no_grad():
        def total(step):
            q = {k: t.detach() + step * leaf[k].grad for k, t in leaf.items()}
            x = q["table"][ids.cpu()] * p["scale"]
            x = F.layer_norm(x, (d,), q["w1"], q["b1"], 1e-5) @ q["mid"]
            x = F.layer_norm(x, (d,), q["w2"], q["b2"], 1e-5)
            per = F.cross_entropy(x @ q["table"].t(), targets.cpu(), ignore_index=-100, reduction="none")
            return float((per * p["g"].double().cpu()).sum())
        step = 1e-4
        slope = (total(step) - total(-step)) / (2 * step)
    dot = sum(float((_np(got[n_]) * leaf[k].grad.numpy()).sum()) for n_, k in names.items())
    # Central differences: relative error of order step^2 times the third
    # derivative over the first; 1e-3 leaves room for a ratio of 1e5.
    assert abs(slope - dot) < 1e-3 * abs(dot)
    # And the hidden matrix takes its Muon step.
    m = torch.zeros_like(p["mid"])
    before = p["mid"].clone()
    nsa.muon_step(p["mid"], got["dmid"].contiguous(), m, lr=0.02)
    torch.cuda.synchronize()
    assert torch.equal(m, got["dmid"]) and not torch.equal(before, p["mid"]) and torch.isfinite(p["mid"]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_operators_on_another_stream_and_captured(dtype):
    dev = _dev()
    ids, targets, p = _chain_state(300, 128, 500, dtype, dev, seed=1)
    want = _chain(ids, targets, p)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = _chain(ids, targets, p)
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(side[k], want[k]), k


def _ops_only(ids, targets, p):
    """The library's own calls of the chain (no library product inside a graph)."""
    e = nsa.embedding(ids, p["table"], scale=p["scale"])
    a, m1, r1 = nsa.layer_norm(e, p["w1"], p["b1"])
    loss, lse = nsa.linear_cross_entropy(a, p["table"], targets)
    dh, dtable = nsa.linear_cross_entropy_backward(a, p["table"], targets, lse, p["g"])
    de, dw1, db1 = nsa.layer_norm_backward(dh, e, m1, r1, p["w1"])
    nsa.embedding_backward(ids, de, p["table"].shape[0], scale=p["scale"], out=dtable, accumulate=True)
    return [loss, lse, dtable, de, dw1, db1]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_captured_steps_replay_equal_to_eager(dtype):
    dev = _dev()
    n, d, v = 500, 192, 700
    ids, targets, p = _chain_state(n, d, v, dtype, dev, seed=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _ops_only(ids, targets, p)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    # Two graphs over the same inputs, each with workspaces of its own.
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = _ops_only(ids, targets, p)
        graphs.append((g, outs))
    for i in range(3):
        new_ids, new_t, new_p = _chain_state(n, d, v, dtype, dev, seed=10 + i)
        ids.copy_(new_ids)
        targets.copy_(new_t)
        for k in p:
            if k != "scale":
                p[k].copy_(new_p[k])
        want = _ops_only(ids, targets, p)
        torch.cuda.synchronize()
        for g, outs in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, outs in graphs:
            for a, b in zip(outs, want):
                assert torch.equal(a, b), i


def test_caller_owned_workspaces():
    dev = _dev()
    ids, targets, p = _chain_state(260, 100, 333, torch.bfloat16, dev, seed=4)
    x = nsa.embedding(ids, p["table"])
    y, mean, rstd = nsa.layer_norm(x)
    loss, lse = nsa.linear_cross_entropy(y, p["table"], targets)
    n, d, v = 260, 100, 333

    def ws(nbytes):
        return torch.full((nbytes + 256,), 255, dtype=torch.uint8, device=dev)  # NaNs

    a = nsa.linear_cross_entropy(y, p["table"], targets, workspace=ws(nsa.linear_cross_entropy_workspace_size(n, d, v, aligned=False)))
    assert torch.equal(a[0], loss) and torch.equal(a[1], lse)
    need = nsa.linear_cross_entropy_workspace_size(n, d, v, aligned=False, backward=True)
    b = nsa.linear_cross_entropy_backward(y, p["table"], targets, lse, p["g"], workspace=ws(need))
    c = nsa.linear_cross_entropy_backward(y, p["table"], targets, lse, p["g"])
    assert torch.equal(b[0], c[0]) and torch.equal(b[1], c[1])
    b = nsa.layer_norm_backward(y, x, mean, rstd, workspace=ws(nsa.layer_norm_workspace_size(n, d)))
    c = nsa.layer_norm_backward(y, x, mean, rstd)
    assert all(torch.equal(i, j) for i, j in zip(b, c))
    b = nsa.embedding_backward(ids, y, v, workspace=ws(nsa.embedding_workspace_size(n, v, d)))
    assert torch.equal(b, nsa.embedding_backward(ids, y, v))
