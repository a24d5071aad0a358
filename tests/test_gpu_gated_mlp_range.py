"""The gated feed-forward block far from one: activations of the largest
numbers, and fp16 operands of the products that are past fp16's numbers, above
or below.
"""

import numpy as np
import pytest
import torch

import oracle
import newton_schulz_matrix_amd as nsa
from test_gpu_gated_mlp import ACTS, DTYPES, HALF_STEP, U32, _close, _dev, _inputs, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_activations_of_any_finite_number(act, dtype):
    # One column of a gate for each size.  Both value and slope end at 0 on the
    # left and at a and 1 on the right, exactly from |a| = 128 on, where exp(-|a|)
    # is below fp32's smallest number.
    dev = _dev()
    print(f"activation {act} {dtype}", flush=True)
    sizes = np.array([128, 1e3, 1e6, 1e12, 1.1e13, 1.3e13, 1e14, 1e18, 1e19, 2e19, 1e25, 1e30, 1e38, 3.3e38])
    a = torch.tensor(np.concatenate([-sizes, sizes])).to(DTYPES[dtype]).to(dev)
    n, d, f = 130, 72, a.numel()
    x = torch.zeros(n, d, dtype=DTYPES[dtype], device=dev)
    x[:, 0], x[:, 1] = 1.0, 2.0 ** -100
    wg, wu = torch.zeros(f, d, dtype=x.dtype, device=dev), torch.zeros(f, d, dtype=x.dtype, device=dev)
    wg[:, 0], wu[:, 1] = a, 1.0
    wd = torch.zeros(d, f, dtype=x.dtype, device=dev)
    wd[:f] = torch.eye(f, device=dev, dtype=x.dtype)
    dy = torch.ones(n, d, dtype=x.dtype, device=dev)
    right = (a > 0).to(x.dtype)
    for rows in (2, n):
        y, gate, up = nsa.gated_mlp(x[:rows], wg, wu, wd, activation=act)
        assert torch.equal(gate[0], a.float()) and bool((up == 2.0 ** -100).all())
        # h = 2^-100 act(a): exact, and its sum has one term.
        assert torch.equal(y[:, :f].float(), (a * right * 2.0 ** -100).float().expand(rows, f))
    up = torch.full_like(gate, 0.5)
    dx, dwg, dwu, dwd = nsa.gated_mlp_backward(dy, x, wg, wu, wd, gate, up, activation=act, need_dx=False)
    # da = b slope, db = value: sums of n equal terms, of powers of two times
    # the values' digits, in fp32 (a sum of 130 terms is off by 131 u32).
    big = a.double() * right.double() * (n * 2.0 ** -100)
    assert torch.equal(dwg[:, 0].double(), right.double() * 0.5 * n)
    u = HALF_STEP[dtype]
    assert ((dwu[:, 1].double() - big).abs() <= (u + 132 * U32) * big).all()


# ---------------------------------------------------------------------------
# fp16: the products' own operands h, da and db beyond the type's numbers.
# ---------------------------------------------------------------------------
TINY = 2.0 ** -25
# The last three: several tiles a work-group in each launch, and the largest
# tiles (tests/test_block_builds_host.py checks that every fp16 build is reached).
SHAPES = [(5, 64, 128), (9, 72, 136), (40, 192, 320), (48, 256, 1411), (130, 128, 256), (300, 200, 703), (700, 264, 512), (1003, 520, 1407),
          (3000, 264, 3001), (3000, 1536, 264), (700, 264, 3001)]


def _unit(peak):
    """Half the smallest step that a row (or all) of an operand is held in:
    fp16's own between 2^-10 and its largest number; outside, the peak is taken
    to [2^14, 2^15)."""
    scaled = peak * 2.0 ** -39
    inside = (peak >= 2.0 ** -10 * 0.99) & (peak <= 65504 * 1.01)
    return np.where(inside, np.maximum(TINY, scaled), np.where(peak == 0, TINY, scaled))


def _range_inputs(n, d, f, dev, kind, seed=0):
    t = _inputs(n, d, f, "fp16", dev, seed)
    rows = slice(2, 3) if kind.endswith("row") else slice(None)
    if kind in ("large", "large row"):
        # |a| and |b| some 2^10: h past 2^16, y well inside.
        t["x"][rows] *= 2.0 ** 10
        t["wd"] *= 2.0 ** -10
    elif kind.startswith("tiny"):
        t["x"][rows] *= 2.0 ** -8
        t["wg"] *= 2.0 ** -5
        t["wu"] *= 2.0 ** -5
        t["wd"] *= 2.0 ** 8
    elif kind.startswith("small dy"):
        t["dy"][rows] *= 2.0 ** -20
        t["x"] *= 2.0 ** 6
        t["wg"] *= 2.0 ** -6
        t["wu"] *= 2.0 ** -6
    elif kind.startswith("large dy"):
        # da and db some 2^15 and more, h some 2^-20, results inside the type.
        t["dy"][rows] *= 2.0 ** 12
        t["x"] *= 2.0 ** -6
        t["wg"] *= 2.0 ** -4
        t["wu"] *= 2.0 ** -4
        t["wd"] *= 2.0 ** 13
    return t


def _forward(t, act, save=True, **kw):
    return nsa.gated_mlp(t["x"], t["wg"], t["wu"], t["wd"], activation=act, save=save, **kw)


@pytest.mark.parametrize("kind", ["large", "large row", "tiny", "tiny row"])
@pytest.mark.parametrize("n,d,f", SHAPES)
def test_fp16_products_of_h_past_the_type(n, d, f, kind):
    dev = _dev()
    act = "silu"
    print(f"fp16 forward {n}x{d}x{f} {kind}", flush=True)
    t = _range_inputs(n, d, f, dev, kind, seed=n)
    m = {k: _np(v) for k, v in t.items()}
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    y, gate, up = _forward(t, act, status=st)
    assert int(st.item()) == 0
    y64, a, b, h = oracle.gated_mlp(m["x"], m["wg"], m["wu"], m["wd"], act)
    if kind == "large":
        assert np.abs(h).max() > 65536
    u, ax = HALF_STEP["fp16"], np.abs(m["x"])
    ea, eb = (d + 1) * U32 * (ax @ np.abs(m["wg"]).T), (d + 1) * U32 * (ax @ np.abs(m["wu"]).T)
    value = np.abs(oracle.activation(a, act)[0])
    eh = 1.13 * ea * (np.abs(b) + eb) + (value + 1.13 * ea) * eb + 8 * U32 * np.abs(a * b)
    operand = eh + u * (np.abs(h) + eh) + _unit(np.abs(h).max(1, keepdims=True))
    wd = np.abs(m["wd"]).T
    ey = operand @ wd + (f + 1) * U32 * ((np.abs(h) + operand) @ wd)
    _close(y, y64, u * np.abs(y64) + (1 + u) * ey + TINY, "y")
    # A row in range does not depend on the others.
    if kind.endswith("row"):
        rest = [i for i in range(n) if i != 2]
        t["x"][2] = 0
        assert torch.equal(_forward(t, act)[0][rest], y[rest])
    again = _forward(t, act, save=False)[0]
    assert torch.equal(again[3:], y[3:])


def test_a_row_is_finite_alone_and_among_others():
    # The few-row form keeps h in fp32; a batch's rows are as finite.
    dev = _dev()
    t = _range_inputs(64, 128, 256, dev, "large")
    for n in (1, 4, 5, 8, 9, 64):
        y = nsa.gated_mlp(t["x"][:n], t["wg"], t["wu"], t["wd"])[0]
        assert torch.isfinite(y).all(), n


@pytest.mark.parametrize("kind", ["large", "large row", "tiny", "small dy", "small dy row", "large dy", "large dy row"])
@pytest.mark.parametrize("n,d,f", SHAPES)
def test_fp16_gradients_of_operands_past_the_type(n, d, f, kind):
    dev = _dev()
    act = "gelu"
    print(f"fp16 backward {n}x{d}x{f} {kind}", flush=True)
    t = _range_inputs(n, d, f, dev, kind, seed=n + 1)
    if kind in ("large", "large row"):
        t["dy"] *= 2.0 ** -14
    m = {k: _np(v) for k, v in t.items()}
    _, gate, up = _forward(t, act)
    a, b = _np(gate), _np(up)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    got = nsa.gated_mlp_backward(t["dy"], t["x"], t["wg"], t["wu"], t["wd"], gate, up, activation=act, status=st)
    o = oracle.gated_mlp_backward(m["dy"], m["x"], m["wg"], m["wu"], m["wd"], a, b, act)
    u = HALF_STEP["fp16"]
    value, slope = (np.abs(v) for v in oracle.activation(a, act))
    aa, ab, dy, x = np.abs(a), np.abs(b), np.abs(m["dy"]), np.abs(m["x"])
    edh = (d + 1) * U32 * (dy @ np.abs(m["wd"]))
    dh = np.abs(o["dh"]) + edh
    # Slopes are formed to 8 + 4 |a| + |a|^3 steps while they still change.
    eslope = U32 * (8 + 4 * np.minimum(aa, 16) + np.minimum(aa, 16) ** 3)
    eda = ab * slope * edh + dh * ab * eslope + 3 * U32 * np.abs(o["da"])
    edb = value * edh + dh * 8 * U32 * aa + 2 * U32 * np.abs(o["db"])
    eh = 8 * U32 * aa * ab
    zpeak = np.maximum(np.abs(o["da"]), np.abs(o["db"])).max(1, keepdims=True)

    def held(x, e, unit):
        return e + u * (np.abs(x) + e) + unit

    def sums(parts, count, result):
        err = sum(ep @ q + (count + 1) * U32 * ((np.abs(p) + ep) @ q) for p, ep, q in parts)
        return u * np.abs(result) + (1 + u) * err + TINY

    rows, every, hs = _unit(zpeak), _unit(zpeak.max()), _unit(np.abs(o["h"]).max())
    dar, dbr = held(o["da"], eda, rows), held(o["db"], edb, rows)
    dae, dbe, he = held(o["da"], eda, every), held(o["db"], edb, every), held(o["h"], eh, hs)
    bounds = {"dx": sums([(o["da"], dar, np.abs(m["wg"])), (o["db"], dbr, np.abs(m["wu"]))], 2 * f, o["dx"]),
              "dwg": sums([(o["da"].T, dae.T, x)], n, o["dwg"]), "dwu": sums([(o["db"].T, dbe.T, x)], n, o["dwu"]),
              "dwd": sums([(o["h"].T, he.T, dy)], n, o["dwd"].T).T}
    for g, name in zip(got, ("dx", "dwg", "dwu", "dwd")):
        # Results past the type are infinite, as they should be; of the oracle's
        # more than half are within it (0.61 of dw_gate at 3000 x 1536 x 264).
        fits = np.abs(o[name]) < 65000
        assert fits.mean() > 0.5, name
        _close(g[torch.from_numpy(fits).to(dev)], o[name][fits], bounds[name][fits], name)
    assert int(st.item()) == 0 or not all((np.abs(o[k]) < 65000).all() for k in ("dx", "dwg", "dwu", "dwd"))
    dx, *_ = nsa.gated_mlp_backward(t["dy"], t["x"], t["wg"], t["wu"], t["wd"], gate, up, activation=act, need_dw=False)
    _, *dw = nsa.gated_mlp_backward(t["dy"], t["x"], t["wg"], t["wu"], t["wd"], gate, up, activation=act, need_dx=False)
    assert torch.equal(dx, got[0]) and all(torch.equal(p, q) for p, q in zip(dw, got[1:]))


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_fp16_non_finite_rows_change_no_other_row(value):
    dev = _dev()
    t = _range_inputs(140, 128, 192, dev, "large")
    w = (t["wg"], t["wu"], t["wd"])
    rest = [i for i in range(140) if i != 2]
    want, gate, up = nsa.gated_mlp(t["x"], *w)
    dx = nsa.gated_mlp_backward(t["dy"], t["x"], *w, gate, up, need_dw=False)[0]
    t["x"][2] = value
    y, gate, up = nsa.gated_mlp(t["x"], *w)
    assert torch.equal(y[rest], want[rest])
    got = nsa.gated_mlp_backward(t["dy"], t["x"], *w, gate, up, need_dw=False)[0]
    assert torch.equal(got[rest], dx[rest])


def test_fp16_range_captured_and_replayed():
    # The same graph over inputs inside and outside the type's range.
    dev = _dev()
    n, d, f = 300, 200, 703
    t = _range_inputs(n, d, f, dev, "")
    w = (t["wg"], t["wu"], t["wd"])

    def step():
        y, gate, up = nsa.gated_mlp(t["x"], *w)
        return (y, gate, up) + nsa.gated_mlp_backward(t["dy"], t["x"], *w, gate, up)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i, kind in enumerate(("", "large row", "", "small dy", "large", "large dy row", "")):
        fresh = _range_inputs(n, d, f, dev, kind, seed=20 + i)
        for k in t:
            t[k].copy_(fresh[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        want = step()
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(got, want)), kind


def test_fp16_range_on_two_streams():
    dev = _dev()
    sets = [_range_inputs(300, 200, 703, dev, kind, seed=i) for i, kind in enumerate(("large row", "small dy"))]

    def step(t):
        w = (t["wg"], t["wu"], t["wd"])
        y, gate, up = nsa.gated_mlp(t["x"], *w)
        return (y, gate, up) + nsa.gated_mlp_backward(t["dy"], t["x"], *w, gate, up)

    want = [step(t) for t in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for k, t in enumerate(sets):
            with torch.cuda.stream(streams[k]):
                got.append((k, step(t)))
    torch.cuda.synchronize()
    for k, out in got:
        assert all(torch.equal(p, q) for p, q in zip(out, want[k]))
