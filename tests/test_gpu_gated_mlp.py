"""The gated feed-forward block on the GPU against the fp64 oracle.

Bounds are worst cases of the arithmetic, with u32 = 2^-24 and u half a step
of the stored type (bf16 2^-8, fp16 2^-11, fp32 2^-24): a sum of m products
in fp32, in any order, is off by at most (m + 1) u32 times the sum of their
magnitudes; an operand that is rounded is off by u of itself.
"""

import numpy as np
import pytest
import torch

import oracle
import newton_schulz_matrix_amd as nsa
from newton_schulz_matrix_amd import _binding as B

from block_cases import MLP_RUNS

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U32 = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}
ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, want, bound, what):
    got = _np(got).reshape(want.shape)
    off = np.abs(got - want)
    worst = float(np.max(off / np.maximum(bound, 1e-300))) if off.size else 0.0
    print(f"{what}: worst error {worst:.3f} of the bound", flush=True)
    assert np.all(off <= bound), (what, worst)


def _poisoned(shape, dtype, dev):
    return torch.full(shape, float("nan"), dtype=dtype, device=dev)


def _inputs(n, d, f, dtype, dev, seed=0):
    g = torch.Generator().manual_seed(seed)

    def make(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=g)).to(DTYPES[dtype]).to(dev)

    return dict(x=make(n, d, scale=1.5), wg=make(f, d, scale=d ** -0.5), wu=make(f, d, scale=d ** -0.5),
                wd=make(d, f, scale=f ** -0.5), dy=make(n, d))


def _forward_bounds(x, wg, wu, wd, a, b, act, dtype, y, save):
    u, tiny, d, f = HALF_STEP[dtype], TINY[dtype], x.shape[1], wg.shape[0]
    us, ts = HALF_STEP[save], TINY[save]
    ax = np.abs(x)
    ea, eb = (d + 1) * U32 * (ax @ np.abs(wg).T), (d + 1) * U32 * (ax @ np.abs(wu).T)
    value = np.abs(oracle.activation(a, act)[0])
    # Every activation's slope is below 1.13; its value is formed to 8 steps of a.
    eh = 1.13 * ea * (np.abs(b) + eb) + (value + 1.13 * ea) * eb + 8 * U32 * np.abs(a) * np.abs(b)
    h = value * np.abs(b)
    operand = eh + u * (h + eh) + tiny
    ey = operand @ np.abs(wd).T + (f + 1) * U32 * ((h + operand) @ np.abs(wd).T)
    return us * np.abs(a) + (1 + us) * ea + ts, us * np.abs(b) + (1 + us) * eb + ts, u * np.abs(y) + (1 + u) * ey + tiny


def _backward_bounds(o, dy, x, wg, wu, wd, a, b, act, dtype):
    u, tiny, (n, d), f = HALF_STEP[dtype], TINY[dtype], x.shape, wg.shape[0]
    value, slope = (np.abs(v) for v in oracle.activation(a, act))
    aa, ab = np.abs(a), np.abs(b)
    edh = (d + 1) * U32 * (np.abs(dy) @ np.abs(wd))
    dh = np.abs(o["dh"]) + edh
    # Slopes are formed to (8 + 4 |a| + |a|^3) steps of 1 (1 - s next to 1).
    eslope = U32 * (8 + 4 * aa + aa ** 3)
    eda = ab * slope * edh + dh * ab * eslope + 3 * U32 * np.abs(o["da"])
    edb = value * edh + dh * 8 * U32 * aa + 2 * U32 * np.abs(o["db"])
    eda, edb = eda + u * (np.abs(o["da"]) + eda) + tiny, edb + u * (np.abs(o["db"]) + edb) + tiny
    eh = 8 * U32 * aa * ab
    eh = eh + u * (np.abs(o["h"]) + eh) + tiny
    da, db, h = np.abs(o["da"]) + eda, np.abs(o["db"]) + edb, np.abs(o["h"]) + eh

    def final(grad, err):
        return u * np.abs(grad) + (1 + u) * err + tiny

    return {"dx": final(o["dx"], eda @ np.abs(wg) + edb @ np.abs(wu) + (2 * f + 2) * U32 * (da @ np.abs(wg) + db @ np.abs(wu))),
            "dwg": final(o["dwg"], eda.T @ np.abs(x) + (n + 1) * U32 * (da.T @ np.abs(x))),
            "dwu": final(o["dwu"], edb.T @ np.abs(x) + (n + 1) * U32 * (db.T @ np.abs(x))),
            "dwd": final(o["dwd"], np.abs(dy).T @ eh + (n + 1) * U32 * (np.abs(dy).T @ h))}


def _check(n, d, f, dtype, act="silu", strided=0, seed=0, fused=False, save="fp32"):
    dev = _dev()
    print(f"gated mlp {n}x{d}x{f} {dtype} {act} strided {strided} save {save}", flush=True)
    t = _inputs(n, d, f, dtype, dev, seed)
    if strided:
        for name, v in t.items():
            wide = _poisoned((v.shape[0], v.shape[1] + strided), v.dtype, dev)
            wide[:, 1:v.shape[1] + 1] = v
            t[name] = wide[:, 1:v.shape[1] + 1]
    if fused:
        both = torch.cat([t["wg"], t["wu"]])
        t["wg"], t["wu"] = both[:f], both[f:]
    m = {k: _np(v) for k, v in t.items()}
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    w = (t["wg"], t["wu"], t["wd"])
    y, gate, up = nsa.gated_mlp(t["x"], *w, activation=act, status=st, out=_poisoned((n, d), DTYPES[dtype], dev),
                                save=True if save == "fp32" else DTYPES[save])
    assert gate.dtype == up.dtype == DTYPES[save]
    y64, a64, b64, _ = oracle.gated_mlp(m["x"], m["wg"], m["wu"], m["wd"], act)
    ba, bb, by = _forward_bounds(m["x"], m["wg"], m["wu"], m["wd"], a64, b64, act, dtype, y64, save)
    _close(gate, a64, ba, "gate")
    _close(up, b64, bb, "up")
    _close(y, y64, by, "y")
    # The projections are left for backward without changing y.
    alone = nsa.gated_mlp(t["x"], *w, activation=act, save=False)
    assert alone[1] is None and alone[2] is None and torch.equal(alone[0], y)

    outs = dict(out_dx=_poisoned((n, d), y.dtype, dev), out_dw_gate=_poisoned((f, d), y.dtype, dev),
                out_dw_up=_poisoned((f, d), y.dtype, dev), out_dw_down=_poisoned((d, f), y.dtype, dev))
    got = nsa.gated_mlp_backward(t["dy"], t["x"], *w, gate, up, activation=act, status=st, **outs)
    a, b = _np(gate), _np(up)
    o = oracle.gated_mlp_backward(m["dy"], m["x"], m["wg"], m["wu"], m["wd"], a, b, act)
    bounds = _backward_bounds(o, m["dy"], m["x"], m["wg"], m["wu"], m["wd"], a, b, act, dtype)
    for g, name in zip(got, ("dx", "dwg", "dwu", "dwd")):
        _close(g, o[name], bounds[name], name)
    assert int(st.item()) == 0
    # One kind of gradient alone is the same.
    dx, *none = nsa.gated_mlp_backward(t["dy"], t["x"], *w, gate, up, activation=act, need_dw=False)
    assert none == [None] * 3 and torch.equal(dx, got[0])
    none, *dw = nsa.gated_mlp_backward(t["dy"], t["x"], *w, gate, up, activation=act, need_dx=False)
    assert none is None and all(torch.equal(p, q) for p, q in zip(dw, got[1:]))


@pytest.mark.parametrize("n,d,f,dtype", MLP_RUNS)
def test_matches_the_oracle(n, d, f, dtype):
    _check(n, d, f, dtype, seed=n + d + f)


@pytest.mark.parametrize("n,d,f", [(1, 72, 40), (4, 77, 203), (130, 128, 256), (150, 100, 333), (1003, 520, 1407)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_projections_saved_in_the_datas_type(n, d, f, dtype):
    _check(n, d, f, dtype, seed=11, save=dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,d,f", [(2, 96, 70), (150, 192, 320), (300, 200, 700)])
def test_every_activation(n, d, f, dtype, act):
    _check(n, d, f, dtype, act=act, seed=7)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("strided", [0, 64, 3])
@pytest.mark.parametrize("n", [1, 6, 130, 400])
def test_strides_and_weights_that_share_a_tensor(n, strided, dtype):
    _check(n, 128, 320, dtype, strided=strided, seed=3)
    if not strided:
        _check(n, 128, 320, dtype, fused=True, seed=4)


def test_any_rank_and_outputs_given():
    dev = _dev()
    t = _inputs(60, 128, 192, "bf16", dev)
    x, dy = t["x"].view(3, 4, 5, 128), t["dy"].view(3, 4, 5, 128)
    w = (t["wg"], t["wu"], t["wd"])
    y, gate, up = nsa.gated_mlp(x, *w)
    assert y.shape == x.shape and gate.shape == up.shape == (3, 4, 5, 192)
    assert torch.equal(y.view(60, 128), nsa.gated_mlp(t["x"], *w)[0])
    dx = nsa.gated_mlp_backward(dy, x, *w, gate, up)[0]
    assert dx.shape == x.shape
    assert torch.equal(dx.view(60, 128), nsa.gated_mlp_backward(t["dy"], t["x"], *w, gate.view(60, 192), up.view(60, 192))[0])
    # Rows behind a result's last column and rows stay as they were.
    wide = torch.full((64, 150), 7.0, dtype=torch.bfloat16, device=dev)
    nsa.gated_mlp(t["x"], *w, out=wide[2:62, 1:129])
    assert torch.equal(wide[2:62, 1:129], y.view(60, 128))
    wide[2:62, 1:129] = 7.0
    assert bool((wide == 7.0).all())


@pytest.mark.parametrize("n", [1, 50])
def test_gradients_against_differences(n):
    # The call's own forward in fp32, along random directions, central
    # differences of step e in fp64 arithmetic around it: the third
    # derivative's share is of the order e^2 and the forward's rounding
    # (some 2^-20 of the sum's terms) over e.
    dev = _dev()
    t = _inputs(n, 96, 130, "fp32", dev, seed=9)
    names = ("x", "wg", "wu", "wd")
    y, gate, up = nsa.gated_mlp(*(t[k] for k in names), activation="gelu_tanh")
    grads = nsa.gated_mlp_backward(t["dy"], *(t[k] for k in names), gate, up, activation="gelu_tanh")
    gen = torch.Generator().manual_seed(1)
    for name, grad in zip(names, grads):
        direction = torch.randn(t[name].shape, generator=gen).to(dev)
        direction /= direction.norm() / t[name].norm()
        e = 2.0 ** -6

        def value(sign):
            moved = dict(t, **{name: t[name] + sign * e * direction})
            y = nsa.gated_mlp(*(moved[k] for k in names), activation="gelu_tanh", save=False)[0]
            return float((y.double() * t["dy"].double()).sum())

        slope = (value(1) - value(-1)) / (2 * e)
        terms = float((y.double() * t["dy"].double()).abs().sum())
        want = float((grad.double() * direction.double()).sum())
        assert abs(slope - want) <= terms * (2.0 ** -20 / e + 8 * e * e), name


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_no_rows(dtype):
    dev = _dev()
    t = _inputs(0, 40, 24, dtype, dev)
    w = (t["wg"], t["wu"], t["wd"])
    y, gate, up = nsa.gated_mlp(t["x"], *w)
    assert y.shape == (0, 40) and gate.shape == (0, 24)
    got = nsa.gated_mlp_backward(t["dy"], t["x"], *w, gate, up)
    assert got[0].shape == (0, 40) and all(float(g.abs().max()) == 0.0 for g in got[1:])
    assert [g.shape for g in got[1:]] == [w[0].shape, w[1].shape, w[2].shape]


@pytest.mark.parametrize("n,d,f", [(3, 96, 70), (140, 100, 170), (140, 128, 192)])
@pytest.mark.parametrize("where", ["x", "wg", "wu", "wd", "dy"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_non_finite_values_are_reported_and_stay_in_their_rows(n, d, f, where, value):
    dev = _dev()
    t = _inputs(n, d, f, "bf16", dev, seed=5)
    t[where][2, 1] = value
    w = (t["wg"], t["wu"], t["wd"])
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    y, gate, up = nsa.gated_mlp(t["x"], *w, status=st)
    assert bool(st.item()) == (where != "dy")
    rows = [i for i in range(n) if i != 2]
    if where == "x":
        assert torch.isfinite(y[rows].float()).all() and torch.isfinite(gate[rows].float()).all()
    if where == "wd":
        assert torch.isfinite(y[:, [i for i in range(d) if i != 2]].float()).all()
    st.zero_()
    got = nsa.gated_mlp_backward(t["dy"], t["x"], *w, gate, up, status=st)
    assert int(st.item()) == B.NS_ERR_NONFINITE | B.STATUS_AT_OUTPUT
    if where in ("x", "dy"):
        assert torch.isfinite(got[0][rows].float()).all()


def test_a_gate_that_overflows_is_reported():
    # fp16: a = 2^17 is infinite when stored, y = a b Wd with a small b is not.
    dev = _dev()
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    for n in (2, 40):
        x = torch.zeros(n, 64, dtype=torch.float16, device=dev)
        x[:, 0], x[:, 1] = 2.0 ** 9, 2.0 ** -4
        wg, wu = torch.zeros(64, 64, dtype=torch.float16, device=dev), torch.zeros(64, 64, dtype=torch.float16, device=dev)
        wg[:, 0], wu[:, 1] = 2.0 ** 8, 2.0 ** -10
        wd = torch.full((64, 64), 2.0 ** -6, dtype=torch.float16, device=dev)
        st.zero_()
        y, gate, up = nsa.gated_mlp(x, wg, wu, wd, status=st, save=torch.float16)
        assert torch.isfinite(y).all() and torch.isinf(gate).all()
        assert int(st.item()) == B.NS_ERR_NONFINITE | B.STATUS_AT_OUTPUT
        st.zero_()
        for save in (False, True):
            nsa.gated_mlp(x, wg, wu, wd, status=st, save=save)
            assert int(st.item()) == 0


def test_equal_calls_give_equal_bits():
    dev = _dev()
    for n, d, f in ((4, 512, 1000), (300, 1000, 731), (2000, 520, 1407)):
        t = _inputs(n, d, f, "bf16", dev, seed=2)
        w = (t["wg"], t["wu"], t["wd"])
        runs = []
        for _ in range(3):
            y, gate, up = nsa.gated_mlp(t["x"], *w)
            runs.append((y, gate, up) + nsa.gated_mlp_backward(t["dy"], t["x"], *w, gate, up))
        for other in runs[1:]:
            assert all(torch.equal(p, q) for p, q in zip(runs[0], other))


@pytest.mark.parametrize("n,d,f", [(1, 256, 300), (48, 256, 3000), (700, 264, 512)])
def test_captured_and_replayed(n, d, f):
    dev = _dev()
    t = _inputs(n, d, f, "bf16", dev)
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
    for seed in range(3):
        fresh = _inputs(n, d, f, "bf16", dev, 10 + seed)
        for k in t:
            t[k].copy_(fresh[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        assert all(torch.equal(p, q) for p, q in zip(got, step()))


def test_two_streams_with_their_own_workspaces():
    dev = _dev()
    sets = [_inputs(700, 264, 512, "bf16", dev, seed) for seed in (1, 2)]
    want = [nsa.gated_mlp(t["x"], t["wg"], t["wu"], t["wd"])[0] for t in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for k, t in enumerate(sets):
            with torch.cuda.stream(streams[k]):
                got[k].append(nsa.gated_mlp(t["x"], t["wg"], t["wu"], t["wd"])[0])
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(y, want[k]) for y in got[k])


def test_python_refusals():
    dev = _dev()
    t = _inputs(6, 8, 16, "bf16", dev)
    x, wg, wu, wd, dy = t["x"], t["wg"], t["wu"], t["wd"], t["dy"]
    y, gate, up = nsa.gated_mlp(x, wg, wu, wd)
    for args, kw in (((x.cpu(), wg, wu, wd), {}), ((x, wg.cpu(), wu, wd), {}), ((x, wg[:, :7], wu, wd), {}),
                     ((x, wg, wu[:15], wd), {}), ((x, wg, wu, wd.t()), {}), ((x, wg, wu, wd[:7]), {}),
                     ((x, wg.float(), wu, wd), {}), ((x, wg, wu, wd), dict(activation="tanh")),
                     ((x, wg, wu, wd), dict(out=torch.zeros(6, 8, device=dev))), ((x, wg[:0], wu[:0], wd[:, :0]), {}),
                     ((x, wg, wu, wd), dict(workspace=torch.zeros(4096)))):
        with pytest.raises(ValueError):
            nsa.gated_mlp(*args, **kw)
    for bad in (torch.float16, torch.float64):
        with pytest.raises(TypeError):
            nsa.gated_mlp(x, wg, wu, wd, save=bad)
    with pytest.raises(TypeError):
        nsa.gated_mlp_backward(dy, x, wg, wu, wd, gate.half(), up.half())
    with pytest.raises(TypeError):
        nsa.gated_mlp(*(v.double() for v in (x, wg, wu, wd)))
    for args, kw in (((dy[:5], x, wg, wu, wd, gate, up), {}), ((dy.float(), x, wg, wu, wd, gate, up), {}),
                     ((dy, x, wg, wu, wd, gate[:5], up), {}), ((dy, x, wg, wu, wd, gate, up.half()), {}),
                     ((dy, x, wg, wu, wd, gate, torch.zeros(6, 20, device=dev)[:, :16]), {}),
                     ((dy, x, wg, wu, wd, gate, up), dict(out_dw_down=torch.zeros(8, 15, dtype=torch.bfloat16, device=dev)))):
        with pytest.raises(ValueError):
            nsa.gated_mlp_backward(*args, **kw)
    with pytest.raises(nsa.NSError):
        nsa.gated_mlp(x, wg, wu, wd, workspace=torch.zeros(256, dtype=torch.uint8, device=dev)[:100])
