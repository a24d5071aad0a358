"""The norms before and after a block on the GPU against the fp64 oracle.

Bounds are worst cases of the arithmetic, with u32 = 2^-24 and u half a step
of the stored type (bf16 2^-8, fp16 2^-11, fp32 2^-24).
"""

import numpy as np
import pytest
import torch

import oracle
import newton_schulz_matrix_amd as nsa
from newton_schulz_matrix_amd import _binding as B

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TYPES = [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"), ("fp32", "fp32")]
U32 = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}
# Depth of a row sum: up to 24 elements per thread (20 for the longest rows
# here in the looping kernels), six exchanges, sixteen waves, one division.
DEPTH = 56
EPS = 2.0 ** -20
SCALE = 0.75


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _close(got, want, bound, what):
    got = _np(got)
    assert got.shape == want.shape, what
    off = np.abs(got - want)
    worst = float(np.max(off / np.maximum(bound, 1e-300))) if off.size else 0.0
    print(f"{what}: worst error {worst:.3f} of the bound", flush=True)
    assert np.all(off <= bound), (what, worst)


def _poisoned(shape, dtype, dev):
    return torch.full(shape, float("nan"), dtype=dtype, device=dev)


def _inputs(rows, cols, dtype, pdtype, groups, dev, seed):
    g = torch.Generator().manual_seed(seed)

    def make(*shape, to=dtype, scale=1.0, mean=0.0):
        return (mean + scale * torch.randn(*shape, generator=g)).to(DTYPES[to]).to(dev)

    return dict(x=make(rows, cols), z=make(rows, cols, scale=3.0), ds=make(rows, cols), dy=make(rows, cols),
                gate=None if groups is None else make(groups, cols, to=pdtype, scale=0.5, mean=0.5),
                wb=make(cols, to=pdtype, scale=0.1, mean=1.0), w=make(cols, to=pdtype, scale=0.1, mean=1.0))


def _forward_bounds(x, z, gate, wb, w, norm_branch, dtype, s, y, rs):
    rows, cols = x.shape
    g = np.ones((rows, cols)) if gate is None else np.repeat(gate, rows // gate.shape[0], 0)
    wb = np.ones(cols) if wb is None else wb
    w = np.ones(cols) if w is None else w
    rel_rb = (DEPTH / 2 + 4) * U32 if norm_branch else 0.0
    branch = np.abs(s - SCALE * x)
    es = 1.05 * (U32 * (2 * np.abs(SCALE * x) + np.abs(s) + 4 * branch) + rel_rb * branch)
    # The second mean square: the stream's errors weighted by the stream.
    rel_rs = 1.05 * ((np.abs(s) * es).sum(1) / np.maximum((s * s).sum(1), 1e-300) + (DEPTH / 2 + 4) * U32)
    ey = np.abs(w) * rs[:, None] * es + np.abs(y) * (rel_rs[:, None] + 3 * U32)
    u = HALF_STEP[dtype]
    return rel_rb, rel_rs, u * np.abs(s) + (1 + u) * es + TINY[dtype], u * np.abs(y) + (1 + u) * 1.05 * ey + TINY[dtype]


def _backward_bounds(o, ds, dy, s, z, rb, rs, gate, wb, w, dtype, pdtype, per_group, scale=SCALE):
    rows, cols = o["g"].shape
    u, up = HALF_STEP[dtype], HALF_STEP[pdtype]
    w = np.ones(cols) if w is None else w
    wb = np.ones(cols) if wb is None else wb
    eg = U32 * np.abs(o["g"])
    b = {}
    if dy is not None:
        r = rs[:, None]
        shat, uu = np.abs(s * r), np.abs(dy * w)
        m = np.abs(np.mean(s * r * dy * w, 1, keepdims=True))
        em = (DEPTH + 4) * U32 * np.mean(uu * shat, 1, keepdims=True)
        eg = eg + 1.05 * r * (shat * em + U32 * (4 * uu + 5 * shat * m)) + U32 * (0 if ds is None else np.abs(ds))
        b["dw"] = up * np.abs(o["dw"]) + TINY[pdtype] + 1.05 * U32 * (rows + 4) * (np.abs(dy) * shat).sum(0)
    b["dx"] = u * np.abs(o["dx"]) + TINY[dtype] + 1.05 * abs(scale) * (eg + 2 * U32 * np.abs(o["g"]))
    if z is not None:
        r = np.ones((rows, 1)) if rb is None else rb[:, None]
        g = np.ones((rows, cols)) if gate is None else np.repeat(np.abs(gate), rows // gate.shape[0], 0)
        bhat, aw = np.abs(z * r), np.abs(wb)
        a = aw * g * np.abs(o["g"])
        ea = aw * g * eg + 3 * U32 * a
        ez = ea
        if rb is not None:
            sign = np.sign(z) * bhat
            m2 = np.abs(np.mean(wb * (np.ones(1) if gate is None else np.repeat(gate, rows // gate.shape[0], 0)) * o["g"] * sign, 1, keepdims=True))
            em2 = np.mean(bhat * ea, 1, keepdims=True) + (DEPTH + 4) * U32 * np.mean(a * bhat, 1, keepdims=True)
            ez = r * (ea + bhat * em2 + U32 * (4 * a + 5 * bhat * m2))
        b["dz"] = u * np.abs(o["dz"]) + TINY[dtype] + 1.1 * ez
        terms, eterms = np.abs(o["dgate"]), bhat * aw * eg + 4 * U32 * np.abs(o["dgate"])
        if gate is not None:
            groups = gate.shape[0]
            total = o["dgate"].reshape(groups, -1, cols).sum(1)
            b["dgate"] = (up * np.abs(total) + TINY[pdtype]
                          + 1.1 * (eterms + U32 * per_group * terms).reshape(groups, -1, cols).sum(1))
        b["dwb"] = (up * np.abs(o["dwb"]) + TINY[pdtype]
                    + 1.1 * (g * bhat * eg + U32 * (rows + 5) * g * bhat * np.abs(o["g"])).sum(0))
    return b


def _check(rows, cols, dtype, pdtype, groups, norm_branch=True, use=("gate", "wb", "w"), ds=True, dy=True, strided=False,
           seed=0):
    dev = _dev()
    print(f"residual norm {rows}x{cols} {dtype}/{pdtype} groups {groups} norm_branch {norm_branch} {use}", flush=True)
    t = _inputs(rows, cols, dtype, pdtype, groups, dev, seed)
    for name in ("gate", "wb", "w"):
        if name not in use:
            t[name] = None
    if strided:
        for name in ("x", "z", "ds", "dy"):
            wide = _poisoned((rows, cols + 3), t[name].dtype, dev)
            wide[:, 1:cols + 1] = t[name]
            t[name] = wide[:, 1:cols + 1]
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    n = {k: _np(v) for k, v in t.items()}
    s, y, rb, rs = nsa.residual_norm(t["x"], t["z"], gate=t["gate"], scale=SCALE, branch_weight=t["wb"], weight=t["w"],
                                     norm_branch=norm_branch, eps=EPS, status=st,
                                     out=_poisoned((rows, cols), t["x"].dtype, dev),
                                     out_norm=_poisoned((rows, cols), t["x"].dtype, dev))
    s64, y64, rb64, rs64 = oracle.residual_norm(n["x"], n["z"], n["gate"], SCALE, n["wb"], n["w"], norm_branch, EPS)
    rel_rb, rel_rs, bs, by = _forward_bounds(n["x"], n["z"], n["gate"], n["wb"], n["w"], norm_branch, dtype, s64, y64, rs64)
    if norm_branch:
        _close(rb, rb64, rel_rb * rb64, "branch_rstd")
    else:
        assert rb is None
    _close(rs, rs64, rel_rs * rs64, "rstd")
    _close(s, s64, bs, "stream")
    _close(y, y64, by, "normed")

    dst, dyt = t["ds"] if ds else None, t["dy"] if dy else None
    w = t["w"] if dy else None
    got = nsa.residual_norm_backward(dst, dyt, s, t["z"], rb, rs if dy else None, gate=t["gate"], scale=SCALE,
                                     branch_weight=t["wb"], weight=w, status=st,
                                     out=_poisoned((rows, cols), s.dtype, dev),
                                     out_branch=_poisoned((rows, cols), s.dtype, dev))
    sn, rbn, rsn = _np(s), _np(rb), _np(rs)
    dsn, dyn = n["ds"] if ds else None, n["dy"] if dy else None
    o = oracle.residual_norm_backward(dsn, dyn, sn, n["z"], rbn, rsn, n["gate"], SCALE, n["wb"], _np(w))
    per_group = rows // (groups or 1) + 8
    b = _backward_bounds(o, dsn, dyn, sn, n["z"], rbn, rsn, n["gate"], n["wb"], _np(w), dtype, pdtype, per_group)
    _close(got[0], o["dx"], b["dx"], "dresidual")
    _close(got[1], o["dz"], b["dz"], "dbranch")
    if t["gate"] is not None:
        _close(got[2], o["dgate"].reshape(groups, -1, cols).sum(1), b["dgate"], "dgate")
    if t["wb"] is not None:
        _close(got[3], o["dwb"], b["dwb"], "dbranch_weight")
    if w is not None:
        _close(got[4], o["dw"], b["dw"], "dweight")
    assert [g is None for g in got[2:]] == [t["gate"] is None, t["wb"] is None, w is None]
    assert int(st.item()) == 0


# Row widths: the widest of every kernel build in vectors of 16 bytes (8
# 16-bit or 4 fp32 elements), whole and ragged, less than a vector, too long.
WIDTHS = [1, 3, 4, 5, 8, 64, 97, 256, 257, 384, 500, 512, 513, 768, 769, 1000, 1024, 1025, 1536, 1537, 2048, 2049, 4096, 4097, 8192,
          8193, 20001]


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dtype,pdtype", TYPES)
def test_matches_the_oracle_at_every_width(cols, dtype, pdtype):
    rows = 40 if cols < 3000 else 6
    _check(rows, cols, dtype, pdtype, 2, seed=cols)


@pytest.mark.parametrize("rows,groups", [(1, 1), (2, 2), (7, 7), (7, 1), (60, 60), (60, 20), (600, 1), (600, 3), (3000, 1500),
                                         (1030, 1030), (4200, 600), (2048, 512)])
@pytest.mark.parametrize("cols", [40, 6, 9000])
@pytest.mark.parametrize("dtype,pdtype", [("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
def test_gates_shared_by_any_number_of_rows(rows, groups, cols, dtype, pdtype):
    if cols == 9000 and rows > 700:
        rows, groups = 520 * (rows // groups if rows > groups else 1), 520
        if rows > 1100:
            rows, groups = 1040, 520
    _check(rows, cols, dtype, pdtype, groups, seed=rows)


@pytest.mark.parametrize("cols", [768, 1001, 5, 8200])
@pytest.mark.parametrize("kw", [dict(norm_branch=False), dict(use=()), dict(use=("w",)), dict(use=("gate",)),
                                dict(use=("wb",), norm_branch=False), dict(ds=False), dict(dy=False),
                                dict(dy=False, use=(), norm_branch=False), dict(strided=True)])
def test_parts_that_are_left_out(cols, kw):
    for dtype, pdtype in (("bf16", "bf16"), ("fp32", "fp32"), ("fp16", "fp32")):
        _check(9, cols, dtype, pdtype, 3 if "gate" in kw.get("use", ("gate",)) else None, seed=cols, **kw)


@pytest.mark.parametrize("cols", [64, 1001, 3, 8200])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_a_norm_alone(cols, dtype):
    dev = _dev()
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(2, 5, cols, generator=g).to(DTYPES[dtype]).to(dev)
    w = (1 + 0.1 * torch.randn(cols, generator=g)).to(DTYPES[dtype]).to(dev)
    dy, ds = torch.randn(2, 5, cols, generator=g).to(x), torch.randn(2, 5, cols, generator=g).to(x)
    stream, y, rb, rs = nsa.residual_norm(x, weight=w, eps=EPS)
    assert stream is x and rb is None and rs.shape == (2, 5)
    x64 = _np(x).reshape(10, cols)
    _, y64, _, rs64 = oracle.residual_norm(x64, None, weight=_np(w), eps=EPS)
    rel = (DEPTH / 2 + 4) * U32
    _close(rs.view(-1), rs64, rel * rs64, "rstd")
    _close(y.view(10, cols), y64, (HALF_STEP[dtype] + rel + 4 * U32) * np.abs(y64) + TINY[dtype], "normed")
    for d in (None, ds):
        dx, dz, dgate, dwb, dw = nsa.residual_norm_backward(d, dy, x, rstd=rs, weight=w)
        assert dz is None and dgate is None and dwb is None
        rs2, d64 = _np(rs).reshape(-1), None if d is None else _np(d).reshape(10, cols)
        o = oracle.residual_norm_backward(d64, _np(dy).reshape(10, cols), x64, None, None, rs2, weight=_np(w))
        b = _backward_bounds(o, d64, _np(dy).reshape(10, cols), x64, None, None, rs2, None, None, _np(w), dtype, dtype, 1, 1.0)
        _close(dx.view(10, cols), o["dx"], b["dx"], "dresidual")
        _close(dw, o["dw"], b["dw"], "dweight")


@pytest.mark.parametrize("cols", [72, 1001, 8200])
def test_results_written_over_inputs(cols):
    dev = _dev()
    t = _inputs(50, cols, "bf16", "bf16", 5, dev, 3)
    kw = dict(gate=t["gate"], scale=SCALE, branch_weight=t["wb"], weight=t["w"])
    s, y, rb, rs = nsa.residual_norm(t["x"], t["z"], **kw)
    x, z = t["x"].clone(), t["z"].clone()
    s2, y2, _, _ = nsa.residual_norm(x, z, out=x, out_norm=z, **kw)
    assert s2 is x and y2 is z and torch.equal(s, x) and torch.equal(y, z)
    want = nsa.residual_norm_backward(t["ds"], t["dy"], s, t["z"], rb, rs, **kw)
    ds, dy = t["ds"].clone(), t["dy"].clone()
    got = nsa.residual_norm_backward(ds, dy, s, t["z"], rb, rs, out=ds, out_branch=dy, **kw)
    assert got[0] is ds and got[1] is dy
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [64, 1001, 3, 8200])
def test_no_rows(cols):
    dev = _dev()
    x = torch.zeros(0, cols, device=dev)
    gate = torch.ones(3, cols, device=dev)
    w = torch.ones(cols, device=dev)
    s, y, rb, rs = nsa.residual_norm(x, x.clone(), gate=gate, branch_weight=w, weight=w)
    assert s.shape == y.shape == (0, cols) and rb.numel() == rs.numel() == 0
    got = nsa.residual_norm_backward(x, x.clone(), s, x.clone(), rb, rs, gate=gate, branch_weight=w, weight=w)
    assert got[2].shape == (3, cols) and all(float(g.abs().max()) == 0.0 for g in got[2:])


@pytest.mark.parametrize("cols", [64, 1001, 8200])
@pytest.mark.parametrize("where", ["x", "z", "gate", "ds", "dy"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_non_finite_values_are_reported_and_stay_in_their_row(cols, where, value):
    dev = _dev()
    t = _inputs(12, cols, "bf16", "fp32", 12, dev, 1)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    t[where][5, cols // 2] = value
    kw = dict(gate=t["gate"], branch_weight=t["wb"], weight=t["w"], status=st)
    s, y, rb, rs = nsa.residual_norm(t["x"], t["z"], **kw)
    assert bool(st.item()) == (where in ("x", "z", "gate"))
    keep = [i for i in range(12) if i != 5]
    assert torch.isfinite(s[keep].float()).all() and torch.isfinite(y[keep].float()).all()
    st.zero_()
    dx, dz, dgate, dwb, dw = nsa.residual_norm_backward(t["ds"], t["dy"], s, t["z"], rb, rs, **kw)
    assert int(st.item()) == B.NS_ERR_NONFINITE | B.STATUS_AT_OUTPUT
    for g in (dx, dz, dgate):
        assert torch.isfinite(g[keep].float()).all()


@pytest.mark.parametrize("cols", [64, 8200])
def test_squares_past_fp32_are_reported(cols):
    dev = _dev()
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    x, z = torch.ones(3, cols, device=dev), torch.ones(3, cols, device=dev)
    z[1] = 1e25
    nsa.residual_norm(x, z, status=st, norm_out=False)
    assert int(st.item()) == B.NS_ERR_NONFINITE | B.STATUS_AT_OUTPUT
    # A row of zeros is finite: rstd is 1 / sqrt(eps).
    st.zero_()
    s, y, rb, rs = nsa.residual_norm(torch.zeros_like(x), torch.zeros_like(z), status=st)
    assert int(st.item()) == 0 and float(y.abs().max()) == 0 and float(rb[0]) == pytest.approx(1e3, rel=1e-6)


def test_equal_calls_give_equal_bits():
    dev = _dev()
    t = _inputs(5000, 768, "bf16", "fp32", 10, dev, 2)
    kw = dict(gate=t["gate"], branch_weight=t["wb"], weight=t["w"])
    runs = []
    for _ in range(3):
        s, y, rb, rs = nsa.residual_norm(t["x"], t["z"], **kw)
        runs.append((s, y, rb, rs) + nsa.residual_norm_backward(t["ds"], t["dy"], s, t["z"], rb, rs, **kw))
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_captured_and_replayed():
    dev = _dev()
    t = _inputs(300, 1001, "bf16", "bf16", 3, dev, 2)
    kw = dict(gate=t["gate"], branch_weight=t["wb"], weight=t["w"])

    def step():
        s, y, rb, rs = nsa.residual_norm(t["x"], t["z"], **kw)
        return (s, y, rb, rs) + nsa.residual_norm_backward(t["ds"], t["dy"], s, t["z"], rb, rs, **kw)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        fresh = _inputs(300, 1001, "bf16", "bf16", 3, dev, 10 + seed)
        for k in t:
            t[k].copy_(fresh[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_python_refusals():
    dev = _dev()
    x, z = torch.zeros(6, 8, device=dev), torch.zeros(6, 8, device=dev)
    w, gate, r = torch.ones(8, device=dev), torch.ones(2, 8, device=dev), torch.ones(6, device=dev)
    half = w.half()
    for kw in (dict(branch=z[:5]), dict(branch=z.half()), dict(branch=z.cpu()), dict(gate=gate), dict(branch_weight=w),
               dict(scale=2.0), dict(norm_out=False), dict(out=x.clone()), dict(branch=z, gate=torch.ones(4, 8, device=dev)),
               dict(branch=z, gate=torch.ones(2, 7, device=dev)), dict(branch=z, gate=torch.ones(0, 8, device=dev)),
               dict(branch=z, weight=w[:7]), dict(branch=z, out=x[:5]), dict(branch=z.t().contiguous().t())):
        with pytest.raises(ValueError):
            nsa.residual_norm(x, **kw)
    for kw in (dict(weight=half), dict(branch=z, gate=gate.half()), dict(branch=z, weight=w.double())):
        with pytest.raises(TypeError):
            nsa.residual_norm(x, **kw)
    with pytest.raises(TypeError):
        nsa.residual_norm(x.half(), z.half(), branch_weight=half, weight=w)
    with pytest.raises(nsa.NSError):
        nsa.residual_norm(x, z, eps=-1.0)
    back = nsa.residual_norm_backward
    for args, kw in (((None, None, x), {}), ((x, x, x), {}), ((x, None, x), dict(weight=w)), ((x, None, x), dict(gate=gate)),
                     ((x, None, x), dict(scale=0.5)), ((x[:5], None, x), {}), ((x, x.half(), x), dict(rstd=r)),
                     ((x, x, x, z), dict(rstd=r[:5])), ((x, None, x, z, r[:5]), {}), ((x, None, x), dict(out_branch=z)),
                     ((x, None, x, z), dict(workspace=torch.empty(16, device="cpu")))):
        with pytest.raises(ValueError):
            back(*args, **kw)
    with pytest.raises(nsa.NSError):
        back(x, None, x, z, workspace=torch.empty(300, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError, match="device tensor"):
        nsa.residual_norm(x.cpu())
