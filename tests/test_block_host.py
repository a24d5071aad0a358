"""AdamW, residual norms and the gated feed-forward block without a device:
the oracle's pins, the workspace queries and every refusal of the C entry
points (made on the host before anything is enqueued; no device pointer is
dereferenced)."""

import ctypes
import os
import struct

import numpy as np
import pytest
import torch

import oracle
import newton_schulz_matrix_amd as nsa
from newton_schulz_matrix_amd import _binding as B

built = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libnsortho.so not built")

INV, DT, WSP = 1, 2, 3
PTR = 1 << 20  # stands for a device pointer
ENTRY = struct.Struct("=6Qq2f4i")  # ns_adamw_tensor


# ---------------------------------------------------------------------------
# AdamW.
# ---------------------------------------------------------------------------

def test_oracle_adamw_against_closed_forms():
    g, p = np.array([0.5, -2.0, 0.0]), np.array([1.0, 1.0, 1.0])
    m = v = np.zeros(3)
    q = p
    for t in range(1, 6):
        before = q
        q, m, v = oracle.adamw(q, g, m, v, 0.01, t, (0.9, 0.99), 1e-30, 0.0)
        # A constant gradient: the corrected moments are g and g^2.
        assert np.allclose(m, (1 - 0.9 ** t) * g) and np.allclose(v, (1 - 0.99 ** t) * g * g)
        assert np.allclose(q, before - 0.01 * np.sign(g))
    q, _, _ = oracle.adamw(p, 0 * g, 0 * p, 0 * p, 0.01, 1, weight_decay=0.5)
    assert np.allclose(q, p * (1 - 0.005))
    q, m, v = oracle.adamw(p, 4 * g, 0 * p, 0 * p, 0.01, 1, grad_scale=0.25)
    assert np.allclose(m, 0.1 * g) and np.allclose(v, 0.05 * g * g)


def _adamw(beta1=0.9, beta2=0.95, eps=1e-8, step=1, d_step=None, count=1, table=True, **kw):
    e = dict(param=PTR, grad=PTR, m=PTR, v=PTR, scales=0, copy=0, numel=10, lr=1e-3, wd=0.1, pt=0, gt=0, ct=0, zero=0)
    e.update(kw)
    raw = bytearray(ENTRY.pack(*(e[k] or 0 for k in ("param", "grad", "m", "v", "scales", "copy", "numel", "lr",
                                                              "wd", "pt", "gt", "ct", "zero"))))
    arr = bytes(raw) if table else None
    return B.lib().ns_adamw_step(arr, count, beta1, beta2, eps, step, d_step, None, None, None, None)


@built
def test_adamw_refusals():
    for name in ("param", "grad", "m", "v"):
        assert _adamw(**{name: None}) == INV, name
    for kw in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=-1e-9),
               dict(eps=float("inf")), dict(step=0), dict(step=-3), dict(count=-1), dict(table=False), dict(numel=-1),
               dict(numel=(1 << 40) + 1), dict(lr=float("nan")), dict(wd=float("inf")), dict(zero=1)):
        assert _adamw(**kw) == INV, kw
    assert _adamw(pt=3) == DT and _adamw(gt=7) == DT and _adamw(copy=PTR, ct=3) == DT
    # Nothing to do: no launch.
    assert _adamw(count=0, table=False) == 0
    assert _adamw(numel=0, param=None, grad=None, m=None, v=None) == 0


@built
def test_adamw_table_entry_has_the_headers_layout():
    text = open(os.path.join(os.path.dirname(B.PKG), "include", "nsortho.h")).read()
    body = text[text.index("typedef struct ns_adamw_tensor {"):text.index("} ns_adamw_tensor;")]
    names = [line.split()[-1].rstrip(";").lstrip("*") for line in body.splitlines()[1:] if line.strip()]
    assert names == ["param", "grad", "exp_avg", "exp_avg_sq", "scales", "copy", "numel", "lr", "weight_decay",
                     "param_dtype", "grad_dtype", "copy_dtype", "reserved"]
    assert ENTRY.size == 6 * 8 + 8 + 2 * 4 + 4 * 4


def test_adamw_states_and_host_tensors():
    p = [torch.zeros(3, 100), torch.zeros(0), torch.zeros(1)]
    m, v, scales = nsa.adamw_states(p)
    assert scales is None and all(t.dtype == torch.float32 and t.shape == q.shape for t, q in zip(m + v, p + p))
    m, v, scales = nsa.adamw_states(p, bits=8)
    assert [tuple(s.shape) for s in scales] == [(2, 2), (2, 0), (2, 1)]
    assert all(t.dtype == torch.float8_e4m3fn for t in m + v)
    with pytest.raises(ValueError, match="device tensor"):
        nsa.adamw_step(p, p, m, v, lr=1e-3, step=1, scales=scales)


# ---------------------------------------------------------------------------
# Norms before and after a block.
# ---------------------------------------------------------------------------

def _slope(f, x, direction, step=1e-5):
    return (f(x + step * direction) - f(x - step * direction)) / (2 * step)


@pytest.mark.parametrize("norm_branch", [True, False])
@pytest.mark.parametrize("groups", [None, 1, 3, 6])
def test_oracle_residual_norm_gradients_against_differences(norm_branch, groups):
    rng = np.random.default_rng(5)
    x, z = rng.normal(size=(6, 9)), rng.normal(size=(6, 9))
    gate = None if groups is None else rng.normal(size=(groups, 9))
    wb, w = rng.normal(size=9), rng.normal(size=9)
    ds, dy = rng.normal(size=(6, 9)), rng.normal(size=(6, 9))
    s, y, rb, rs = oracle.residual_norm(x, z, eps=0.0)
    assert np.allclose((y * y).mean(1), 1) and np.allclose(((z * rb[:, None]) ** 2).mean(1), 1)

    def value(x=x, z=z, gate=gate, wb=wb, w=w):
        s, y, _, _ = oracle.residual_norm(x, z, gate, 0.7, wb, w, norm_branch)
        return (ds * s).sum() + (dy * y).sum()

    s, y, rb, rs = oracle.residual_norm(x, z, gate, 0.7, wb, w, norm_branch)
    o = oracle.residual_norm_backward(ds, dy, s, z, rb if norm_branch else None, rs, gate, 0.7, wb, w)
    for name, at, grad in (("x", x, o["dx"]), ("z", z, o["dz"]), ("wb", wb, o["dwb"]), ("w", w, o["dw"])):
        d = rng.normal(size=at.shape)
        assert _slope(lambda v: value(**{name: v}), at, d) == pytest.approx((grad * d).sum(), rel=1e-6), name
    if groups is not None:
        d = rng.normal(size=gate.shape)
        dgate = o["dgate"].reshape(groups, -1, 9).sum(1)
        assert _slope(lambda v: value(gate=v), gate, d) == pytest.approx((dgate * d).sum(), rel=1e-6)


def test_oracle_residual_norm_without_a_branch():
    rng = np.random.default_rng(6)
    x, w, dy = rng.normal(size=(4, 5)), rng.normal(size=5), rng.normal(size=(4, 5))
    s, y, _, rs = oracle.residual_norm(x, None, weight=w)
    o = oracle.residual_norm_backward(None, dy, s, None, None, rs, weight=w)
    d = rng.normal(size=x.shape)
    slope = _slope(lambda v: (dy * oracle.residual_norm(v, None, weight=w)[1]).sum(), x, d)
    assert slope == pytest.approx((o["dx"] * d).sum(), rel=1e-6)


def _norm(X=PTR, ldx=8, Z=PTR, ldz=8, rows=4, cols=8, dtype=B.NS_BF16, gate=PTR, groups=2, wb=PTR, w=PTR, pt=B.NS_FP32,
          scale=1.0, nb=1, eps=1e-6, S=PTR, lds=8, Y=PTR, ldy=8):
    return B.lib().ns_residual_norm(X, ldx, Z, ldz, rows, cols, dtype, gate, groups, wb, w, pt, scale, nb, eps, S, lds,
                                    Y, ldy, None, None, None, None)


@built
def test_residual_norm_refusals():
    for kw in (dict(X=None), dict(S=None), dict(ldx=7), dict(ldz=7), dict(lds=7), dict(ldy=7), dict(rows=-1),
               dict(rows=1 << 31, groups=1), dict(cols=0), dict(cols=(1 << 24) + 1, ldx=1 << 25, ldz=1 << 25, lds=1 << 25, ldy=1 << 25),
               dict(groups=0), dict(groups=3), dict(groups=8), dict(groups=-1), dict(scale=float("nan")), dict(nb=2),
               dict(eps=-1.0), dict(eps=float("inf")), dict(Z=None), dict(Z=None, gate=None, wb=None),
               dict(Z=None, gate=None, wb=None, S=None, scale=0.5), dict(Z=None, gate=None, wb=None, S=None, Y=None)):
        assert _norm(**kw) == INV, kw
    assert _norm(dtype=5) == DT and _norm(pt=B.NS_FP16) == DT
    assert _norm(rows=0, X=None, Z=PTR, S=None, Y=None) == 0


def _norm_back(dS=PTR, ldds=8, dY=PTR, lddy=8, S=PTR, lds=8, Z=PTR, ldz=8, rows=4, cols=8, dtype=B.NS_BF16, rb=PTR,
               rs=PTR, gate=PTR, groups=2, wb=PTR, w=PTR, pt=B.NS_FP32, scale=1.0, dX=PTR, lddx=8, dZ=PTR, lddz=8,
               dg=PTR, dwb=PTR, dw=PTR, ws=256, n=1 << 30):
    return B.lib().ns_residual_norm_backward(dS, ldds, dY, lddy, S, lds, Z, ldz, rows, cols, dtype, rb, rs, gate, groups,
                                             wb, w, pt, scale, dX, lddx, dZ, lddz, dg, dwb, dw, None, ws, n, None)


@built
def test_residual_norm_backward_refusals():
    for kw in (dict(dS=None, dY=None), dict(S=None), dict(rs=None), dict(dZ=None), dict(dY=None), dict(dY=None, w=None),
               dict(ldds=7), dict(lddy=7), dict(lds=7), dict(ldz=7), dict(lddx=7), dict(lddz=7), dict(groups=0),
               dict(groups=3), dict(gate=None, groups=0), dict(rows=-1), dict(cols=0), dict(scale=float("inf")),
               dict(Z=None), dict(Z=None, gate=None, dg=None, wb=None, dwb=None),
               dict(Z=None, gate=None, dg=None, wb=None, dwb=None, dZ=None, scale=0.5),
               dict(Z=None, gate=None, dg=None, wb=None, dwb=None, dZ=None, dX=None),
               dict(rows=0, groups=1 << 40)):
        assert _norm_back(**kw) == INV, kw
    assert _norm_back(dtype=5) == DT and _norm_back(pt=B.NS_FP16) == DT
    assert _norm_back(ws=None) == WSP and _norm_back(ws=100) == WSP and _norm_back(n=100) == WSP
    assert nsa.residual_norm_workspace_size(0, 8) >= 256 and nsa.residual_norm_workspace_size(-1, 8) == 0
    assert nsa.residual_norm_workspace_size(4, 0) == 0
    # No rows and nothing wanted.
    assert _norm_back(rows=0, dg=None, dwb=None, dw=None) == 0


# ---------------------------------------------------------------------------
# The gated feed-forward block.
# ---------------------------------------------------------------------------
ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


@pytest.mark.parametrize("act", ACTS)
def test_oracle_activations(act):
    a = np.array([-30.0, -4.0, -1.0, -0.3, 0.2, 1.0, 3.0, 30.0])
    value, slope = oracle.activation(a, act)
    e = 1e-6
    assert np.allclose(slope, (oracle.activation(a + e, act)[0] - oracle.activation(a - e, act)[0]) / (2 * e), atol=1e-8)
    at_one = {"silu": 1 / (1 + np.exp(-1.0)), "gelu": 0.841344746, "gelu_tanh": 0.841191991, "relu": 1.0}[act]
    assert value[5] == pytest.approx(at_one, rel=1e-8) and value[7] == pytest.approx(30.0) and abs(value[0]) < 1e-10


@pytest.mark.parametrize("act", ACTS)
def test_oracle_gated_mlp_gradients_against_differences(act):
    rng = np.random.default_rng(8)
    at = {"x": rng.normal(size=(4, 5)), "w_gate": rng.normal(size=(7, 5)), "w_up": rng.normal(size=(7, 5)),
          "w_down": rng.normal(size=(5, 7))}
    dy = rng.normal(size=(4, 5))
    _, a, b, h = oracle.gated_mlp(**at, act=act)
    o = oracle.gated_mlp_backward(dy, **at, a=a, b=b, act=act)
    assert np.allclose(o["h"], h)
    for name, grad in (("x", "dx"), ("w_gate", "dwg"), ("w_up", "dwu"), ("w_down", "dwd")):
        d = rng.normal(size=at[name].shape)
        slope = _slope(lambda v: (dy * oracle.gated_mlp(**dict(at, **{name: v}), act=act)[0]).sum(), at[name], d, 1e-6)
        assert slope == pytest.approx((o[grad] * d).sum(), rel=1e-5), name


def _mlp(X=PTR, ldx=64, G=PTR, ldg=64, U=PTR, ldu=64, D=PTR, ldd=128, rows=40, cols=64, inner=128, dtype=B.NS_BF16, act=0,
         Y=PTR, ldy=64, gate=PTR, up=PTR, lds=128, save=B.NS_FP32, ws=256, nb=1 << 40):
    return B.lib().ns_gated_mlp(X, ldx, G, ldg, U, ldu, D, ldd, rows, cols, inner, dtype, act, Y, ldy, gate, up, lds, save,
                                None, ws, nb, None)


def _mlp_back(dY=PTR, lddy=64, X=PTR, ldx=64, G=PTR, ldg=64, U=PTR, ldu=64, D=PTR, ldd=128, gate=PTR, up=PTR, lds=128,
              rows=40, cols=64, inner=128, dtype=B.NS_BF16, act=0, dX=PTR, lddx=64, dG=PTR, lddg=64, dU=PTR, lddu=64,
              dD=PTR, lddd=128, save=B.NS_FP32, ws=256, nb=1 << 40):
    return B.lib().ns_gated_mlp_backward(dY, lddy, X, ldx, G, ldg, U, ldu, D, ldd, gate, up, lds, save, rows, cols, inner, dtype,
                                         act, dX, lddx, dG, lddg, dU, lddu, dD, lddd, None, ws, nb, None)


@built
def test_gated_mlp_refusals():
    for call, pointers, strides in (
            (_mlp, ("X", "G", "U", "D", "Y", "gate", "up"), ("ldx", "ldg", "ldu", "ldd", "ldy", "lds")),
            (_mlp_back, ("dY", "X", "G", "U", "D", "gate", "up"),
             ("lddy", "ldx", "ldg", "ldu", "ldd", "lds", "lddx", "lddg", "lddu", "lddd"))):
        for name in pointers:
            assert call(**{name: None}) == INV, name
        for name in strides:
            assert call(**{name: 63}) == INV and call(**{name: (1 << 23) + 1}) == INV, name
        for kw in (dict(rows=-1), dict(rows=(1 << 22) + 1), dict(cols=0), dict(inner=0), dict(cols=(1 << 20) + 1),
                   dict(inner=(1 << 20) + 1), dict(act=4), dict(act=-1), dict(rows=1 << 22, inner=1 << 19)):
            assert call(**kw) == INV, kw
        assert call(dtype=3) == DT and call(save=B.NS_FP16) == DT
        assert call(ws=None) == WSP and call(ws=100) == WSP and call(nb=16) == WSP
    assert _mlp(rows=0, X=None, Y=None, ws=None, nb=0) == 0
    assert _mlp_back(rows=0, dG=None, dU=None, dD=None, ws=None, nb=0) == 0
    # Nothing wanted, nothing enqueued.
    assert _mlp_back(dX=None, dG=None, dU=None, dD=None) == 0
    # A misaligned operand needs the copies' workspace too.
    need = nsa.gated_mlp_workspace_size(40, 64, 128)
    assert nsa.gated_mlp_workspace_size(40, 64, 128, aligned=False) > need
    assert _mlp(X=PTR + 2, nb=need) == WSP and _mlp(ldg=128, ldu=192, nb=need) == WSP
    need = nsa.gated_mlp_workspace_size(40, 64, 128, backward=True)
    assert _mlp_back(dY=PTR + 2, nb=need) == WSP
    assert nsa.gated_mlp_workspace_size(-1, 64, 128) == 0 and nsa.gated_mlp_workspace_size(4, 0, 128) == 0
    assert nsa.plan_gated_mlp(0, 64, 128) == [] and nsa.plan_gated_mlp(0, 64, 128, backward=True) == ["zero<bf16>"]
    with pytest.raises(nsa.NSError):
        nsa.plan_gated_mlp(4, 64, 0)


@built
def test_the_cases_reach_every_build_of_the_gated_mlp():
    import itertools

    from block_cases import MLP_RUNS
    types = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

    def builds(n, d, f, t, aligned, backward):
        return {e + (" back" if backward else "") for e in nsa.plan_gated_mlp(n, d, f, types[t], aligned, backward)
                if "=" not in e}

    every, covered = set(), set()
    for n, d, f, t, aligned, backward in itertools.product(
            [1, 2, 3, 4, 5, 8, 9, 48, 129, 300, 513, 1003, 3000, 8192, 20000], [1, 5, 64, 77, 768, 1000, 4096],
            [1, 3, 64, 203, 1407, 2048, 14336], types, (True, False), (True, False)):
        every |= builds(n, d, f, t, aligned, backward)
    for n, d, f, t in MLP_RUNS:
        for backward in (False, True):
            covered |= builds(n, d, f, t, True, backward)
    assert every - covered == set()


@built
def test_block_calls_refuse_host_tensors():
    x, w = torch.zeros(4, 8), torch.zeros(8, 8)
    for call in (lambda: nsa.gated_mlp(x, w, w, w), lambda: nsa.gated_mlp_backward(x, x, w, w, w, x, x),
                 lambda: nsa.residual_norm(x, x), lambda: nsa.residual_norm_backward(x, None, x)):
        with pytest.raises(ValueError, match="device tensor"):
            call()


@built
def test_results_in_one_place_are_refused():
    # Addresses that nothing is launched on: each call ends at the check.
    a, b = PTR, PTR + 4096
    assert _norm(S=a, Y=a) == INV
    assert _norm_back(dX=b, dZ=b) == INV
    assert _mlp(gate=a, up=a, nb=1 << 40) == INV
    for same in (("dX", "dG"), ("dX", "dD"), ("dG", "dU"), ("dU", "dD")):
        outs = dict(dX=a, dG=a + 256, dU=a + 512, dD=a + 768)
        outs[same[1]] = outs[same[0]]
        assert _mlp_back(nb=1 << 40, **outs) == INV, same
