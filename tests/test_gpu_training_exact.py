"""Calls of the training step's operators that must give the same bits:
other strides and alignment, ignored rows, captured and replayed steps.
"""

import pytest
import torch

import newton_schulz_matrix_amd as nsa
from newton_schulz_matrix_amd import _binding as B

import test_gpu_training as base

pytestmark = pytest.mark.gpu

DTYPES = base.DTYPES


def _inside(t, lead, off):
    """(the whole buffer, t's copy inside it): rows `lead` apart, `off` in."""
    whole = torch.full((t.shape[0], lead), float("nan"), dtype=t.dtype, device=t.device)
    part = whole[:, off:off + t.shape[1]]
    part.copy_(t)
    return whole, part


@pytest.mark.parametrize("cols", [3, 96, 97, 768, 1001, 4097, 9000, 20001])
@pytest.mark.parametrize("dtype,pdtype", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_layer_norm_on_strided_rows_equals_contiguous(cols, dtype, pdtype):
    # A row's sums do not depend on where it starts: equal to the last bit.
    dev = base._dev()
    print(f"layer norm strides {cols} {dtype}/{pdtype}", flush=True)
    x, w, b, dy = base._norm_inputs(21, cols, dtype, pdtype, dev, seed=cols)
    y, mean, rstd = nsa.layer_norm(x, w, b)
    want = nsa.layer_norm_backward(dy, x, mean, rstd, w)
    for lead, off in ((cols + 32, 0), (cols + 33, 0), (cols + 32, 3), (cols + 1, 1)):
        xs, dys = _inside(x, lead, off)[1], _inside(dy, lead, off)[1]
        out, o = _inside(torch.zeros_like(x), lead, off)
        got = nsa.layer_norm(xs, w, b, out=o)
        assert torch.equal(o, y) and torch.equal(got[1], mean) and torch.equal(got[2], rstd)
        dout, do = _inside(torch.zeros_like(x), lead, off)
        dx, dw, db = nsa.layer_norm_backward(dys, xs, mean, rstd, w, out=do)
        assert torch.equal(do, want[0]) and torch.equal(dw, want[1]) and torch.equal(db, want[2])
        for whole in (out, dout):  # nothing beside the rows is written
            assert torch.isnan(whole[:, :off]).all() and torch.isnan(whole[:, off + cols:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,d,v", [(70, 64, 300), (300, 72, 500)])
def test_ignored_rows_equal_rows_with_a_bad_target(n, d, v, dtype):
    # The same gradients, bit for bit; the ignored id is one inside the
    # vocabulary that no other row has.
    dev = base._dev()
    h, w, t, dloss = base._xent_inputs(n, d, v, dtype, dev, seed=n, ignored=0.0)
    t %= v - 1
    lse = nsa.linear_cross_entropy(h, w, t)[1]
    bad, ignored = t.clone(), t.clone()
    bad[3], bad[4], bad[n - 1] = v, -1, 1 << 40
    ignored[[3, 4, n - 1]] = v - 1
    st = base._word(dev)
    want = nsa.linear_cross_entropy_backward(h, w, bad, lse, dloss, status=st)
    assert int(st.item()) == B.STATUS_BAD_INDEX
    st.zero_()
    got = nsa.linear_cross_entropy_backward(h, w, ignored, lse, dloss, ignore_index=v - 1, status=st)
    assert int(st.item()) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # And those of the other rows alone: dh's rows, and dw, whose sums take
    # zeros for the rows left out.
    keep = torch.ones(n, dtype=torch.bool, device=dev)
    keep[[3, 4, n - 1]] = False
    weight = torch.where(keep, dloss, torch.zeros_like(dloss))
    alone = nsa.linear_cross_entropy_backward(h, w, t, lse, weight)
    assert torch.count_nonzero(got[0][~keep]) == 0 and torch.equal(got[0], alone[0]) and torch.equal(got[1], alone[1])


def _step(ids, targets, p, out, st):
    """Every operator once, into the caller's own outputs, and one number for
    the losses' gradients."""
    nsa.embedding(ids, p["table"], scale=p["scale"], out=out["e"], status=st)
    _, mean, rstd = nsa.layer_norm(out["e"], p["w1"], p["b1"], out=out["a"], status=st)
    loss, lse = nsa.linear_cross_entropy(out["a"], p["table"], targets, status=st)
    nsa.linear_cross_entropy_backward(out["a"], p["table"], targets, lse, 0.25, out_dh=out["dh"], out_dw=out["dt"], status=st)
    _, dw, db = nsa.layer_norm_backward(out["dh"], out["e"], mean, rstd, p["w1"], out=out["dh"], status=st)
    nsa.embedding_backward(ids, out["dh"], p["table"].shape[0], scale=p["scale"], out=out["dt"], accumulate=True, status=st)
    return [loss, lse, dw, db]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,d,v", [(300, 128, 500), (3, 72, 200), (1000, 264, 20000)])
def test_a_step_captured_on_a_side_stream_replays_equal_to_eager(n, d, v, dtype):
    dev = base._dev()
    print(f"captured step n={n} d={d} v={v} {dtype}", flush=True)
    ids, targets, p = base._chain_state(n, d, v, DTYPES[dtype], dev, seed=1)

    def outputs():
        rows = {k: torch.zeros(n, d, dtype=DTYPES[dtype], device=dev) for k in ("e", "a", "dh")}
        return {**rows, "dt": torch.zeros(v, d, dtype=DTYPES[dtype], device=dev)}

    out, eager = outputs(), outputs()
    st, est = base._word(dev), base._word(dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(ids, targets, p, out, st)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            rest = _step(ids, targets, p, out, st)
    torch.cuda.synchronize()
    for i in range(3):
        new_ids, new_t, new_p = base._chain_state(n, d, v, DTYPES[dtype], dev, seed=20 + i)
        if i == 2:
            new_ids[1] = v + 5  # reported from inside the graph as well
        ids.copy_(new_ids)
        targets.copy_(new_t)
        for k in p:
            if k != "scale":
                p[k].copy_(new_p[k])
        st.zero_()
        est.zero_()
        want = _step(ids, targets, p, eager, est)
        torch.cuda.synchronize()
        graph.replay()
        # The program's own work on the same tensors behind the replay.
        again = nsa.linear_cross_entropy(out["a"], p["table"], targets)[0]
        torch.cuda.synchronize()
        assert torch.equal(again, want[0])
        for a, b in zip(rest, want):
            assert torch.equal(a, b), i
        for k in out:
            assert torch.equal(out[k], eager[k]), (i, k)
        assert int(st.item()) == int(est.item()) == (B.STATUS_BAD_INDEX if i == 2 else 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_steps_on_two_streams_at_once(dtype):
    dev = base._dev()
    sizes = [(700, 264, 9000), (300, 128, 500)]
    inputs = [base._chain_state(n, d, v, DTYPES[dtype], dev, seed=i) for i, (n, d, v) in enumerate(sizes)]

    def run(i):
        (n, d, v), (ids, targets, p) = sizes[i], inputs[i]
        rows = {k: torch.zeros(n, d, dtype=DTYPES[dtype], device=dev) for k in ("e", "a", "dh")}
        out = {**rows, "dt": torch.zeros(v, d, dtype=DTYPES[dtype], device=dev)}
        return _step(ids, targets, p, out, base._word(dev)) + list(out.values())

    want = [run(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(i))
    torch.cuda.synchronize()
    for i in range(2):
        for one in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(one, want[i]))
