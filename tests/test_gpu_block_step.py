"""A training step of a small model made of the library's operators alone.

Tied embedding, a norm, a gated feed-forward block in a residual stream with a
layer scale, the output projection's cross entropy; all gradients by hand;
Muon for the matrices and AdamW (8-bit and fp32 moments, 16-bit copies of fp32
masters) for the rest.
"""

import numpy as np
import pytest
import torch

import newton_schulz_matrix_amd as nsa

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
VOCAB, COLS, INNER = 211, 96, 200
SCALE, EPS = 0.75, 1e-5


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _model(dtype, dev, seed=0, ptype=torch.float32):
    g = torch.Generator().manual_seed(seed)

    def make(*shape, scale, to=dtype, mean=0.0):
        return (mean + scale * torch.randn(*shape, generator=g)).to(to).to(dev)

    return dict(table=make(VOCAB, COLS, scale=0.4), wg=make(INNER, COLS, scale=COLS ** -0.5),
                wu=make(INNER, COLS, scale=COLS ** -0.5), wd=make(COLS, INNER, scale=INNER ** -0.5),
                first=make(COLS, scale=0.1, mean=1.0, to=ptype), gate=make(1, COLS, scale=0.2, mean=0.6, to=ptype),
                branch=make(COLS, scale=0.1, mean=1.0, to=ptype), last=make(COLS, scale=0.1, mean=1.0, to=ptype))


def _ids(shape, dev, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(VOCAB, shape, generator=g).to(dev), torch.randint(VOCAB, shape, generator=g).to(dev)


def _forward(p, ids, targets, act, status=None):
    x = nsa.embedding(ids, p["table"], status=status)
    _, x1, _, r1 = nsa.residual_norm(x, weight=p["first"], eps=EPS, status=status)
    z, a, b = nsa.gated_mlp(x1, p["wg"], p["wu"], p["wd"], activation=act, status=status)
    s, h, rb, r2 = nsa.residual_norm(x, z, gate=p["gate"], scale=SCALE, branch_weight=p["branch"], weight=p["last"],
                                     eps=EPS, status=status)
    loss, lse = nsa.linear_cross_entropy(h.view(-1, COLS), p["table"], targets.view(-1), status=status)
    return loss, (x, x1, r1, z, a, b, s, h, rb, r2, lse)


def _backward(p, ids, targets, act, kept, status=None):
    x, x1, r1, z, a, b, s, h, rb, r2, lse = kept
    dh, dtable = nsa.linear_cross_entropy_backward(h.view(-1, COLS), p["table"], targets.view(-1), lse,
                                                   1.0 / targets.numel(), status=status)
    dx, dz, dgate, dbranch, dlast = nsa.residual_norm_backward(
        None, dh.view(s.shape), s, z, rb, r2, gate=p["gate"], scale=SCALE, branch_weight=p["branch"], weight=p["last"],
        status=status)
    dx1, dwg, dwu, dwd = nsa.gated_mlp_backward(dz, x1, p["wg"], p["wu"], p["wd"], a, b, activation=act, status=status)
    # The residual stream's gradient joins that of the first norm in one call's dstream.
    dx, _, _, _, dfirst = nsa.residual_norm_backward(dx, dx1, x, rstd=r1, weight=p["first"], status=status)
    nsa.embedding_backward(ids, dx, VOCAB, out=dtable, accumulate=True, status=status)
    return dict(table=dtable, wg=dwg, wu=dwu, wd=dwd, first=dfirst, gate=dgate, branch=dbranch, last=dlast)


def _exact(p, ids, targets, act):
    """Loss and gradients in 64 bits on the CPU."""
    q = {k: v.detach().double().cpu().requires_grad_() for k, v in p.items()}

    def norm(t):
        return t * (t.square().mean(-1, keepdim=True) + EPS).rsqrt()

    acts = dict(silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu, relu=torch.relu,
                gelu_tanh=lambda t: torch.nn.functional.gelu(t, approximate="tanh"))
    x = q["table"][ids.cpu()]
    x1 = norm(x) * q["first"]
    z = (acts[act](x1 @ q["wg"].t()) * (x1 @ q["wu"].t())) @ q["wd"].t()
    s = SCALE * x + q["gate"] * norm(z) * q["branch"]
    logits = (norm(s) * q["last"]) @ q["table"].t()
    loss = torch.nn.functional.cross_entropy(logits.reshape(-1, VOCAB), targets.cpu().view(-1))
    loss.backward()
    return float(loss.detach()), {k: v.grad for k, v in q.items()}


# A chain of 9 operators, forward and back.  In norms: a result stored with
# half a step u is off by u of itself; a sum of K <= 211 products in fp32 by at
# most (K + 1) u32 of its terms' magnitudes, which for terms of random signs
# are sqrt(K) times the sum; an operator hands on the errors of its inputs at
# most doubled in norm (norms and activations have slopes about 1, the two
# paths of the stream add).  So 2 * 9 * (u_stored * 3 roundings an operator +
# 212 * 15 u32): 3.4e-3 with everything in fp32.  In bf16 the worst case is no
# bound worth having; roundings of random sign join as the root of their
# number: sqrt(2 * 9 * 3) u doubled, 0.06.
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("shape", [(1,), (3,), (2, 9), (5, 61)])
@pytest.mark.parametrize("dtype,bound", [(torch.float32, 2 * 9 * (3 + 212 * 15) * U32), (torch.bfloat16, 0.06)])
def test_loss_and_every_gradient(shape, act, dtype, bound):
    dev = _dev()
    p = _model(dtype, dev)
    ids, targets = _ids(shape, dev, 5)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    loss, kept = _forward(p, ids, targets, act, status)
    got = _backward(p, ids, targets, act, kept, status)
    want_loss, want = _exact(p, ids, targets, act)
    assert abs(float(loss.double().mean()) - want_loss) <= bound * want_loss
    for k, v in want.items():
        off = float((got[k].double().cpu() - v).norm() / v.norm())
        print(k, off, flush=True)
        assert got[k].shape == p[k].shape and got[k].dtype == p[k].dtype
        assert off <= bound, k
    assert int(status.item()) == 0


def test_gradients_against_differences():
    # L(p + t q) - L(p - t q) = 2 t <dL, q> + t^3 L'''/3; the mean loss of 305
    # tokens in fp32 is off by about 1e-6.  Along the gradient itself, scaled so
    # that the step moves the loss by about 2e-2, that is 1e-4 of it, and
    # the cubic term a few parts in a thousand.
    dev = _dev()
    p = _model(torch.float32, dev, seed=3)
    ids, targets = _ids((5, 61), dev, 7)
    loss, kept = _forward(p, ids, targets, "silu")
    grads = _backward(p, ids, targets, "silu", kept)
    for k, g in grads.items():
        t = 1e-2 / float(g.double().square().sum())
        both = []
        for sign in (1, -1):
            moved = dict(p, **{k: (p[k].double() + sign * t * g.double()).float()})
            both.append(float(_forward(moved, ids, targets, "silu")[0].double().mean()))
        print(k, both[0] - both[1], flush=True)
        assert abs(both[0] - both[1] - 2e-2) <= 2e-2 * 0.05, k


class _Trainer:
    """Muon on the three matrices, AdamW on the rest: the tied table as an
    fp32 master with 8-bit moments and a 16-bit copy, the vectors with fp32
    moments."""

    MATRICES = ("wg", "wu", "wd")
    VECTORS = ("first", "gate", "branch", "last")

    def __init__(self, dev, act="silu"):
        self.p = _model(torch.bfloat16, dev, seed=11)
        self.act = act
        self.momentum = [torch.zeros(self.p[k].shape, dtype=torch.float32, device=dev) for k in self.MATRICES]
        self.master = self.p["table"].float()
        m, v, s = nsa.adamw_states([self.master], bits=8)
        mv, vv, _ = nsa.adamw_states([self.p[k] for k in self.VECTORS])
        self.m, self.v, self.s = m + mv, v + vv, s + [None] * len(mv)
        self.ids, self.targets = (torch.zeros(4, 33, dtype=torch.int64, device=dev) for _ in range(2))
        self.step = torch.ones(1, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.loss = torch.zeros(4 * 33, dtype=torch.float32, device=dev)

    def state(self):
        return [self.p[k] for k in self.p] + self.momentum + [self.master] + self.m + self.v + [self.s[0], self.step]

    def run(self):
        loss, kept = _forward(self.p, self.ids, self.targets, self.act, self.status)
        g = _backward(self.p, self.ids, self.targets, self.act, kept, self.status)
        self.loss.copy_(loss)
        for k, m in zip(self.MATRICES, self.momentum):
            nsa.muon_step(self.p[k], g[k], m, lr=0.02, status=self.status)
        nsa.adamw_step([self.master] + [self.p[k] for k in self.VECTORS], [g["table"]] + [g[k] for k in self.VECTORS],
                       self.m, self.v, lr=[1e-3] + [3e-3] * 4, step=self.step, weight_decay=[0.1] + [0.0] * 4,
                       scales=self.s, copies=[self.p["table"]] + [None] * 4, status=self.status)
        self.step.add_(1)


def test_steps_captured_are_the_eager_ones():
    dev = _dev()
    eager, graphed = _Trainer(dev), _Trainer(dev)
    start = [t.clone() for t in graphed.state()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.run()
    for t, v in zip(graphed.state(), start):
        t.copy_(v)
    for i in range(4):
        ids, targets = _ids((4, 33), dev, 100 + i)
        for tr in (eager, graphed):
            tr.ids.copy_(ids)
            tr.targets.copy_(targets)
        graph.replay()
        eager.run()
        torch.cuda.synchronize()
        assert torch.equal(eager.loss, graphed.loss), i
        for n, (a, b) in enumerate(zip(eager.state(), graphed.state())):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (i, n)
    assert int(eager.status.item()) == int(graphed.status.item()) == 0
    assert int(eager.step.item()) == 5
    assert torch.equal(eager.p["table"], eager.master.bfloat16())
    assert all(not torch.equal(a, b) for a, b in zip(eager.state()[:8], start[:8]))


def test_two_models_on_two_streams():
    dev = _dev()
    alone, beside = [_Trainer(dev, a) for a in ("silu", "gelu")], [_Trainer(dev, a) for a in ("silu", "gelu")]
    for pair in (alone, beside):
        for i, tr in enumerate(pair):
            ids, targets = _ids((4, 33), dev, 200 + i)
            tr.ids.copy_(ids)
            tr.targets.copy_(targets)
    for tr in alone:
        for _ in range(3):
            tr.run()
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in beside]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s, tr in zip(streams, beside):
            with torch.cuda.stream(s):
                tr.run()
    torch.cuda.synchronize()
    for a, b in zip(alone, beside):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a.state(), b.state()))


def test_two_graphs_that_share_a_workspace():
    # Replayed one after the other on one stream, each leaves nothing behind
    # that the other reads.
    dev = _dev()
    g = torch.Generator().manual_seed(1)
    runs = []
    need = max(nsa.gated_mlp_workspace_size(n, 160, 320, torch.bfloat16, False, True) for n in (7, 200)) + 256
    need = max(need, nsa.residual_norm_workspace_size(200, 160) + 256)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev)

    def make(*shape):
        return (0.1 * torch.randn(*shape, generator=g)).bfloat16().to(dev)

    for n in (7, 200):
        x, dy, wg, wu, wd, w = make(n, 160), make(n, 160), make(320, 160), make(320, 160), make(160, 320), make(160)

        def step(x=x, dy=dy, wg=wg, wu=wu, wd=wd, w=w):
            s, h, _, r = nsa.residual_norm(x, weight=w)
            y, a, b = nsa.gated_mlp(h, wg, wu, wd, workspace=ws)
            dh, *dw = nsa.gated_mlp_backward(dy, h, wg, wu, wd, a, b, workspace=ws)
            dx, _, _, _, dweight = nsa.residual_norm_backward(dy, dh, s, rstd=r, weight=w, workspace=ws)
            return [y, a, b, dh, *dw, dx, dweight]

        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        runs.append((graph, out, want, step))  # step holds the inputs that the graph reads
    for _ in range(3):
        for graph, out, want, _ in runs:
            for t in out:
                t.fill_(float("nan"))
            graph.replay()
        torch.cuda.synchronize()
        for _, out, want, _ in runs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        ws.fill_(255)


def test_arguments_that_are_no_tensors():
    dev = _dev()
    x = torch.ones(4, 8, device=dev)
    w = torch.ones(8, device=dev)
    wg, wd = torch.ones(6, 8, device=dev), torch.ones(8, 6, device=dev)
    a = torch.ones(4, 6, device=dev)
    r = torch.ones(4, device=dev)
    host = np.ones((4, 8), np.float32)
    for call in (lambda: nsa.residual_norm(x, host), lambda: nsa.residual_norm(x, weight=[1.0] * 8),
                 lambda: nsa.residual_norm(x, x, gate=2.0), lambda: nsa.residual_norm(x, scale="1"),
                 lambda: nsa.residual_norm(x, out_norm=host), lambda: nsa.residual_norm_backward(x, host, x, rstd=r),
                 lambda: nsa.residual_norm_backward(x, x, x, rstd=host), lambda: nsa.residual_norm_backward(x, None, x, workspace=1),
                 lambda: nsa.gated_mlp(x, wg, wg, [1]), lambda: nsa.gated_mlp(x, wg, wg, wd, workspace="w"),
                 lambda: nsa.gated_mlp(x, wg, wg, wd, out=host), lambda: nsa.gated_mlp(x, wg, wg, wd, save=1),
                 lambda: nsa.gated_mlp_backward(host, x, wg, wg, wd, a, a), lambda: nsa.gated_mlp_backward(x, x, wg, wg, wd, a, None),
                 lambda: nsa.gated_mlp_backward(x, x, wg, wg, wd, a, a, out_dw_up=3),
                 lambda: nsa.adamw_step([x], [host], [x.clone()], [x.clone()], lr=1e-3, step=1),
                 lambda: nsa.adamw_step([x], [x], [None], [x.clone()], lr=1e-3, step=1),
                 lambda: nsa.adamw_step([x], [x.clone()], [x.clone()], [x.clone()], lr="1", step=1),
                 lambda: nsa.adamw_step([x], [x.clone()], [x.clone()], [x.clone()], lr=[None], step=1)):
        with pytest.raises((TypeError, ValueError)):
            call()
    assert bool((x == 1).all())


def test_axes_of_any_number_and_single_columns():
    dev = _dev()
    g = torch.Generator().manual_seed(2)

    def make(*shape):
        return torch.randn(*shape, generator=g).to(dev)

    x, z, w = make(2, 3, 5, 12), make(2, 3, 5, 12), make(12)
    gate = make(2, 3, 12)  # one row for 5 of the data's
    flat = nsa.residual_norm(x.view(30, 12), z.view(30, 12), gate=gate.view(6, 12), weight=w)
    full = nsa.residual_norm(x, z, gate=gate, weight=w)
    assert full[0].shape == x.shape and full[2].shape == (2, 3, 5)
    assert all(torch.equal(a.reshape(-1), b.reshape(-1)) for a, b in zip(full, flat))
    one = nsa.residual_norm(x[0, 0, 0], weight=w)
    assert one[3].shape == () and torch.equal(one[1], nsa.residual_norm(x[0, 0, :1], weight=w)[1][0])
    back = nsa.residual_norm_backward(x, z, full[0], z, full[2], full[3], gate=gate, weight=w)
    assert back[2].shape == gate.shape and back[0].shape == x.shape
    # One column and one inner unit.
    x, wg, wu, wd = make(9, 1), make(1, 1), make(1, 1), make(1, 1)
    y, a, b = nsa.gated_mlp(x, wg, wu, wd, activation="relu")
    want = torch.relu(x.double() * wg.double()) * (x.double() * wu.double()) * wd.double()
    assert bool(((y.double() - want).abs() <= 8 * U32 * want.abs()).all())
    dx, dwg, dwu, dwd = nsa.gated_mlp_backward(torch.ones_like(x), x, wg, wu, wd, a, b, activation="relu")
    want = 2 * (x.double() * wg.double()).clamp(min=0) * wu.double() * wd.double()
    assert bool(((dx.double() - want).abs() <= 8 * U32 * want.abs()).all())
    s, h, rb, r = nsa.residual_norm(x, x.clone(), weight=torch.ones(1, device=dev))
    assert s.shape == h.shape == x.shape and r.shape == (9,)


@pytest.mark.parametrize("n,d,f", [(3, 72, 130), (60, 96, 200), (300, 128, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_feed_forward_results_written_over_inputs(n, d, f, dtype):
    dev = _dev()
    g = torch.Generator().manual_seed(n)

    def make(*shape):
        return torch.randn(*shape, generator=g).to(dtype).to(dev)

    x, dy, wg, wu, wd = make(n, d), make(n, d), make(f, d), make(f, d), make(d, f)
    y, a, b = nsa.gated_mlp(x, wg, wu, wd)
    over = x.clone()
    assert nsa.gated_mlp(over, wg, wu, wd, out=over)[0] is over and torch.equal(over, y)
    want = nsa.gated_mlp_backward(dy, x, wg, wu, wd, a, b)
    over = [t.clone() for t in (dy, wg, wu, wd)]
    got = nsa.gated_mlp_backward(over[0], x, *over[1:], a, b, out_dx=over[0], out_dw_gate=over[1], out_dw_up=over[2],
                                 out_dw_down=over[3])
    assert all(p is q for p, q in zip(got, over)) and all(torch.equal(p, q) for p, q in zip(got, want))
    over = x.clone()
    assert torch.equal(nsa.gated_mlp_backward(dy, over, wg, wu, wd, a, b, need_dw=False, out_dx=over)[0], want[0])
    # One matrix in both places.
    y, a, b = nsa.gated_mlp(x, wg, wg, wd)
    assert torch.equal(a, b)


def test_gates_of_many_wide_rows():
    # 256 rows of a gate, each of 2^20 columns, are summed over 2 rows each.
    dev = _dev()
    rows, cols, groups = 512, 1 << 20, 256
    g = torch.Generator(device=dev).manual_seed(4)

    def make(*shape):
        return torch.randn(*shape, device=dev, generator=g).bfloat16()

    x, z, ds, dy, gate = make(rows, cols), make(rows, cols), make(rows, cols), make(rows, cols), make(groups, cols)
    s, y, rb, rs = nsa.residual_norm(x, z, gate=gate)
    dgate = nsa.residual_norm_backward(ds, dy, s, z, rb, rs, gate=gate)[2]
    for i in range(0, groups, 32):
        c = slice(2 * i, 2 * i + 64)
        r64, shat = rs[c].double()[:, None], s[c].double() * rs[c].double()[:, None]
        u = dy[c].double()
        top = ds[c].double() + r64 * (u - shat * (u * shat).mean(1, keepdim=True))
        bhat = z[c].double() * rb[c].double()[:, None]
        want = (top * bhat).view(32, 2, cols).sum(1)
        size = ((top.abs() + 1) * bhat.abs()).view(32, 2, cols).sum(1)
        # Rounded once to bf16; top to its mean, a sum of 2^20 terms taken by
        # 1024 threads, of 1024 steps and 20 more.
        assert bool(((dgate[i:i + 32].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1056 * U32 * size).all())


def test_a_large_gate_without_rows():
    dev = _dev()
    gate = torch.ones(5000, 65536, dtype=torch.bfloat16, device=dev)
    none = torch.empty(0, 65536, dtype=torch.bfloat16, device=dev)
    r = torch.empty(0, device=dev)
    got = nsa.residual_norm_backward(none, none, none, none, r, r, gate=gate, weight=gate[0])
    assert got[2].shape == gate.shape and not bool(got[2].any()) and not bool(got[4].any())
