"""AdamW over many tensors on the GPU against the fp64 oracle.

Bounds are worst cases of the arithmetic, with u32 = 2^-24 and u half a step
of the stored type (bf16 2^-8, fp16 2^-11, fp32 2^-24, e4m3 2^-4).
"""

import numpy as np
import pytest
import torch

import oracle
import newton_schulz_matrix_amd as nsa
from newton_schulz_matrix_amd import _binding as B

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U32 = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
BETAS, EPS = (0.9, 0.95), 1e-8


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _np(t):
    return t.detach().cpu().to(torch.float32 if t.dtype == torch.float8_e4m3fn else t.dtype).double().numpy()


def _close(got, want, bound, what):
    got = _np(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, what
    off = np.abs(got - want)
    worst = float(np.max(off / np.maximum(bound, 1e-300))) if off.size else 0.0
    assert np.all(off <= bound), (what, worst)
    return worst


def _decode(code, scale, blocks=256):
    flat = _np(code).reshape(-1)
    return (flat * np.repeat(_np(scale), blocks)[:flat.size] / 448.0).reshape(tuple(code.shape))


def _quantized(x, up):
    """(codes, tops): test inputs in the 8-bit form (any codes would do)."""
    flat = x.reshape(-1)
    pad = torch.nn.functional.pad(flat, (0, -flat.numel() % 256)).view(-1, 256)
    top = pad.abs().amax(1).clamp(min=2.0 ** -100)
    q = pad * (448 / top)[:, None]
    if up:
        q = torch.where((q > 0) & (q < 2.0 ** -9), torch.full_like(q, 2.0 ** -9), q)
    return q.view(-1)[:flat.numel()].view(x.shape).to(torch.float8_e4m3fn), top


class _Set:
    """Tensors of a step, with copies of what they held before."""

    def __init__(self, shapes, ptypes, gtypes, bits, dev, seed=0, offset=0, copies=None):
        gen = torch.Generator().manual_seed(seed)

        def make(value, dtype):
            # `offset`: elements between a 16-byte boundary and the tensor.
            t = torch.zeros(value.numel() + offset, dtype=dtype, device=dev)[offset:].view(value.shape)
            t.copy_(value)
            return t

        self.p, self.g, self.m, self.v, self.scales, self.copies = [], [], [], [], [], []
        for i, shape in enumerate(shapes):
            size = torch.exp(2 * torch.randn(shape, generator=gen)) * 1e-3
            self.p.append(make(torch.randn(shape, generator=gen), ptypes[i % len(ptypes)]))
            self.g.append(make(torch.randn(shape, generator=gen) * size, gtypes[i % len(gtypes)]))
            m = 0.3 * torch.randn(shape, generator=gen) * size
            v = size * size * torch.rand(shape, generator=gen)
            if bits[i % len(bits)] == 32:
                self.m.append(make(m, torch.float32))
                self.v.append(make(v, torch.float32))
                self.scales.append(None)
            else:
                (cm, tm), (cv, tv) = _quantized(m, False), _quantized(v.sqrt(), True)
                self.m.append(make(cm, torch.float8_e4m3fn))
                self.v.append(make(cv, torch.float8_e4m3fn))
                self.scales.append(torch.stack([tm, tv]).to(dev))
            ct = copies[i % len(copies)] if copies else None
            self.copies.append(None if ct is None else make(torch.full(shape, float("nan")), ct))
        self.before = [tuple(None if t is None else t.clone() for t in row)
                       for row in zip(self.p, self.g, self.m, self.v, self.scales)]

    def step(self, **kw):
        args = dict(lr=1e-2, step=7, betas=BETAS, eps=EPS, weight_decay=0.1)
        args.update(kw)
        nsa.adamw_step(self.p, self.g, self.m, self.v, scales=self.scales, copies=self.copies, **args)

    def check(self, lr, step, decay, grad_scale=1.0):
        worst = 0.0
        for i, (p0, g0, m0, v0, s0) in enumerate(self.before):
            if p0.numel() == 0:
                continue
            rate = lr[i] if isinstance(lr, (list, tuple)) else lr
            wd = decay[i] if isinstance(decay, (list, tuple)) else decay
            if s0 is None:
                m64, v64 = _np(m0), _np(v0)
            else:
                m64, v64 = _decode(m0, s0[0]), _decode(v0, s0[1]) ** 2
            p, m, v = oracle.adamw(_np(p0), _np(g0), m64, v64, rate, step, BETAS, EPS, wd, grad_scale)
            g = _np(g0) * grad_scale
            # m: of the decoded moment 1 / 448, the unit and the product, then
            # beta, product and sum (6); of the gradient its scaling, 1 - beta,
            # product and sum (4); and 1 for the second order.  v: the squares
            # of those, so at most 10, its root half of that and 1 of its own.
            em = 7 * U32 * (BETAS[0] * np.abs(m64) + (1 - BETAS[0]) * np.abs(g))
            root = np.sqrt(v / (1 - BETAS[1] ** step))
            update = np.abs(m) / (1 - BETAS[0] ** step) / (root + EPS)
            # The root: half of v's 10 steps, 3 of its own and of its factor;
            # then eps, the quotient, two factors of m's and lr's two.
            ep = rate / (1 - BETAS[0] ** step) / (root + EPS) * em + 16 * U32 * rate * update
            ep = ep + U32 * (4 * rate * wd + 2) * np.abs(_np(p0)) + U32 * rate * update
            u = HALF_STEP[p0.dtype]
            worst = max(worst, _close(self.p[i], p, u * (np.abs(p) + ep) + ep + TINY[p0.dtype], f"p[{i}]"))
            if self.copies[i] is not None:
                t = self.copies[i].dtype
                _close(self.copies[i], p, HALF_STEP[t] * (np.abs(p) + ep) + ep + TINY[t], f"copy[{i}]")
            if s0 is None:
                _close(self.m[i], m, em, f"m[{i}]")
                _close(self.v[i], v, 10 * U32 * v + 2.0 ** -149, f"v[{i}]")
                continue
            for name, code, want, err, row in (("m", self.m[i], m, em, 0), ("root", self.v[i], np.sqrt(v), 7 * U32 * np.sqrt(v), 1)):
                top = oracle.state_tops(want)
                # The largest of a block is off by no more than its elements
                # are (m's two terms may cancel, so not relative to itself).
                _close(self.scales[i][row], top, oracle.state_tops(err, least=0.0), f"scale of {name}[{i}]")
                unit = np.repeat(top, 256)[:want.size].reshape(want.shape) / 448
                # Half an e4m3 step, 2^-4 relative or half of 2^-9 below its
                # normal numbers; positive roots down there go up, by 2^-9 at most.
                bound = 2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -10) + unit * (2.0 ** -10 if name == "m" else 2.0 ** -9) + 2 * err
                _close(_decode(code, self.scales[i][row]), want, bound, f"{name}[{i}]")
                if name == "root":
                    assert np.all((_np(code) > 0) == (want > 0)), "positive roots keep a positive code"
        print(f"adamw: worst error of p {worst:.3f} of the bound", flush=True)


SIZES = [(1,), (7,), (8,), (9,), (255,), (256,), (257,), (2047,), (2048,), (2049,), (0,), (3, 5, 7), (50, 333), (128, 4096)]


@pytest.mark.parametrize("bits", [(32,), (8,), (8, 32)])
@pytest.mark.parametrize("ptype,gtype", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16"),
                                         ("bf16", "fp32"), ("fp16", "bf16"), ("fp32", "fp16")])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_one_step_matches_the_oracle(bits, ptype, gtype, offset):
    dev = _dev()
    print(f"adamw {bits} {ptype}/{gtype} offset {offset}", flush=True)
    s = _Set(SIZES, [DTYPES[ptype]], [DTYPES[gtype]], bits, dev, seed=offset, offset=offset,
             copies=[torch.bfloat16, None, torch.float16])
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    s.step(status=st)
    s.check(1e-2, 7, 0.1)
    assert int(st.item()) == 0


def test_more_tensors_than_a_launch_takes_with_their_own_rates():
    dev = _dev()
    gen = np.random.default_rng(3)
    shapes = [(int(n),) for n in gen.integers(1, 9000, 149)]
    lr, wd = [float(x) for x in gen.uniform(1e-4, 1e-1, 149)], [float(x) for x in gen.choice([0.0, 0.1], 149)]
    s = _Set(shapes, list(DTYPES.values()), [torch.bfloat16, torch.float32], (32, 8, 8, 32, 8), dev)
    s.step(lr=lr, weight_decay=wd)
    s.check(lr, 7, wd)


def test_device_scalars_and_a_captured_step():
    # The step, the clipping coefficient and the schedule's factor are read
    # when the kernels run: every replay takes their values of that time.
    dev = _dev()
    shapes = [(300, 70), (5000,), (3,)] * 20
    step = torch.zeros(1, dtype=torch.int32, device=dev)
    clip, factor = torch.ones(1, device=dev), torch.ones(1, device=dev)
    s = _Set(shapes, [torch.bfloat16, torch.float32], [torch.bfloat16], (8, 32), dev)
    start = [t.clone() for row in (s.p, s.m, s.v) for t in row] + [t.clone() for t in s.scales if t is not None]

    def buffers():
        return s.p + s.m + s.v + [t for t in s.scales if t is not None]

    def reset():
        for t, t0 in zip(buffers(), start):
            t.copy_(t0)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        s.step(step=step + 1, grad_scale=clip, lr_scale=factor)
    torch.cuda.synchronize()
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        s.step(step=step, grad_scale=clip, lr_scale=factor)
    reset()
    step.zero_()
    values = [(1.0, 1.0), (0.25, 0.5), (0.5, 2.0)]
    replayed = []
    for c, f in values:
        clip.fill_(c)
        factor.fill_(f)
        graph.replay()
        torch.cuda.synchronize()
        replayed.append([t.clone() for t in buffers()])
        assert torch.isfinite(s.p[0].float()).all()
    reset()
    for t, (c, f) in enumerate(values):
        clip.fill_(c)
        factor.fill_(f)
        s.step(step=torch.full((1,), t + 1, dtype=torch.int32, device=dev), grad_scale=clip, lr_scale=factor)
        for a, b in zip(replayed[t], buffers()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # A step given as a number is the same up to the correction factors' roundings.
    reset()
    clip.fill_(0.5)
    s.before = [tuple(None if t is None else t.clone() for t in row) for row in zip(s.p, s.g, s.m, s.v, s.scales)]
    s.step(step=torch.full((1,), 3, dtype=torch.int32, device=dev), grad_scale=clip,
           lr_scale=torch.full((1,), 0.5, device=dev), lr=4e-2)
    s.check(2e-2, 3, 0.1, grad_scale=0.5)


def test_equal_calls_give_equal_bits_and_grads_stay():
    dev = _dev()
    runs = []
    for _ in range(2):
        s = _Set([(513, 77), (1000,)], [torch.bfloat16], [torch.bfloat16], (8, 32), dev, seed=4)
        s.step()
        assert all(torch.equal(g, b[1]) for g, b in zip(s.g, s.before))
        runs.append(s)
    for a, b in zip(runs[0].p + runs[0].m + runs[0].v, runs[1].p + runs[1].m + runs[1].v):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_states_and_zero_gradients(bits):
    dev = _dev()
    p = [torch.randn(1000, device=dev)]
    g = [torch.randn(1000, device=dev)]
    g[0][:300] = 0
    m, v, scales = nsa.adamw_states(p, bits=bits)
    before = p[0].clone()
    nsa.adamw_step(p, g, m, v, lr=0.1, step=1, scales=scales, weight_decay=0.0)
    # The first step goes by lr along the gradient's sign.
    # Relative: m and its correction 4 steps, the root and its 6, quotient,
    # eps 1e-8 beside a gradient, the product and the difference.
    want = before.double() - 0.1 * torch.sign(g[0].double()) * (g[0].double().abs() / (g[0].double().abs() + EPS))
    assert ((p[0].double() - want).abs() <= 16 * U32 * 0.1 + U32 * want.abs()).all()
    assert torch.equal(p[0][:300], before[:300])
    nsa.adamw_step(p, g, m, v, lr=0.1, step=2, scales=scales, weight_decay=0.0)
    assert torch.equal(p[0][:300], before[:300]) and torch.isfinite(p[0]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_tiny_roots_do_not_blow_the_update_up(bits):
    # One element of a block has a gradient 2^-30 of another's: its root is
    # below the smallest code, and 20 steps never move it by more than lr
    # each (a root that became 0 would let the next step go by sqrt(20) lr).
    dev = _dev()
    g = [torch.full((512,), 1.0, device=dev)]
    g[0][1::2] = 2.0 ** -30
    p = [torch.zeros(512, device=dev)]
    m, v, scales = nsa.adamw_states(p, bits=bits)
    for t in range(1, 21):
        before = p[0].clone()
        nsa.adamw_step(p, g, m, v, lr=1e-3, step=t, scales=scales, weight_decay=0.0)
        # A rounded root is off by 2^-4 and a rounded m too.
        assert (p[0] - before).abs().max().item() <= 1e-3 * (1 + 2.0 ** -3)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 3e38])
@pytest.mark.parametrize("bits", [32, 8])
def test_non_finite_results_are_reported(bits, value):
    dev = _dev()
    s = _Set([(3000,), (700,)], [torch.float32], [torch.float32], (bits,), dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    s.step(status=st)
    assert int(st.item()) == 0
    s.g[1][600] = value
    s.step(status=st)
    assert int(st.item()) == B.NS_ERR_NONFINITE | B.STATUS_AT_OUTPUT
    # Nothing outside the tensor's own block of 256 is touched by it.
    assert torch.isfinite(s.p[0]).all() and torch.isfinite(s.p[1][:512]).all()
    if bits == 8:
        assert torch.isfinite(s.scales[0]).all() and torch.isfinite(s.scales[1][:, :2]).all()
        assert torch.isfinite(s.m[1].float()[:512]).all() and torch.isfinite(s.v[1].float()[:512]).all()


def test_runs_on_the_current_stream():
    dev = _dev()
    s = _Set([(1000, 1000)], [torch.bfloat16], [torch.bfloat16], (32,), dev)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.g[0].mul_(1)
        s.step()
        got = s.p[0].clone()
    stream.synchronize()
    s.check(1e-2, 7, 0.1)
    assert torch.equal(got, s.p[0])


def test_python_refusals():
    dev = _dev()
    p, g = [torch.zeros(300, device=dev)], [torch.zeros(300, device=dev)]
    m, v, _ = nsa.adamw_states(p)
    m8, v8, s8 = nsa.adamw_states(p, bits=8)

    def call(p=p, g=g, m=m, v=v, **kw):
        nsa.adamw_step(p, g, m, v, lr=kw.pop("lr", 1e-3), step=kw.pop("step", 1), **kw)

    call()
    call(m=m8, v=v8, scales=s8)
    for kw, error in [
            (dict(g=[]), ValueError), (dict(scales=[None, None]), ValueError), (dict(copies=[]), ValueError),
            (dict(p=[torch.zeros(300)]), ValueError), (dict(g=[torch.zeros(300)]), ValueError),
            (dict(g=[torch.zeros(299, device=dev)]), ValueError),
            (dict(g=[torch.zeros(300, dtype=torch.float64, device=dev)]), TypeError),
            (dict(p=[torch.zeros(600, device=dev)[::2]]), ValueError),
            (dict(m=m8, v=v8), ValueError), (dict(scales=s8), ValueError), (dict(m=m8), TypeError),
            (dict(m=m8, v=v8, scales=[torch.zeros(2, 1, device=dev)]), ValueError),
            (dict(m=[torch.zeros(300, dtype=torch.float16, device=dev)]), TypeError),
            (dict(copies=[torch.zeros(299, device=dev)]), ValueError),
            (dict(v=m), ValueError), (dict(copies=p), ValueError),
            (dict(lr=[1.0, 2.0]), ValueError), (dict(step=0), ValueError),
            (dict(step=torch.ones(1, dtype=torch.int64, device=dev)), TypeError),
            (dict(step=torch.ones(2, dtype=torch.int32, device=dev)), ValueError),
            (dict(grad_scale=torch.ones(1)), ValueError), (dict(grad_scale=2.0), TypeError),
            (dict(lr_scale=torch.ones(1, dtype=torch.float64, device=dev)), TypeError),
            (dict(lr=float("nan")), nsa.NSError), (dict(betas=(1.0, 0.9)), nsa.NSError),
            (dict(betas=(0.9, -0.1)), nsa.NSError), (dict(eps=-1.0), nsa.NSError),
            (dict(weight_decay=float("inf")), nsa.NSError)]:
        with pytest.raises(error):
            call(**kw)
    with pytest.raises(ValueError):
        nsa.adamw_states(p, bits=16)
    # The same tensor twice in one list.
    with pytest.raises(ValueError, match="twice"):
        nsa.adamw_step(p * 2, g * 2, m + [m[0].clone()], v + [v[0].clone()], lr=1e-3, step=1)
    nsa.adamw_step([], [], [], [], lr=1e-3, step=1)
