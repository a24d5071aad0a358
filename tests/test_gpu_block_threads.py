"""Calls of the block's operators from several Python threads at once, each on a
stream of its own: the same bits as one after the other."""

import threading

import pytest
import torch

import newton_schulz_matrix_amd as nsa

pytestmark = pytest.mark.gpu


def _step(seed, dtype):
    """One block's norms, feed-forward half, gradients and AdamW; all results."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def make(*shape, scale=1.0):
        return (scale * torch.randn(*shape, device="cuda", generator=g)).to(dtype)

    n, d, f = 200 + 7 * seed, 264, 520
    x, z, dy, ds = make(n, d), make(n, d), make(n, d), make(n, d)
    wg, wu, wd = make(f, d, scale=d ** -0.5), make(f, d, scale=d ** -0.5), make(d, f, scale=f ** -0.5)
    w = torch.ones(d, device="cuda")
    out = []
    for _ in range(10):
        s, y, rb, rs = nsa.residual_norm(x, z, weight=w, branch_weight=w)
        o, gate, up = nsa.gated_mlp(y, wg, wu, wd)
        dx, dwg, dwu, dwd = nsa.gated_mlp_backward(dy, y, wg, wu, wd, gate, up)
        grads = nsa.residual_norm_backward(ds, dx, s, z, rb, rs, weight=w, branch_weight=w)
        params = [t.float() for t in (wg, wu, wd)]
        m, v, scales = nsa.adamw_states(params, bits=8)
        nsa.adamw_step(params, [dwg, dwu, dwd], m, v, lr=1e-3, step=1, scales=scales)
        out.append([s, y, o, dx, dwg, dwu, dwd, *params, *scales, *(t for t in grads if t is not None)])
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_threads_on_their_own_streams(dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    count = 4
    want = [_step(k, dtype) for k in range(count)]
    torch.cuda.synchronize()
    got, errors = [None] * count, []

    def run(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                got[k] = _step(k, dtype)
            stream.synchronize()
        except BaseException as e:  # shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(count)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert errors == [] and not any(t.is_alive() for t in threads)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for p, q in zip(a, b):
            assert all(torch.equal(s, t) for s, t in zip(p, q))
