"""AdamW where its states run out of range: a NaN gradient among 8-bit
moments, second moments below the smallest normal number, and codes and
scales that are the documented fp32 formula's to the bit.
"""

import numpy as np
import pytest
import torch

import newton_schulz_matrix_amd as nsa
from newton_schulz_matrix_amd import _binding as B
from test_gpu_adamw import BETAS, DTYPES, U32, _Set, _dev

pytestmark = pytest.mark.gpu

NAN_CODE = 0x7F  # e4m3's NaN but for its sign


def _codes(t):
    return t.view(torch.uint8)


@pytest.mark.parametrize("place", [0, 255, 600, 767, 999])
@pytest.mark.parametrize("ptype", ["bf16", "fp32"])
def test_a_nan_stays_in_its_element(place, ptype):
    # Two runs that differ in one element of one gradient, whose moments are
    # zeros, so that without the NaN it has no share in its block's scales.
    dev = _dev()
    print(f"adamw nan at {place} {ptype}", flush=True)
    sets = [_Set([(1000,)], [DTYPES[ptype]], [torch.float32], (8,), dev, seed=2) for _ in range(2)]
    other = torch.ones(1000, dtype=torch.bool, device=dev)
    other[place] = False
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    for s, value in zip(sets, (0.0, float("nan"))):
        _codes(s.m[0])[place] = 0
        _codes(s.v[0])[place] = 0
        s.g[0][place] = value
        st.zero_()
        s.step(status=st)
        assert int(st.item()) == (B.NS_ERR_NONFINITE | B.STATUS_AT_OUTPUT if value else 0)
    plain, hit = sets
    for step in (7, 8, 9):
        assert torch.equal(plain.scales[0], hit.scales[0])
        for a, b in ((plain.p[0], hit.p[0]), (_codes(plain.m[0]), _codes(hit.m[0])), (_codes(plain.v[0]), _codes(hit.v[0]))):
            assert torch.equal(a[other], b[other])
        assert torch.isnan(hit.p[0][place])
        assert int(_codes(hit.m[0])[place]) & 0x7F == NAN_CODE and int(_codes(hit.v[0])[place]) & 0x7F == NAN_CODE
        # What follows moves the others as ever.
        before = plain.p[0].clone()
        for s in sets:
            s.g[0].copy_(s.before[0][1]).mul_(0.5)
            s.step(step=step + 1)
        assert (plain.p[0] != before)[other].float().mean().item() > 0.5


def test_a_nan_second_moment_in_fp32_is_not_a_large_one():
    dev = _dev()
    s = _Set([(700,)], [torch.float32], [torch.float32], (32,), dev)
    s.v[0][300] = float("nan")
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    s.step(status=st)
    assert int(st.item()) == B.NS_ERR_NONFINITE | B.STATUS_AT_OUTPUT
    assert torch.isnan(s.p[0][300]) and int(torch.isnan(s.p[0]).sum()) == 1


def test_second_moments_below_the_normal_numbers():
    # g = 0 and betas of a half: v is exactly halved.  Without eps the step is
    # lr m / sqrt(v), by the root's half step, its correction factor's and
    # product's (1 each, c2 is 1 here), the reciprocal's step (2 halves), lr c1 m
    # (2) and the sum.
    dev = _dev()
    rng = np.random.default_rng(1)
    bits = np.concatenate([2 ** np.arange(23), [3, 5, 7, 1000, 0x7FFFFF, 0x3FFFFF], rng.integers(1, 1 << 22, 300),
                           0x00800000 * np.arange(1, 60) + rng.integers(0, 1 << 23, 59)]).astype(np.uint32)
    half = bits.view(np.float32)
    v0 = (half.astype(np.float64) * 2).astype(np.float32)
    m0 = (2 * np.sqrt(half.astype(np.float64)) * rng.uniform(0.5, 2.0, half.size)).astype(np.float32)
    p, g = torch.zeros(half.size, device=dev), torch.zeros(half.size, device=dev)
    m, v = torch.from_numpy(m0).to(dev), torch.from_numpy(v0).to(dev)
    nsa.adamw_step([p], [g], [m], [v], lr=1.0, step=2000, betas=(0.5, 0.5), eps=0.0, weight_decay=0.0)
    assert np.array_equal(v.cpu().numpy(), half)
    want = -(m0.astype(np.float64) / 2) / np.sqrt(half.astype(np.float64))
    off = np.abs(p.cpu().double().numpy() - want) / np.abs(want)
    print(f"small moments: worst {off.max() / U32:.2f} half steps of fp32", flush=True)
    assert off.max() <= 8 * U32


def _formula(g, cm, cv, scales, betas):
    """Codes and scales after a step, one rounded fp32 operation at a time."""
    f = np.float32
    b1, a1, b2, a2 = f(betas[0]), f(1.0 - betas[0]), f(betas[1]), f(1.0 - betas[1])
    n = g.size
    unit = np.repeat(scales * (f(1) / f(448)), 256, axis=1)[:, :n]
    with np.errstate(under="ignore"):
        m, r = cm * unit[0], cv * unit[1]
        v = r * r
        m = b1 * m + a1 * g
        v = b2 * v + a2 * g * g
        root = np.sqrt(v)
        tops, codes = [], []
        for x in (m, root):
            top = np.maximum(np.abs(np.pad(x, (0, -n % 256))).reshape(-1, 256).max(1), f(2.0 ** -100))
            inv = f(1) / top * f(448)
            q = x * np.repeat(inv, 256)[:n]
            if x is root:
                q = np.where(root > 0, np.maximum(q, f(2.0 ** -9)), q)
            assert q.dtype == np.float32 and top.dtype == np.float32
            tops.append(top)
            codes.append(torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8))
    return codes, np.stack(tops)


# The other sizes are beyond fp16's numbers.
@pytest.mark.parametrize("gtype,size", [(t, 1.0) for t in DTYPES] + [(t, 2.0 ** e) for t in ("bf16", "fp32")
                                                                      for e in (-72, -66, -40, 40)])
@pytest.mark.parametrize("n", [1, 255, 256, 1003, 50001])
def test_codes_and_scales_are_the_formulas_to_the_bit(n, gtype, size):
    dev = _dev()
    s = _Set([(n,)], [torch.float32], [DTYPES[gtype]], (8,), dev, seed=n)
    s.scales[0].mul_(size)
    s.g[0].mul_(size)
    if n > 300:
        s.g[0][:256] = 0  # a block that only decays
    c = [t.float().cpu().numpy() for t in (s.g[0], s.m[0], s.v[0])]
    scales = s.scales[0].cpu().numpy()
    for step in range(1, 4):
        codes, tops = _formula(*c, scales, BETAS)
        s.step(step=step)
        assert np.array_equal(s.scales[0].cpu().numpy(), tops)
        assert torch.equal(_codes(s.m[0]).cpu(), codes[0]) and torch.equal(_codes(s.v[0]).cpu(), codes[1])
        c[1:] = [t.float().cpu().numpy() for t in (s.m[0], s.v[0])]
        scales = tops
