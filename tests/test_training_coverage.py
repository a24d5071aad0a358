"""The GPU cases of the training step's operators reach every kernel build.

Host only: plan_linear_cross_entropy names the builds that a call launches
without touching a device.
"""

import itertools
import os
import re

import pytest
import torch

from newton_schulz_matrix_amd import _binding as B
import newton_schulz_matrix_amd as nsa

from training_cases import XENT_RUNS

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH),
                                reason="libnsortho.so not built")

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GROUPS = 256  # work-groups of the products' persistent grids

ROWS = [1, 2, 3, 4, 5, 8, 9, 40, 128, 129, 200, 385, 500, 1000, 1025, 3000, 9000, 16384, 20000]
COLS = [1, 3, 5, 64, 72, 77, 200, 768, 1000, 1408, 4096]
VOCABS = [1, 100, 1000, 8191, 32003, 50257, 128000]


def _plan(n, d, v, dtype, aligned, backward):
    return nsa.plan_linear_cross_entropy(n, d, v, DTYPES[dtype], aligned=aligned, backward=backward)


def _builds(plan):
    """The builds of a plan; a gradient's also with whether dH adds up over pieces."""
    names = [e for e in plan if "=" not in e]
    several = [e for e in plan if e.startswith("pieces=") and e != "pieces=1"]
    return set(names) | ({e + " several pieces" for e in names if e.startswith("grads")} if several else set())


def test_the_cases_reach_every_cross_entropy_build():
    every, covered = set(), set()
    for n, d, v, dtype, aligned, backward in itertools.product(ROWS, COLS, VOCABS, DTYPES, (True, False), (True, False)):
        every |= _builds(_plan(n, d, v, dtype, aligned, backward))
    for n, d, v, dtype in XENT_RUNS:
        for backward in (True, False):
            covered |= _builds(_plan(n, d, v, dtype, True, backward))
    assert every - covered == set()
    # Both edges of both products, all three types.
    for t, edges in (("bf16", (128, 192)), ("f16", (128, 192)), ("f32", (64, 128))):
        for e in edges:
            assert {f"dz<{t},{e}>", f"grads<{t},{e}>", f"grads<{t},{e}> several pieces", f"fwd<{t},{e}x{e}>"} <= covered


def test_the_cases_give_work_groups_several_long_tiles():
    # What the waits at a tile's border count on shows only where a
    # work-group goes from one tile to another and a tile is longer than the
    # LDS stages: every dz and grads build has a case of that kind.
    dz, grads = set(), set()
    for n, d, v, dtype in XENT_RUNS:
        plan = _plan(n, d, v, dtype, True, True)
        edge = int(re.search(r",(\d+)>", plan[1])[1])
        pieces, splits = (int(e.split("=")[1]) for e in plan[-2:])
        ktile = 32 if dtype == "fp32" else 64
        up = lambda a, b: -(-a // b)  # noqa: E731
        rows, cols, width = up(n, edge), up(d, edge), up(up(v, pieces), edge)
        if rows * width > GROUPS and up(d, ktile) > 3:
            dz.add((dtype, edge))
        if cols * width > GROUPS and rows * edge // ktile > 3:
            grads.add((dtype, edge, "dw"))
        if rows * cols * splits > GROUPS and width * edge // ktile // splits > 3:
            grads.add((dtype, edge, "dh"))
    for t, edges in (("bf16", (128, 192)), ("fp16", (128, 192)), ("fp32", (64, 128))):
        for e in edges:
            assert (t, e) in dz, (t, e)
            assert {(t, e, "dw"), (t, e, "dh")} <= grads, (t, e, grads)


def test_plan_query_refusals_and_truncation():
    for n, d, v in ((-1, 8, 8), (8, 0, 8), (8, 8, 0), (1 << 23, 8, 1 << 23)):
        with pytest.raises(nsa.NSError):
            nsa.plan_linear_cross_entropy(n, d, v)
    with pytest.raises(TypeError):
        nsa.plan_linear_cross_entropy(8, 8, 8, torch.float64)
    assert nsa.plan_linear_cross_entropy(0, 8, 8) == []
    assert nsa.plan_linear_cross_entropy(0, 8, 8, torch.float32, backward=True) == ["zero<f32>"]
    import ctypes
    fn = B.lib().ns_plan_linear_cross_entropy
    assert fn(8, 8, 8, 5, 1, 1, None, 0) == -1
    need = fn(300, 64, 500, B.NS_BF16, 1, 1, None, 0)
    buf = ctypes.create_string_buffer(b"\x7f" * 40, 40)
    assert fn(300, 64, 500, B.NS_BF16, 1, 1, buf, 9) == need
    whole = " ".join(nsa.plan_linear_cross_entropy(300, 64, 500, backward=True))
    assert need == len(whole) + 1 and buf.raw[:9] == whole[:8].encode() + b"\0" and buf.raw[9:40] == b"\x7f" * 31
