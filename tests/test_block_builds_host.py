"""Host side of the block's operators: the norms' cases reach every kernel
build, calls of the host module leave the interpreter to other threads, and
the library is built where the host module cannot be."""

import ctypes
import importlib
import importlib.util
import itertools
import os

import pytest
import torch

import newton_schulz_matrix_amd as nsa
from newton_schulz_matrix_amd import _binding as B
from newton_schulz_matrix_amd import build as nsbuild
from resnorm_cases import MORE_WIDTHS, build_of

built = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libnsortho.so not built")


def test_the_widths_reach_every_build_of_the_residual_norms():
    from test_gpu_residual_norm import WIDTHS
    types = [(2, 2), (2, 4), (4, 4)]
    every = {(t, build_of(c, *t)) for c, t in itertools.product(range(1, 8200), types)}
    covered = {(t, build_of(c, *t)) for c, t in itertools.product(WIDTHS + MORE_WIDTHS, types)}
    assert every - covered == set()
    # Element by element: less than a vector, and too long.
    assert any(c < 4 for c in WIDTHS) and any(c > 8192 for c in WIDTHS)


@built
def test_the_range_cases_reach_every_fp16_build_of_the_gated_mlp():
    from test_gpu_gated_mlp_range import SHAPES

    def builds(sizes, aligned):
        return {(e, backward) for n, d, f in sizes for backward in (False, True)
                for e in nsa.plan_gated_mlp(n, d, f, torch.float16, aligned, backward) if e.startswith(("again", "products", "join"))}

    sweep = itertools.product([5, 9, 48, 129, 300, 513, 1003, 3000, 8192, 20000], [1, 64, 77, 768, 4096], [1, 64, 203, 1407, 2048, 14336])
    every = set().union(*(builds([size], aligned) for size in sweep for aligned in (True, False)))
    assert every and every - builds(SHAPES, True) == set()


@built
def test_calls_of_the_host_module_leave_the_interpreter_to_other_threads():
    # In place of an entry point stands Python's own question whether the
    # calling thread holds the interpreter's lock: 1 would come back as a
    # status, 0 as the call's results.
    marshal = importlib.import_module("newton_schulz_matrix_amd._marshal")
    held = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    assert ctypes.pythonapi.PyGILState_Check() == 1

    def address(name):
        return ctypes.cast(getattr(B.lib(), name), ctypes.c_void_p).value

    x, w, stat = torch.zeros(6, 8), torch.zeros(8), torch.zeros(6)
    got = marshal.residual_norm(held, x, x, None, 1.0, None, w, True, True, 1e-6, True, None, None, None, 0)
    assert isinstance(got, tuple) and got[0].shape == (6, 8) and got[3].shape == (6,)
    got = marshal.residual_norm_backward(held, address("ns_residual_norm_workspace_size"), x, x, x, x, stat, stat, None, 1.0,
                                         None, w, True, None, None, None, None, 0)
    assert isinstance(got, tuple) and got[4].shape == (8,)
    wide, down = torch.zeros(16, 8), torch.zeros(8, 16)
    size = address("ns_gated_mlp_workspace_size")
    y, gate, up = marshal.gated_mlp(held, size, x, wide, wide, down, 0, True, None, None, None, 0)
    assert y.shape == (6, 8) and gate.shape == up.shape == (6, 16)
    got = marshal.gated_mlp_backward(held, size, x, wide, wide, down, x, gate, up, 0, True, True, None, None, None, None, None,
                                     None, 0)
    assert isinstance(got, tuple) and got[1].shape == (16, 8)


def _small_build(monkeypatch, tmp_path):
    """The build's paths in a folder of their own, with the shortest source."""
    try:
        nsbuild.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    monkeypatch.setattr(nsbuild, "SOURCES", ["optim.hip"])
    monkeypatch.setattr(nsbuild, "LIB_PATH", str(tmp_path / "libnsortho.so"))
    monkeypatch.setattr(nsbuild, "MARSHAL_PATH", str(tmp_path / "_marshal.so"))


def test_the_library_is_built_without_a_host_compiler(monkeypatch, tmp_path):
    _small_build(monkeypatch, tmp_path)
    monkeypatch.setenv("CXX", "/bin/false")
    with pytest.raises(RuntimeError, match="is built, but the host module"):
        nsbuild.build()
    assert hasattr(ctypes.CDLL(nsbuild.LIB_PATH), "ns_adamw_step") and not os.path.exists(nsbuild.MARSHAL_PATH)
    os.remove(nsbuild.LIB_PATH)
    monkeypatch.setenv("CXX", "no such compiler")
    with pytest.raises(RuntimeError, match="is built, but the host module"):
        nsbuild.build()
    assert os.path.exists(nsbuild.LIB_PATH)
    os.remove(nsbuild.LIB_PATH)
    assert nsbuild.build_library() == nsbuild.LIB_PATH and os.path.exists(nsbuild.LIB_PATH)


def test_the_library_is_built_without_torch(monkeypatch, tmp_path):
    _small_build(monkeypatch, tmp_path)
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: None)
    assert nsbuild.build() == nsbuild.LIB_PATH
    assert os.path.exists(nsbuild.LIB_PATH) and not os.path.exists(nsbuild.MARSHAL_PATH)
