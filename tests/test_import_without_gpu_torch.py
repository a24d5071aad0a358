"""The package imports, and its host-only parts work, with a torch whose
private stream functions are missing (a build for no GPU has none)."""

import os
import subprocess
import sys

import pytest

from newton_schulz_matrix_amd import _binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import newton_schulz_matrix_amd as nsa
assert nsa.gram_flops(64, 128, 5) > 0
assert len(nsa.root_coefficients(2048, 8192)) == 5
x = torch.zeros(4, 8)
try:
    nsa.layer_norm(x)
except ValueError as e:
    assert "device tensor" in str(e)
else:
    raise AssertionError("a host tensor was not refused")
if BUILT:
    assert nsa.plan_kernels(64, 128)
    assert nsa.layer_norm_workspace_size(4, 8) > 0
print("fine")
"""


def test_import_and_host_parts():
    program = PROGRAM.replace("BUILT", str(os.path.exists(B.LIB_PATH)))
    got = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "fine" in got.stdout, got.stderr


@pytest.mark.gpu
def test_calls_without_the_private_stream_function():
    # On a GPU the public function serves in its place, also on another stream
    # than the default one.
    program = """
import torch
del torch._C._cuda_getCurrentRawStream
import newton_schulz_matrix_amd as nsa
from newton_schulz_matrix_amd import _training as T
x = torch.randn(50, 96, device="cuda")
want = nsa.layer_norm(x)
s = torch.cuda.Stream()
s.wait_stream(torch.cuda.default_stream())
with torch.cuda.stream(s):
    assert T._raw_stream(0) == s.cuda_stream
    got = nsa.layer_norm(x)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("fine")
"""
    got = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "fine" in got.stdout, got.stderr
