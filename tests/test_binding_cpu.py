"""The Python binding on the host: importing it, where its calls run and what
they keep alive (no GPU needed)."""
import subprocess
import sys

from conftest import ROOT


def test_import_without_a_cuda_build_of_torch():
    """A CPU build of torch lacks the CUDA names; the package imports all the
    same, since the host lookup-table library lives in it."""
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
guards = torch._C._dynamo.guards
if hasattr(guards, "_empty_strided_cuda"):
    del guards._empty_strided_cuda
import ternary_weight_linear_absmax_b200 as bl
from ternary_weight_linear_absmax_b200 import lut_cpu
try:
    bl.bl_layernorm(torch.zeros(2, 64), torch.zeros(64))
except TypeError as e:
    assert "must be a CUDA tensor" in str(e)
else:
    raise AssertionError("accepted a CPU tensor")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
