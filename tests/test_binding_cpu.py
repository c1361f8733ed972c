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


def test_inputs_are_kept_for_the_stream_they_are_read_on(monkeypatch):
    """A call on a stream that is not its inputs' own tells torch so, for every
    tensor and however it is passed: their memory is not handed out again while
    the call runs. Without ``stream`` there is nothing to tell."""
    import contextlib

    import torch

    import ternary_weight_linear_absmax_b200 as bl

    class OnGpu(torch.Tensor):
        is_cuda = True
        device = torch.device("cuda", 0)

        def get_device(self):
            return 0

        def record_stream(self, stream):
            seen.append((id(self), stream))

    class Stream:
        device = torch.device("cuda", 0)

    seen, stream = [], Stream()
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    a, b, c = (torch.zeros(1).as_subclass(OnGpu) for _ in range(3))
    call = bl._placed(lambda *args, **kw: len(args))
    assert call(a, 3, None, b, stream=stream, out=c, pdl=True) == 4
    assert set(seen) == {(id(t), stream) for t in (a, b, c)} and len(seen) == 3
    seen.clear()
    assert call(a, b, out=c) == 2 and seen == []
