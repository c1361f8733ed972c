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


def test_workspaces_are_kept_for_the_stream_they_are_used_on(monkeypatch):
    """A workspace that a call allocates and drops is recorded on the stream that
    the call names: its memory is not handed out again while the kernels run."""
    import torch

    import ternary_weight_linear_absmax_b200 as bl

    class OnGpu(torch.Tensor):
        is_cuda = True

        def record_stream(self, stream):
            seen.append((self.dtype, self.numel(), stream))

    class Stream:
        cuda_stream = 77

    class Library:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: 4096
            return lambda *a: calls.append((name, a[-1])) or 0

    seen, calls, stream = [], [], Stream()
    real = torch.empty
    monkeypatch.setattr(bl, "load", lambda: Library())
    monkeypatch.setattr(torch, "empty", lambda *a, **k: real(*a, dtype=k["dtype"]).as_subclass(OnGpu))

    def t(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)

    M, K, N, i8, u8 = 8, 64, 64, torch.int8, torch.uint8
    x, w, one = t(M, K), t(N, K // 4, dtype=u8), t(1)
    a, acc = t(M, K, dtype=i8), t(M, N, dtype=torch.int32)
    with_workspace = [
        lambda **k: bl.bl_quant_weights(t(N, K), **k), lambda **k: bl.bl_zero_gemm(a, w, **k),
        lambda **k: bl.bl_linear_q(a, t(M), w, one, **k), lambda **k: bl.bl_linear(x, w, one, **k),
        lambda **k: bl.bl_ffn_relu2(x, w, one, w, one, **k), lambda **k: bl.bl_linear_taps(x, w, one, **k),
        lambda **k: bl.bl_ffn_relu2_taps(x, w, one, w, one, **k), lambda **k: bl.bl_ffn_tp_up(x, w, one, **k),
        lambda **k: bl.bl_ffn_tp_down(acc, t(M), one, t(M), w, **k),
        lambda **k: bl.bl_ste_grad_input(x, w, one, **k),
        lambda **k: bl.bl_ste_grad_weight(x, a, t(M), t(N, K), one, **k)]
    for call in with_workspace:
        seen.clear()
        calls.clear()
        call(stream=stream)
        assert [s for _, s in calls] == [77]
        assert seen == [(u8, 4096, stream)], calls
    given = t(4096, dtype=u8)                  # a workspace of the caller's is the caller's to keep
    seen.clear()
    bl.bl_linear(x, w, one, workspace=given, stream=stream)
    assert seen == []


def _fake_block(monkeypatch, calls):
    """A PreNormFFN of stand-in tensors on cuda:1; what it calls is only noted,
    with the device that is current then."""
    import torch

    import ternary_weight_linear_absmax_b200 as bl
    from ternary_weight_linear_absmax_b200 import prenorm_ffn as pf

    class OnGpu(torch.Tensor):
        is_cuda = True
        dev = 1

        def get_device(self):
            return self.dev

    def t(dev=1):
        x = torch.zeros(2, 2).as_subclass(OnGpu)
        x.dev = dev
        return x

    current = [0]

    class DeviceOf:
        def __init__(self, tensor):
            self.dev = tensor.get_device()

        def __enter__(self):
            self.before, current[0] = current[0], self.dev

        def __exit__(self, *exc):
            current[0] = self.before

    monkeypatch.setattr(torch.cuda, "device_of", DeviceOf)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(bl, "_raw_stream", lambda dev: 0)
    outputs = {"bl_layernorm_quant": 6, "bl_relu2_requant_q8": 5, "bl_layernorm_grad_q8": 3}
    for name in ("bl_layernorm_quant", "bl_zero_gemm", "bl_relu2_requant_q8", "bl_linear_q", "bl_ste_grad_weight",
                 "bl_ste_grad_input", "bl_relu2_grad_q8", "bl_layernorm_grad_q8"):
        def fake(*a, name=name, **k):
            calls.append((name, current[0]))
            return tuple(t() for _ in range(outputs[name])) if name in outputs else t()
        monkeypatch.setattr(pf, name, fake)
    return pf.PreNormFFN(t(), t(), t(), t(), t(), t()), t


def test_block_runs_on_its_inputs_device(monkeypatch):
    """The block on a device that is not the current one: every call is made with
    the input's device current, and the one before is current again afterwards."""
    import torch
    calls = []
    blk, t = _fake_block(monkeypatch, calls)
    y, saved = blk.forward(t())
    blk.decode(t())
    blk.backward(t(), saved, t(), t())
    assert len(calls) == 4 + 4 + 6 and {dev for _, dev in calls} == {1}, calls
    assert torch._C._cuda_getDevice() == 0


def test_block_refuses_tensors_of_other_devices(monkeypatch):
    """A matrix, a scale or latent weights on another device than the input are
    refused before any kernel gets their address."""
    import pytest
    calls = []
    blk, t = _fake_block(monkeypatch, calls)
    _, saved = blk.forward(t())
    for name in ("W_up", "W_down", "gamma_down"):
        kept = getattr(blk, name)
        setattr(blk, name, t(0))
        calls.clear()
        for run in (lambda: blk.forward(t()), lambda: blk.decode(t()), lambda: blk.backward(t(), saved, t(), t())):
            with pytest.raises(ValueError, match="expected cuda:1"):
                run()
        assert calls == []
        setattr(blk, name, kept)
    for latent in ((t(0), t()), (t(), t(0))):
        calls.clear()
        with pytest.raises(ValueError, match="expected cuda:1"):
            blk.backward(t(), saved, *latent)
        assert calls == []
    calls.clear()
    with pytest.raises(ValueError, match="expected cuda:0"):
        blk.backward(t(0), saved, t(), t())       # not where the forward ran
    assert calls == []
