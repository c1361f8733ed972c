"""Refusals of the 4-bit weight, layer norm and checkpoint entry points: by the
library on the host before any CUDA call, and by the binding (no GPU needed)."""
import ctypes

import pytest
import torch

BAD_ARG, BAD_SHAPE, BAD_ALIGN, BAD_DTYPE, BAD_WS = 1, 2, 3, 4, 8


@pytest.fixture(scope="module")
def lib():
    from ternary_weight_linear_absmax_b200 import _lib
    from ternary_weight_linear_absmax_b200 import build as b
    b.build()
    return _lib.load()


@pytest.fixture(scope="module")
def p():
    buf = ctypes.create_string_buffer(4096 + 64)
    yield (ctypes.addressof(buf) + 15) & ~15


def test_sizes(lib):
    assert lib.bl_w4_bytes(1, 64) == 1024
    assert lib.bl_w4_bytes(17, 192) == 2 * 2 * 1024
    assert lib.bl_w4_bytes(0, 64) == 0
    assert lib.bl_w4_scale_count(17, 192, 32) == 2 * 2 * 16 * 4
    assert lib.bl_w4_scale_count(17, 192, 48) == 0
    assert lib.bl_w4_bytes(1 << 30, 1 << 20) == (1 << 26) * (1 << 13) * 1024
    assert lib.bl_layernorm_grad_workspace_bytes(0, 64) == 0
    assert lib.bl_layernorm_grad_workspace_bytes(1, 64) >= 2 * 64 * 4


def test_w4_refusals(lib, p):
    q = lib.bl_quant_weights_w4
    assert q(p, 7, 16, 64, 32, p, p, None, None) == BAD_DTYPE
    assert q(p, 0, 16, 100, 32, p, p, None, None) == BAD_SHAPE
    assert q(p, 0, -1, 64, 32, p, p, None, None) == BAD_SHAPE
    assert q(p, 0, 16, 64, 16, p, p, None, None) == BAD_SHAPE
    assert q(None, 0, 16, 64, 32, p, p, None, None) == BAD_ARG
    assert q(p, 0, 16, 64, 32, p + 8, p, None, None) == BAD_ALIGN
    assert q(p, 0, 16, 64, 32, p, p, p + 1, None) == BAD_ALIGN
    assert q(p, 0, 0, 64, 32, p, p, None, None) == 0
    k = lib.bl_pack_w4
    assert k(p, p, None, 16, 64, 32, p, p, p, None) == BAD_ARG     # zeros in without zeros out
    assert k(p, p, p, 16, 64, 32, p, p, None, None) == BAD_ARG
    assert k(p, p, None, 16, 64, 0, p, p, None, None) == BAD_SHAPE
    assert k(p, None, None, 16, 64, 32, p, p, None, None) == BAD_ARG
    u = lib.bl_unpack_w4
    assert u(p, p, None, 16, 64, 32, p, 9, None) == BAD_DTYPE
    assert u(p, p, None, 16, 63, 32, p, 0, None) == BAD_SHAPE
    assert u(p, p, None, 16, 64, 32, None, 0, None) == BAD_ARG
    f = lib.bl_linear_w4
    assert lib.bl_linear_w4_workspace_bytes(5, 64, 32) == 0
    assert lib.bl_linear_w4_workspace_bytes(6, 128, 128) >= 6 * 3 * 128
    assert lib.bl_linear_w4_workspace_bytes(17, 128, 128) >= 2 * 16 * 3 * 128
    assert f(p, 0, 6, 64, p, p, None, 16, 32, p, 1, None, 0, 0, None) == BAD_WS
    assert f(p, 0, 6, 64, p, p, None, 16, 32, p, 1, p, 64, 0, None) == BAD_WS
    assert f(p, 0, 6, 64, p, p, None, 16, 32, p, 1, p + 8, 1 << 20, 0, None) == BAD_ALIGN
    assert f(p, 1, 1, 64, p, p, None, 16, 96, p, 1, None, 0, 0, None) == BAD_SHAPE
    assert f(p, 1, 1, 96, p, p, None, 16, 32, p, 1, None, 0, 0, None) == BAD_SHAPE
    assert f(p, 1, 1, (1 << 22) + 64, p, p, None, 16, 32, p, 1, None, 0, 0, None) == BAD_SHAPE
    assert f(p, 1, 1, 262144 + 64, p, p, None, 16, 32, p, 1, None, 0, 0, None) == BAD_SHAPE
    assert f(None, 1, 0, 262144, None, None, None, 16, 32, None, 1, None, 0, 0, None) == 0
    assert f(p, 1, -1, 64, p, p, None, 16, 32, p, 1, None, 0, 0, None) == BAD_SHAPE
    assert f(p, 2, 1, 64, p, p, None, 16, 32, p, 1, None, 0, 0, None) == BAD_DTYPE
    assert f(p, 1, 1, 64, p, p, None, 16, 32, p, 1, None, 0, 2, None) == BAD_ARG    # BL_FLAG_RAW_I32
    assert f(p + 2, 1, 1, 64, p, p, None, 16, 32, p, 1, None, 0, 0, None) == BAD_ALIGN
    assert f(p, 1, 1, 64, p, p, None, 16, 32, None, 1, None, 0, 0, None) == BAD_ARG
    assert f(None, 1, 0, 64, None, None, None, 16, 32, None, 1, None, 0, 0, None) == 0
    assert f(None, 1, 1, 64, None, None, None, 0, 32, None, 1, None, 0, 0, None) == 0


def test_norm_refusals(lib, p):
    f = lib.bl_layernorm
    assert f(p, 1, 1, 100, p, p, 1e-5, p, 1, p, p, None) == BAD_SHAPE
    assert f(p, 1, -1, 64, p, p, 1e-5, p, 1, p, p, None) == BAD_SHAPE
    assert f(p, 3, 1, 64, p, p, 1e-5, p, 1, p, p, None) == BAD_DTYPE
    assert f(p, 1, 1, 64, p, p, 0.0, p, 1, p, p, None) == BAD_ARG
    assert f(p, 1, 1, 64, None, p, 1e-5, p, 1, p, p, None) == BAD_ARG
    assert f(p, 1, 1, 64, p, p + 4, 1e-5, p, 1, p, p, None) == BAD_ALIGN
    assert f(p, 1, 0, 64, None, None, 1e-5, None, 1, None, None, None) == 0
    q = lib.bl_layernorm_quant
    assert q(p, 1, 1, 64, p, p, 1e-5, float("inf"), p, p, p, p, p, p, None) == BAD_ARG
    assert q(p, 1, 1, 64, p, p, 1e-5, 1e-5, p, p, p, p, p, None, None) == BAD_ARG   # half a checkpoint
    assert q(p, 1, 1, 64, p, p, 1e-5, 1e-5, None, p, p, p, p, p, None) == BAD_ARG
    g = lib.bl_layernorm_grad
    assert g(p, 1, p, 1, p, p, p, 1, 64, p, 1, p, p, None, 0, None) == BAD_WS
    assert g(p, 1, p, 1, p, p, p, 1, 64, p, 1, p, p, p, 16, None) == BAD_WS
    assert g(p, 1, p, 5, p, p, p, 1, 64, p, 1, p, p, p, 4096, None) == BAD_DTYPE
    assert g(p, 1, p, 1, p, p, p, 1, 65, p, 1, p, p, p, 4096, None) == BAD_SHAPE
    assert g(p, 1, p, 1, None, p, p, 1, 64, p, 1, p, p, p, 4096, None) == BAD_ARG
    assert g(p, 1, p, 1, p, p, p, 1, 64, p, 1, None, p, p, 4096, None) == BAD_ARG
    h = lib.bl_layernorm_grad_q8
    assert h(p, 1, p, None, p, p, 1, 64, p, 1, p, p, p, 4096, None) == BAD_ARG
    assert h(p, 1, p, p + 4, p, p, 1, 64, p, 1, p, p, p, 4096, None) == BAD_ALIGN
    assert h(p, 1, p, p, p, p, 1, 64, p, 1, p, p, p, 8, None) == BAD_WS


def test_relu2_refusals(lib, p):
    f = lib.bl_relu2_requant_q8
    assert f(p, p, p, 1, 100, 1e-5, p, p, p, p, p, None) == BAD_SHAPE
    assert f(p, p, p, 1, 64, -1.0, p, p, p, p, p, None) == BAD_ARG
    assert f(p, p, None, 1, 64, 1e-5, p, p, p, p, p, None) == BAD_ARG
    assert f(p, p, p, 1, 64, 1e-5, p, p, p, p + 1, p, None) == BAD_ALIGN
    assert f(p, p, p, 1, 64, 1e-5, p, p, p, p, None, None) == BAD_ARG      # half a checkpoint
    assert f(None, None, None, 0, 64, 1e-5, None, None, None, None, None, None) == 0
    g = lib.bl_relu2_grad_q8
    assert g(p, 0, p, p, 1, 32, p, 1, None) == BAD_SHAPE
    assert g(p, 0, p, p, 1, 64, p, 4, None) == BAD_DTYPE
    assert g(p, 0, p, None, 1, 64, p, 1, None) == BAD_ARG
    assert g(None, 0, None, None, 0, 64, None, 1, None) == 0


def test_binding_refusals():
    """The binding refuses CPU tensors, wrong types and shapes, and groups that
    the format does not have, before it calls the library."""
    import ternary_weight_linear_absmax_b200 as bl
    x = torch.zeros(2, 64)
    for call in (lambda: bl.bl_quant_weights_w4(x), lambda: bl.bl_layernorm(x, x[0]),
                 lambda: bl.bl_linear_w4(x, x, x, 16), lambda: bl.bl_relu2_grad_q8(x, x, x),
                 lambda: bl.bl_layernorm_quant(x, x[0]), lambda: bl.bl_layernorm_grad(x, x, x, x, x),
                 lambda: bl.bl_relu2_requant_q8(x, x, x), lambda: bl.bl_unpack_w4(x, x, 2, 64),
                 lambda: bl.bl_pack_w4(x, x), lambda: bl.bl_layernorm_grad_q8(x, x, x, x, x)):
        with pytest.raises(TypeError, match="must be a CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="group"):
        bl.bl_quant_weights_w4(x, 48)
    W4 = torch.zeros(1, 1, 1024, dtype=torch.uint8)
    sc = torch.zeros(1, 1, 8, 2, 2, dtype=torch.bfloat16)
    assert bl._check_w4(W4, sc, None, 16, 64) == 64
    for bad in (lambda: bl._check_w4(W4, sc, None, 17, 64), lambda: bl._check_w4(W4, sc, None, 16, 192),
                lambda: bl._check_w4(W4, sc[:, :, :, :1], W4, 16, 64), lambda: bl._w4_group(sc[0]),
                lambda: bl._matrix(sc, "X")):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError, match="scales must be"):
        bl._check_w4(W4, sc.float(), None, 16, 64)
    with pytest.raises(TypeError, match="zeros must be"):
        bl._check_w4(W4, sc, sc, 16, 64)


def test_binding_refuses_missing_tensors():
    """None in the place of a tensor that a call cannot do without; those it can
    do without may be left out."""
    import ternary_weight_linear_absmax_b200 as bl
    with pytest.raises(TypeError, match="weight must be a CUDA tensor"):
        bl._on(weight=None, bias=None)
    for call in (lambda: bl.bl_quant_weights_w4(None), lambda: bl.bl_layernorm(None, None),
                 lambda: bl.bl_linear_w4(None, None, None, 16),
                 lambda: bl.bl_quant_weights_w4(group=128, W=None)):
        with pytest.raises(TypeError, match="must be a CUDA tensor"):
            call()


def test_binding_places_calls_by_any_tensor():
    """The device and stream of a call by keyword come from its first tensor,
    whatever stands before it."""
    import ternary_weight_linear_absmax_b200 as bl

    class OnGpu(torch.Tensor):
        is_cuda = True
        device = torch.device("cuda", 1)

    class Stream:
        device = torch.device("cuda", 0)

    t = torch.zeros(1).as_subclass(OnGpu)
    for kw in ({"W": t}, {"group": 32, "W": t}, {"zeros": None, "X": t}):
        with pytest.raises(ValueError, match="stream is on cuda:0"):
            bl._placed(lambda **k: None)(stream=Stream(), **kw)
