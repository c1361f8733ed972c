"""BitNet b1.58 BitLinear forward on B200 (sm_100a): Python binding.

Thin marshalling layer over the C ABI of ``libbitlinear.so``
(``include/bitlinear.h``): each function has the name of the C entry point,
takes CUDA ``torch.Tensor`` arguments, allocates outputs and workspace with
torch, and passes raw device pointers plus the current CUDA stream. Every
computation happens in the library's CUDA kernels; there is no fallback.

Method: "BitNet b1.58 — quantização ternária, BitLinear, Zero-GEMM" (AbsMean
ternary weights, AbsMax per-token INT8 activations, INT32 add/subtract/skip
contraction, dequantisation by γ·γ_A/127) with the API names of the
utils/bit_layers.py library of "Arquitetura Hibrida Multimodal para
bitnet.cpp" (quantise_weights_ternary, quantise_activations_8bit, BitLinear,
ReLUSquared).
"""
from __future__ import annotations

import functools

import torch

from . import _lib
from ._lib import BL_BF16, BL_F32, BL_FLAG_PDL, BL_FLAG_RAW_I32, BitLinearError, BlTaps, check, load

__all__ = [
    "bl_quant_weights", "bl_quant_acts", "bl_zero_gemm", "bl_linear_q", "bl_linear",
    "bl_linear_noalloc", "bl_ffn_relu2", "bl_linear_taps", "bl_ffn_relu2_taps",
    "bl_ffn_tp_up", "bl_ffn_tp_down", "bl_dequant_i32", "bl_ste_grad_input", "bl_ste_grad_weight",
    "bl_pack_radix3", "bl_linear_radix3", "bl_pack_lut_index", "bl_linear_lut",
    "bl_quant_weights_w4", "bl_pack_w4", "bl_unpack_w4", "bl_linear_w4",
    "bl_layernorm", "bl_layernorm_quant", "bl_layernorm_grad", "bl_layernorm_grad_q8",
    "bl_relu2_requant_q8", "bl_relu2_grad_q8",
    "bl_probe_pdl_floor", "bl_check_device_error", "bl_selftest_wait_timeout",
    "bl_gemv_max_tokens", "bl_contraction_path", "workspace_bytes", "BitLinearError", "load", "BL_FLAG_PDL",
]

_DT = {torch.float32: BL_F32, torch.bfloat16: BL_BF16}


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _dt(t: torch.Tensor, what: str) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"{what}: dtype {t.dtype} not supported (float32 or bfloat16)")
    return _DT[t.dtype]


def _cuda(t: torch.Tensor, what: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t


def _shape(t: torch.Tensor, shape: tuple, what: str) -> None:
    """The library takes plain pointers and sizes: every tensor handed to it
    must have exactly the shape the sizes describe, or a kernel would read or
    write past it."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _atleast(t: torch.Tensor, n: int, what: str) -> None:
    if t.numel() < n:
        raise ValueError(f"{what} must hold at least {n} elements, got {t.numel()}")


def _ws(nbytes: int, device, stream=None) -> torch.Tensor | None:
    """Workspace of one call. It is dropped when the call returns, while the
    kernels may still run: recorded on the stream that they run on."""
    if nbytes == 0:
        return None
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if stream is not None:
        t.record_stream(stream)
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def bl_gemv_max_tokens() -> int:
    return int(load().bl_gemv_max_tokens())


def bl_contraction_path(M: int, N: int, K: int, sms: int, split_ws_bytes: int = 0) -> int:
    """Kernel that contracts M int8 tokens with an N × K packed matrix on a
    device of `sms` SMs: 0 GEMV, 1 warp-level int8 MMA, 2 tensor-core tiles,
    3 tensor-core tiles with K split (-1: invalid sizes). Host logic only."""
    return int(load().bl_contraction_path(M, N, K, sms, split_ws_bytes))


def workspace_bytes(op: str, M: int, K: int, N: int) -> int:
    """Workspace size for 'quant_weights', 'zero_gemm', 'linear_q', 'linear'
    or 'ffn' (for 'ffn', N is the hidden size H)."""
    L = load()
    if op == "quant_weights":
        return int(L.bl_quant_weights_workspace_bytes(N, K))
    return int(getattr(L, f"bl_{op}_workspace_bytes" if op != "ffn" else "bl_ffn_workspace_bytes")(M, K, N))


def bl_quant_weights(W: torch.Tensor, eps: float = 1e-5, *, out=None, gamma=None,
                     workspace=None, stream=None):
    """quantise_weights_ternary: W [N, K] fp32/bf16 → (packed uint8 [N, K/4], γ fp32 [1])."""
    _cuda(W, "W")
    N, K = W.shape
    if out is None:
        out = torch.empty((N, K // 4), dtype=torch.uint8, device=W.device)
    _cuda(out, "out")
    _shape(out, (N, K // 4), "out")
    if gamma is None:
        gamma = torch.empty((1,), dtype=torch.float32, device=W.device)
    _cuda(gamma, "gamma")
    _atleast(gamma, 1, "gamma")
    L = load()
    if workspace is None:
        workspace = _ws(int(L.bl_quant_weights_workspace_bytes(N, K)), W.device, stream)
    else:
        _cuda(workspace, "workspace")
    check(L.bl_quant_weights(W.data_ptr(), _dt(W, "W"), N, K, float(eps), out.data_ptr(),
                             gamma.data_ptr(), _ptr(workspace), _nbytes(workspace),
                             _stream(stream)), "bl_quant_weights")
    return out, gamma


def bl_quant_acts(A: torch.Tensor, eps: float = 1e-5, *, rowsum: bool = True, stream=None):
    """quantise_activations_8bit: A [M, K] → (A_q int8 [M,K], γ_A fp32 [M], Σ A_q int32 [M] or None)."""
    _cuda(A, "A")
    M, K = A.shape
    Aq = torch.empty((M, K), dtype=torch.int8, device=A.device)
    gA = torch.empty((M,), dtype=torch.float32, device=A.device)
    rs = torch.empty((M,), dtype=torch.int32, device=A.device) if rowsum else None
    check(load().bl_quant_acts(A.data_ptr(), _dt(A, "A"), M, K, float(eps), Aq.data_ptr(),
                               gA.data_ptr(), _ptr(rs), _stream(stream)), "bl_quant_acts")
    return Aq, gA, rs


def bl_zero_gemm(A_q: torch.Tensor, W_packed: torch.Tensor, *, stream=None):
    """INT32 contraction acc[M, N] = A_q · W_qᵀ."""
    _cuda(A_q, "A_q")
    _cuda(W_packed, "W_packed")
    M, K = A_q.shape
    N = W_packed.shape[0]
    if W_packed.shape[1] * 4 != K:
        raise ValueError("W_packed must be [N, K/4]")
    acc = torch.empty((M, N), dtype=torch.int32, device=A_q.device)
    L = load()
    ws = _ws(int(L.bl_zero_gemm_workspace_bytes(M, K, N)), A_q.device, stream)
    check(L.bl_zero_gemm(A_q.data_ptr(), M, K, W_packed.data_ptr(), N, acc.data_ptr(), _ptr(ws),
                         _nbytes(ws), _stream(stream)), "bl_zero_gemm")
    return acc


def bl_linear_q(A_q, gamma_A, W_packed, gamma, *, rowsum=None, relu2=False,
                out_dtype=torch.bfloat16, out=None, pdl=False, stream=None):
    """Y = (A_q·W_qᵀ)·(γ_A·γ)/127 (ReLU² optional) from int8 tokens.
    pdl: BL_FLAG_PDL (the kernel before this call does not write W_packed)."""
    for t, n in ((A_q, "A_q"), (gamma_A, "gamma_A"), (W_packed, "W_packed"), (gamma, "gamma")):
        _cuda(t, n)
    M, K = A_q.shape
    N = W_packed.shape[0]
    _shape(W_packed, (N, K // 4), "W_packed")
    if K % 4:
        raise ValueError("K must be a multiple of 4")
    _atleast(gamma_A, M, "gamma_A")
    _atleast(gamma, 1, "gamma")
    if rowsum is not None:
        _cuda(rowsum, "rowsum")
        _atleast(rowsum, M, "rowsum")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=A_q.device)
    _cuda(out, "out")
    _shape(out, (M, N), "out")
    L = load()
    ws = None if rowsum is not None else _ws(int(L.bl_linear_q_workspace_bytes(M, K, N)), A_q.device, stream)
    check(L.bl_linear_q_ex(A_q.data_ptr(), gamma_A.data_ptr(), _ptr(rowsum), M, K,
                           W_packed.data_ptr(), gamma.data_ptr(), N, int(bool(relu2)),
                           out.data_ptr(), _dt(out, "out"), _ptr(ws), _nbytes(ws),
                           BL_FLAG_PDL if pdl else 0, _stream(stream)), "bl_linear_q")
    return out


def bl_linear(A, W_packed, gamma, eps: float = 1e-5, *, relu2=False, out_dtype=torch.bfloat16,
              out=None, workspace=None, pdl=False, stream=None):
    """BitLinear forward: Y [M, N] = dequant(quant(A) · W_qᵀ), ReLU² optional."""
    _cuda(A, "A")
    _cuda(W_packed, "W_packed")
    _cuda(gamma, "gamma")
    M, K = A.shape
    N = W_packed.shape[0]
    _shape(W_packed, (N, K // 4), "W_packed")
    _atleast(gamma, 1, "gamma")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=A.device)
    _cuda(out, "out")
    _shape(out, (M, N), "out")
    L = load()
    if workspace is None:
        workspace = _ws(int(L.bl_linear_workspace_bytes(M, K, N)), A.device, stream)
    else:
        _cuda(workspace, "workspace")
    check(L.bl_linear_ex(A.data_ptr(), _dt(A, "A"), M, K, W_packed.data_ptr(), gamma.data_ptr(),
                         N, float(eps), int(bool(relu2)), out.data_ptr(), _dt(out, "out"),
                         _ptr(workspace), _nbytes(workspace), BL_FLAG_PDL if pdl else 0,
                         _stream(stream)), "bl_linear")
    return out


def bl_linear_noalloc(A, W_packed, gamma, eps: float = 1e-5, *, relu2=False,
                      out_dtype=torch.bfloat16, out=None, stream=None):
    """BitLinear forward that allocates no device memory inside the library
    (for callers without an allocator): the scratch comes from a fixed 4 MiB
    array in the library; larger problems raise BL_ERR_WORKSPACE. Only the
    output (when ``out`` is None) is allocated here, by torch."""
    _cuda(A, "A")
    _cuda(W_packed, "W_packed")
    _cuda(gamma, "gamma")
    M, K = A.shape
    N = W_packed.shape[0]
    _shape(W_packed, (N, K // 4), "W_packed")
    _atleast(gamma, 1, "gamma")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=A.device)
    _cuda(out, "out")
    _shape(out, (M, N), "out")
    check(load().bl_linear_noalloc(A.data_ptr(), _dt(A, "A"), M, K, W_packed.data_ptr(),
                                   gamma.data_ptr(), N, float(eps), int(bool(relu2)),
                                   out.data_ptr(), _dt(out, "out"), _stream(stream)),
          "bl_linear_noalloc")
    return out


def bl_ffn_relu2(X, W_up, gamma_up, W_down, gamma_down, eps: float = 1e-5, *,
                 out_dtype=torch.bfloat16, out=None, workspace=None, pdl=False, stream=None):
    """Ternary FFN block: BitLinear up (K→H), ReLU², per-token requant, BitLinear down (H→K)."""
    for t, n in ((X, "X"), (W_up, "W_up"), (gamma_up, "gamma_up"), (W_down, "W_down"),
                 (gamma_down, "gamma_down")):
        _cuda(t, n)
    M, K = X.shape
    H = W_up.shape[0]
    _shape(W_up, (H, K // 4), "W_up")
    _shape(W_down, (K, H // 4), "W_down")
    _atleast(gamma_up, 1, "gamma_up")
    _atleast(gamma_down, 1, "gamma_down")
    if out is None:
        out = torch.empty((M, K), dtype=out_dtype, device=X.device)
    _cuda(out, "out")
    _shape(out, (M, K), "out")
    L = load()
    if workspace is None:
        workspace = _ws(int(L.bl_ffn_workspace_bytes(M, K, H)), X.device, stream)
    else:
        _cuda(workspace, "workspace")
    check(L.bl_ffn_relu2_ex(X.data_ptr(), _dt(X, "X"), M, K, H, W_up.data_ptr(), gamma_up.data_ptr(),
                            W_down.data_ptr(), gamma_down.data_ptr(), float(eps), out.data_ptr(),
                            _dt(out, "out"), _ptr(workspace), _nbytes(workspace),
                            BL_FLAG_PDL if pdl else 0, _stream(stream)), "bl_ffn_relu2")
    return out


def _taps(M, K, H, device, ffn: bool, cta: int):
    """Allocate tap buffers (torch) and the matching bl_taps structure."""
    t = {"act_q": torch.empty((M, K), dtype=torch.int8, device=device),
         "act_gamma": torch.empty((M,), dtype=torch.float32, device=device),
         "act_rowsum": torch.empty((M,), dtype=torch.int32, device=device)}
    if ffn:
        t.update({"acc_up": torch.empty((M, H), dtype=torch.int32, device=device),
                  "req_q": torch.empty((M, H), dtype=torch.int8, device=device),
                  "req_gamma": torch.empty((M,), dtype=torch.float32, device=device),
                  "req_rowsum": torch.empty((M,), dtype=torch.int32, device=device)})
    s = BlTaps(**{k: v.data_ptr() for k, v in t.items()}, cta=int(cta), reserved=0)
    return t, s


def bl_linear_taps(A, W_packed, gamma, eps: float = 1e-5, *, relu2=False,
                   out_dtype=torch.bfloat16, pdl=False, cta: int = 0, stream=None):
    """bl_linear that also returns the int8 tokens, γ_A and Σ A_q the
    contraction used (for the fused GEMV path: those of CTA ``cta``; -1 =
    the last CTA). Returns (Y, taps dict)."""
    _cuda(A, "A")
    _cuda(W_packed, "W_packed")
    _cuda(gamma, "gamma")
    M, K = A.shape
    N = W_packed.shape[0]
    _shape(W_packed, (N, K // 4), "W_packed")
    _atleast(gamma, 1, "gamma")
    out = torch.empty((M, N), dtype=out_dtype, device=A.device)
    L = load()
    ws = _ws(int(L.bl_linear_workspace_bytes(M, K, N)), A.device, stream)
    taps, s = _taps(M, K, 0, A.device, False, cta)
    check(L.bl_linear_taps(A.data_ptr(), _dt(A, "A"), M, K, W_packed.data_ptr(), gamma.data_ptr(),
                           N, float(eps), int(bool(relu2)), out.data_ptr(), _dt(out, "out"),
                           _ptr(ws), _nbytes(ws), BL_FLAG_PDL if pdl else 0, s,
                           _stream(stream)), "bl_linear_taps")
    return out, taps


def bl_ffn_relu2_taps(X, W_up, gamma_up, W_down, gamma_down, eps: float = 1e-5, *,
                      out_dtype=torch.bfloat16, cta: int = 0, stream=None):
    """bl_ffn_relu2 that also returns X_q, γ_X, Σ X_q, the up-projection
    accumulators, the requantised ReLU² tokens R_q, γ_r and Σ R_q.
    Returns (Y, taps dict)."""
    for t, n in ((X, "X"), (W_up, "W_up"), (gamma_up, "gamma_up"), (W_down, "W_down"),
                 (gamma_down, "gamma_down")):
        _cuda(t, n)
    M, K = X.shape
    H = W_up.shape[0]
    _shape(W_up, (H, K // 4), "W_up")
    _shape(W_down, (K, H // 4), "W_down")
    out = torch.empty((M, K), dtype=out_dtype, device=X.device)
    L = load()
    ws = _ws(int(L.bl_ffn_workspace_bytes(M, K, H)), X.device, stream)
    taps, s = _taps(M, K, H, X.device, True, cta)
    check(L.bl_ffn_relu2_taps(X.data_ptr(), _dt(X, "X"), M, K, H, W_up.data_ptr(),
                              gamma_up.data_ptr(), W_down.data_ptr(), gamma_down.data_ptr(),
                              float(eps), out.data_ptr(), _dt(out, "out"), _ptr(ws), _nbytes(ws),
                              s, _stream(stream)), "bl_ffn_relu2_taps")
    return out, taps


def bl_ffn_tp_up(X, W_up_r, gamma_up, eps: float = 1e-5, *, stream=None):
    """Tensor-parallel FFN, step 1 on this rank's shard of H: returns
    (acc_up int32 [M, H_r], γ_X fp32 [M], rmax fp32 [M] = shard max of r)."""
    _cuda(X, "X")
    _cuda(W_up_r, "W_up_r")
    _cuda(gamma_up, "gamma_up")
    M, K = X.shape
    H_r = W_up_r.shape[0]
    if W_up_r.shape[1] * 4 != K:
        raise ValueError("W_up_r must be [H_r, K/4]")
    acc = torch.empty((M, H_r), dtype=torch.int32, device=X.device)
    gX = torch.empty((M,), dtype=torch.float32, device=X.device)
    rmax = torch.empty((M,), dtype=torch.float32, device=X.device)
    L = load()
    ws = _ws(int(L.bl_ffn_tp_up_workspace_bytes(M, K)), X.device, stream)
    check(L.bl_ffn_tp_up(X.data_ptr(), _dt(X, "X"), M, K, H_r, W_up_r.data_ptr(),
                         gamma_up.data_ptr(), float(eps), acc.data_ptr(), gX.data_ptr(),
                         rmax.data_ptr(), _ptr(ws), _nbytes(ws), _stream(stream)), "bl_ffn_tp_up")
    return acc, gX, rmax


def bl_ffn_tp_down(acc_up, gamma_x, gamma_up, gamma_r, W_down_r, eps: float = 1e-5, *,
                   stream=None):
    """Tensor-parallel FFN, step 3: requantise this shard with the all-ranks
    γ_r and return its partial down-projection (int32 [M, K_out])."""
    for t, n in ((acc_up, "acc_up"), (gamma_x, "gamma_x"), (gamma_up, "gamma_up"),
                 (gamma_r, "gamma_r"), (W_down_r, "W_down_r")):
        _cuda(t, n)
    M, H_r = acc_up.shape
    K_out = W_down_r.shape[0]
    if W_down_r.shape[1] * 4 != H_r:
        raise ValueError("W_down_r must be [K_out, H_r/4]")
    out = torch.empty((M, K_out), dtype=torch.int32, device=acc_up.device)
    L = load()
    ws = _ws(int(L.bl_ffn_tp_down_workspace_bytes(M, H_r)), acc_up.device, stream)
    check(L.bl_ffn_tp_down(acc_up.data_ptr(), gamma_x.data_ptr(), gamma_up.data_ptr(),
                           gamma_r.data_ptr(), M, H_r, W_down_r.data_ptr(), K_out, float(eps),
                           out.data_ptr(), _ptr(ws), _nbytes(ws), _stream(stream)), "bl_ffn_tp_down")
    return out


def bl_dequant_i32(acc, gamma_A, gamma, *, relu2=False, out_dtype=torch.bfloat16, stream=None):
    """Y = acc · ((γ_A·γ)/127) (ReLU² optional) from INT32 accumulators."""
    for t, n in ((acc, "acc"), (gamma_A, "gamma_A"), (gamma, "gamma")):
        _cuda(t, n)
    M, N = acc.shape
    out = torch.empty((M, N), dtype=out_dtype, device=acc.device)
    check(load().bl_dequant_i32(acc.data_ptr(), gamma_A.data_ptr(), gamma.data_ptr(), M, N,
                                int(bool(relu2)), out.data_ptr(), _dt(out, "out"),
                                _stream(stream)), "bl_dequant_i32")
    return out


def bl_pack_radix3(W_packed, K: int, *, out=None, stream=None):
    """2-bit packed [N, K/4] → radix-3 storage [N, row_bytes] (5 weights/byte)."""
    _cuda(W_packed, "W_packed")
    N = W_packed.shape[0]
    _shape(W_packed, (N, K // 4), "W_packed")
    L = load()
    rb = int(L.bl_radix3_row_bytes(K))
    if out is None:
        out = torch.empty((N, rb), dtype=torch.uint8, device=W_packed.device)
    _cuda(out, "out")
    _shape(out, (N, rb), "out")
    check(L.bl_pack_radix3(W_packed.data_ptr(), N, K, out.data_ptr(), _stream(stream)),
          "bl_pack_radix3")
    return out


def bl_linear_radix3(A, W_r3, gamma, eps: float = 1e-5, *, relu2=False, out_dtype=torch.bfloat16,
                     raw=False, out=None, pdl=False, stream=None):
    """BitLinear for ≤ 4 tokens on radix-3 weights (raw=True: INT32 accumulators)."""
    _cuda(A, "A")
    _cuda(W_r3, "W_r3")
    _cuda(gamma, "gamma")
    M, K = A.shape
    N = W_r3.shape[0]
    _shape(W_r3, (N, int(load().bl_radix3_row_bytes(K))), "W_r3")
    _atleast(gamma, 1, "gamma")
    if out is None:
        out = torch.empty((M, N), dtype=torch.int32 if raw else out_dtype, device=A.device)
    _cuda(out, "out")
    _shape(out, (M, N), "out")
    if raw and out.dtype != torch.int32:
        raise TypeError("out must be int32 when raw=True")
    flags = (BL_FLAG_PDL if pdl else 0) | (BL_FLAG_RAW_I32 if raw else 0)
    ydt = BL_F32 if raw else _dt(out, "out")
    check(load().bl_linear_radix3(A.data_ptr(), _dt(A, "A"), M, K, W_r3.data_ptr(), gamma.data_ptr(),
                                  N, float(eps), int(bool(relu2)), out.data_ptr(), ydt, flags,
                                  _stream(stream)), "bl_linear_radix3")
    return out


def bl_pack_lut_index(W_packed, *, out=None, stream=None):
    """2-bit packed [N, K/4] → lookup-table index bytes [N, K/4]."""
    _cuda(W_packed, "W_packed")
    N, Kq = W_packed.shape
    if out is None:
        out = torch.empty((N, Kq), dtype=torch.uint8, device=W_packed.device)
    _cuda(out, "out")
    _shape(out, (N, Kq), "out")
    check(load().bl_pack_lut_index(W_packed.data_ptr(), N, 4 * Kq, out.data_ptr(), _stream(stream)),
          "bl_pack_lut_index")
    return out


def bl_linear_lut(A, W_idx, gamma, eps: float = 1e-5, *, out_dtype=torch.bfloat16, raw=False,
                  out=None, pdl=False, stream=None):
    """BitLinear for one token by table lookup (raw=True: INT32 accumulators)."""
    _cuda(A, "A")
    _cuda(W_idx, "W_idx")
    _cuda(gamma, "gamma")
    M, K = A.shape
    N = W_idx.shape[0]
    _shape(W_idx, (N, K // 4), "W_idx")
    _atleast(gamma, 1, "gamma")
    if out is None:
        out = torch.empty((M, N), dtype=torch.int32 if raw else out_dtype, device=A.device)
    _cuda(out, "out")
    _shape(out, (M, N), "out")
    if raw and out.dtype != torch.int32:
        raise TypeError("out must be int32 when raw=True")
    flags = (BL_FLAG_PDL if pdl else 0) | (BL_FLAG_RAW_I32 if raw else 0)
    check(load().bl_linear_lut(A.data_ptr(), _dt(A, "A"), M, K, W_idx.data_ptr(), gamma.data_ptr(),
                               N, float(eps), out.data_ptr(), BL_F32 if raw else _dt(out, "out"),
                               flags, _stream(stream)), "bl_linear_lut")
    return out


def bl_ste_grad_input(dY, W_packed, gamma, *, stream=None):
    """STE backward, activation gradient dA [M, K] = γ·(dY·W_q) (fp32)."""
    _cuda(dY, "dY")
    _cuda(W_packed, "W_packed")
    _cuda(gamma, "gamma")
    M, N = dY.shape
    if W_packed.shape[0] != N:
        raise ValueError("W_packed must be [N, K/4] with N = dY.shape[1]")
    K = W_packed.shape[1] * 4
    dA = torch.empty((M, K), dtype=torch.float32, device=dY.device)
    L = load()
    ws = _ws(int(L.bl_ste_grad_input_workspace_bytes(M, N, K)), dY.device, stream)
    check(L.bl_ste_grad_input(dY.data_ptr(), _dt(dY, "dY"), M, N, W_packed.data_ptr(),
                              gamma.data_ptr(), K, dA.data_ptr(), _ptr(ws), _nbytes(ws),
                              _stream(stream)), "bl_ste_grad_input")
    return dA


def bl_ste_grad_weight(dY, A_q, gamma_A, W, gamma, eps: float = 1e-5, *, stream=None):
    """STE backward, weight gradient dW [N, K] = mask ⊙ (dYᵀ·Â) (fp32); W are
    the latent weights [N, K] whose clip range makes the mask."""
    for t, n in ((dY, "dY"), (A_q, "A_q"), (gamma_A, "gamma_A"), (W, "W"), (gamma, "gamma")):
        _cuda(t, n)
    M, N = dY.shape
    K = A_q.shape[1]
    if A_q.shape[0] != M or tuple(W.shape) != (N, K):
        raise ValueError("A_q must be [M, K] and W [N, K]")
    dW = torch.empty((N, K), dtype=torch.float32, device=dY.device)
    L = load()
    ws = _ws(int(L.bl_ste_grad_weight_workspace_bytes(M, N, K)), dY.device, stream)
    check(L.bl_ste_grad_weight(dY.data_ptr(), _dt(dY, "dY"), M, N, A_q.data_ptr(),
                               gamma_A.data_ptr(), K, W.data_ptr(), _dt(W, "W"), gamma.data_ptr(),
                               float(eps), dW.data_ptr(), _ptr(ws), _nbytes(ws), _stream(stream)),
          "bl_ste_grad_weight")
    return dW


# ---------------------------------------------------------------------------
# Operators around the ternary product: 4-bit weights, layer norm, 8-bit
# activation checkpoints.


# The current stream's handle and the current device, without the objects that
# torch.cuda.current_stream() and current_device() go through (3 us a call), and
# torch's allocator without its argument parsing (0.8 us against 1.9). Builds of
# torch that lack these names import the package all the same.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
try:
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:  # pragma: no cover
    def _empty_strided_cuda(size, stride, dtype):
        return torch.empty_strided(size, stride, dtype=dtype, device="cuda")


def _new(dtype, *shape):
    """Contiguous uninitialised tensor on the current device and stream."""
    stride, n = [], 1
    for s in reversed(shape):
        stride.append(n)
        n *= s
    return _empty_strided_cuda(shape, tuple(reversed(stride)), dtype)


def _placed(fn):
    """Runs ``fn`` on the device of its first tensor and on ``stream`` (default:
    that device's current one). Outputs and workspace are allocated on that
    stream, and the tensors passed in are recorded on it, so that torch does not
    hand their memory to another one while the call runs."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = next((t for t in (*args, *kw.values()) if isinstance(t, torch.Tensor)), None)
        if first is None or not first.is_cuda:
            return fn(*args, **kw)      # refused there
        if stream is not None:
            if stream.device != first.device:
                raise ValueError(f"stream is on {stream.device}, the tensors on {first.device}")
            with torch.cuda.stream(stream):
                try:
                    return fn(*args, **kw)
                finally:
                    for t in (*args, *kw.values()):
                        if isinstance(t, torch.Tensor) and t.is_cuda:
                            t.record_stream(stream)
        if first.get_device() != torch._C._cuda_getDevice():
            with torch.cuda.device(first.device):
                return fn(*args, **kw)
        return fn(*args, **kw)
    return call


_OPTIONAL = frozenset(("bias", "zeros", "out", "workspace"))


def _on(**tensors) -> int:
    """Checks that the tensors are contiguous and on one CUDA device; returns
    the handle of that device's current stream."""
    dev = -1
    for name, t in tensors.items():
        if t is None and name in _OPTIONAL:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        d = t.get_device()
        if dev < 0:
            dev = d
        elif d != dev:
            raise ValueError(f"{name} is on cuda:{d}, expected cuda:{dev}")
    return _raw_stream(dev)


def _of(t, dtype, shape, what: str) -> None:
    """Type and shape of an argument that may be None."""
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _w4_shapes(N: int, K: int, group: int):
    rb, kb = -(-N // 16), -(-K // 128)
    return (rb, kb, 1024), (rb, kb, 8, 128 // group, 2)


def _w4_group(scales: torch.Tensor) -> int:
    if scales.dim() != 5 or scales.shape[3] not in (1, 2, 4):
        raise ValueError("scales must have shape [ceil(N/16), ceil(K/128), 8, 128/group, 2]")
    return 128 // scales.shape[3]


def _check_w4(W4, scales, zeros, N: int, K: int) -> int:
    group = _w4_group(scales)
    w_shape, s_shape = _w4_shapes(N, K, group)
    _of(W4, torch.uint8, w_shape, "W4")
    _of(scales, torch.bfloat16, s_shape, "scales")
    _of(zeros, torch.uint8, s_shape, "zeros")
    return group


def _matrix(t: torch.Tensor, what: str):
    if t.dim() != 2:
        raise ValueError(f"{what} must be a matrix, got shape {tuple(t.shape)}")
    return t.shape


@_placed
def bl_quant_weights_w4(W, group: int = 128, *, zeros: bool = False):
    """4-bit weights with group scales from W [N, K] fp32/bf16: (W4 uint8
    [ceil(N/16), ceil(K/128), 1024], scales bf16 [.., .., 8, 128/group, 2], zero
    points uint8 of that shape, or None when ``zeros`` is false: symmetric)."""
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    st = _on(W=W)
    N, K = _matrix(W, "W")
    w_shape, s_shape = _w4_shapes(N, K, group)
    W4 = _new(torch.uint8, *w_shape)
    scales = _new(torch.bfloat16, *s_shape)
    zp = _new(torch.uint8, *s_shape) if zeros else None
    check(load().bl_quant_weights_w4(W.data_ptr(), _dt(W, "W"), N, K, group, W4.data_ptr(),
                                     scales.data_ptr(), _ptr(zp), st), "bl_quant_weights_w4")
    return W4, scales, zp


@_placed
def bl_pack_w4(codes, scales, group: int = 128, *, zeros=None):
    """4-bit weights found elsewhere: codes uint8 [N, K/2] (the lower column in
    the low half of a byte), scales bf16 [N, ceil(K/group)], zero points uint8
    of that shape or None → (W4, scales, zero points) as bl_quant_weights_w4."""
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    st = _on(codes=codes, scales=scales, zeros=zeros)
    N, K = _matrix(codes, "codes")
    K *= 2
    _of(codes, torch.uint8, (N, K // 2), "codes")
    _of(scales, torch.bfloat16, (N, -(-K // group)), "scales")
    _of(zeros, torch.uint8, (N, -(-K // group)), "zeros")
    w_shape, s_shape = _w4_shapes(N, K, group)
    W4 = _new(torch.uint8, *w_shape)
    out = _new(torch.bfloat16, *s_shape)
    zp = None if zeros is None else _new(torch.uint8, *s_shape)
    check(load().bl_pack_w4(codes.data_ptr(), scales.data_ptr(), _ptr(zeros), N, K, group,
                            W4.data_ptr(), out.data_ptr(), _ptr(zp), st), "bl_pack_w4")
    return W4, out, zp


@_placed
def bl_unpack_w4(W4, scales, N: int, K: int, *, zeros=None, out_dtype=torch.float32):
    """The matrix [N, K] that packed 4-bit weights stand for."""
    st = _on(W4=W4, scales=scales, zeros=zeros)
    group = _check_w4(W4, scales, zeros, N, K)
    out = _new(out_dtype, N, K)
    check(load().bl_unpack_w4(W4.data_ptr(), scales.data_ptr(), _ptr(zeros), N, K, group,
                              out.data_ptr(), _dt(out, "out"), st), "bl_unpack_w4")
    return out


@_placed
def bl_linear_w4(X, W4, scales, N: int, *, zeros=None, out_dtype=torch.bfloat16, out=None,
                 workspace=None, pdl=False):
    """Y [M, N] = X·Wᵀ for few tokens on 4-bit weights with group scales."""
    st = _on(X=X, W4=W4, scales=scales, zeros=zeros, out=out, workspace=workspace)
    M, K = _matrix(X, "X")
    group = _check_w4(W4, scales, zeros, N, K)
    if out is None:
        out = _new(out_dtype, M, N)
    _shape(out, (M, N), "out")
    L = load()
    if workspace is None and M > 5 and X.dtype == torch.float32:
        workspace = _new(torch.uint8, int(L.bl_linear_w4_workspace_bytes(M, K, group)))
    check(L.bl_linear_w4(X.data_ptr(), _dt(X, "X"), M, K, W4.data_ptr(), scales.data_ptr(),
                         _ptr(zeros), N, group, out.data_ptr(), _dt(out, "out"), _ptr(workspace),
                         _nbytes(workspace), BL_FLAG_PDL if pdl else 0, st), "bl_linear_w4")
    return out


@_placed
def bl_layernorm(X, weight, bias=None, eps: float = 1e-5, *, out_dtype=torch.bfloat16):
    """Layer norm of the rows of X [M, K]: (Y [M, K], mean fp32 [M], rstd fp32 [M])."""
    st = _on(X=X, weight=weight, bias=bias)
    M, K = _matrix(X, "X")
    _of(weight, torch.float32, (K,), "weight")
    _of(bias, torch.float32, (K,), "bias")
    Y = _new(out_dtype, M, K)
    mean = _new(torch.float32, M)
    rstd = _new(torch.float32, M)
    check(load().bl_layernorm(X.data_ptr(), _dt(X, "X"), M, K, weight.data_ptr(), _ptr(bias),
                              float(eps), Y.data_ptr(), _dt(Y, "out"), mean.data_ptr(),
                              rstd.data_ptr(), st), "bl_layernorm")
    return Y, mean, rstd


@_placed
def bl_layernorm_quant(X, weight, bias=None, eps: float = 1e-5, q_eps: float = 1e-5, *,
                       checkpoint: bool = False):
    """Layer norm straight to the int8 tokens that bl_quant_acts would make of
    it: (A_q int8 [M, K], γ_A fp32 [M], Σ A_q int32 [M], rstd fp32 [M], and the
    8-bit checkpoint of the normalised rows for bl_layernorm_grad_q8: int8
    [M, K] and fp32 [M, K/64], or None twice without ``checkpoint``)."""
    st = _on(X=X, weight=weight, bias=bias)
    M, K = _matrix(X, "X")
    _of(weight, torch.float32, (K,), "weight")
    _of(bias, torch.float32, (K,), "bias")
    A_q = _new(torch.int8, M, K)
    gamma = _new(torch.float32, M)
    rowsum = _new(torch.int32, M)
    rstd = _new(torch.float32, M)
    xq = _new(torch.int8, M, K) if checkpoint else None
    xs = _new(torch.float32, M, K // 64) if checkpoint else None
    check(load().bl_layernorm_quant(X.data_ptr(), _dt(X, "X"), M, K, weight.data_ptr(), _ptr(bias),
                                    float(eps), float(q_eps), A_q.data_ptr(), gamma.data_ptr(),
                                    rowsum.data_ptr(), rstd.data_ptr(), _ptr(xq), _ptr(xs), st),
          "bl_layernorm_quant")
    return A_q, gamma, rowsum, rstd, xq, xs


def _norm_grad_out(L, M, K, out_dtype):
    dX = _new(out_dtype, M, K)
    dw = _new(torch.float32, K)
    db = _new(torch.float32, K)
    return dX, dw, db, _new(torch.uint8, int(L.bl_layernorm_grad_workspace_bytes(M, K)))


@_placed
def bl_layernorm_grad(dY, X, mean, rstd, weight, *, out_dtype=torch.bfloat16):
    """Layer norm's backward from the kept input: (dX [M, K], dweight fp32 [K], dbias fp32 [K])."""
    st = _on(dY=dY, X=X, mean=mean, rstd=rstd, weight=weight)
    M, K = _matrix(dY, "dY")
    _shape(X, (M, K), "X")
    _of(mean, torch.float32, (M,), "mean")
    _of(rstd, torch.float32, (M,), "rstd")
    _of(weight, torch.float32, (K,), "weight")
    L = load()
    dX, dw, db, ws = _norm_grad_out(L, M, K, out_dtype)
    check(L.bl_layernorm_grad(dY.data_ptr(), _dt(dY, "dY"), X.data_ptr(), _dt(X, "X"),
                              mean.data_ptr(), rstd.data_ptr(), weight.data_ptr(), M, K,
                              dX.data_ptr(), _dt(dX, "out"), dw.data_ptr(), db.data_ptr(),
                              _ptr(ws), _nbytes(ws), st), "bl_layernorm_grad")
    return dX, dw, db


@_placed
def bl_layernorm_grad_q8(dY, xhat_q, xhat_scale, rstd, weight, *, out_dtype=torch.bfloat16):
    """Layer norm's backward from the 8-bit checkpoint of the normalised rows:
    (dX [M, K], dweight fp32 [K], dbias fp32 [K])."""
    st = _on(dY=dY, xhat_q=xhat_q, xhat_scale=xhat_scale, rstd=rstd, weight=weight)
    M, K = _matrix(dY, "dY")
    _of(xhat_q, torch.int8, (M, K), "xhat_q")
    _of(xhat_scale, torch.float32, (M, K // 64), "xhat_scale")
    _of(rstd, torch.float32, (M,), "rstd")
    _of(weight, torch.float32, (K,), "weight")
    L = load()
    dX, dw, db, ws = _norm_grad_out(L, M, K, out_dtype)
    check(L.bl_layernorm_grad_q8(dY.data_ptr(), _dt(dY, "dY"), xhat_q.data_ptr(),
                                 xhat_scale.data_ptr(), rstd.data_ptr(), weight.data_ptr(), M, K,
                                 dX.data_ptr(), _dt(dX, "out"), dw.data_ptr(), db.data_ptr(),
                                 _ptr(ws), _nbytes(ws), st), "bl_layernorm_grad_q8")
    return dX, dw, db


@_placed
def bl_relu2_requant_q8(acc_up, gamma_x, gamma_up, eps: float = 1e-5, *, checkpoint: bool = True):
    """ReLU² of the FFN, from the up-projection's INT32 accumulators: (R_q int8
    [M, H], γ_r fp32 [M], Σ R_q int32 [M], and the 8-bit checkpoint of
    max(h, 0): uint8 [M, H], fp32 [M, H/64], or None twice without
    ``checkpoint``)."""
    st = _on(acc_up=acc_up, gamma_x=gamma_x, gamma_up=gamma_up)
    M, H = _matrix(acc_up, "acc_up")
    _of(acc_up, torch.int32, (M, H), "acc_up")
    _of(gamma_x, torch.float32, (M,), "gamma_x")
    _of(gamma_up, torch.float32, (1,), "gamma_up")
    R_q = _new(torch.int8, M, H)
    gamma_r = _new(torch.float32, M)
    rowsum = _new(torch.int32, M)
    P_q = _new(torch.uint8, M, H) if checkpoint else None
    p_scale = _new(torch.float32, M, H // 64) if checkpoint else None
    check(load().bl_relu2_requant_q8(acc_up.data_ptr(), gamma_x.data_ptr(), gamma_up.data_ptr(),
                                     M, H, float(eps), R_q.data_ptr(), gamma_r.data_ptr(),
                                     rowsum.data_ptr(), _ptr(P_q), _ptr(p_scale), st),
          "bl_relu2_requant_q8")
    return R_q, gamma_r, rowsum, P_q, p_scale


@_placed
def bl_relu2_grad_q8(dR, P_q, p_scale, *, out_dtype=torch.bfloat16):
    """dH [M, H] = 2·p̂·dR from the 8-bit checkpoint of max(h, 0)."""
    st = _on(dR=dR, P_q=P_q, p_scale=p_scale)
    M, H = _matrix(dR, "dR")
    _of(P_q, torch.uint8, (M, H), "P_q")
    _of(p_scale, torch.float32, (M, H // 64), "p_scale")
    dH = _new(out_dtype, M, H)
    check(load().bl_relu2_grad_q8(dR.data_ptr(), _dt(dR, "dR"), P_q.data_ptr(), p_scale.data_ptr(),
                                  M, H, dH.data_ptr(), _dt(dH, "out"), st), "bl_relu2_grad_q8")
    return dH


def bl_probe_pdl_floor(M: int, K: int, N: int, *, stream=None) -> None:
    """One empty kernel with the decode GEMV's launch shape for (M, K, N)."""
    check(load().bl_probe_pdl_floor(M, K, N, _stream(stream)), "bl_probe_pdl_floor")


def bl_check_device_error(stream=None) -> int:
    """Synchronise the stream; return the library status (0 = BL_OK)."""
    return int(load().bl_check_device_error(_stream(stream)))


def bl_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    check(load().bl_selftest_wait_timeout(int(limit_ns), _stream(stream)),
          "bl_selftest_wait_timeout")
