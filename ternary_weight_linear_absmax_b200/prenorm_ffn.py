"""Pre-norm ternary FFN block for training and decoding: layer norm in front of
the block's int8 tokens, and a backward pass that keeps 8-bit checkpoints only.

    y = x + FFN(LN(x)),  FFN: BitLinear up (K → H), ReLU², BitLinear down (H → K)

Forward (``forward``): bl_layernorm_quant writes the int8 tokens of the
up-projection without the normalised row going through memory, the INT32
up-projection is requantised by bl_relu2_requant_q8, and bl_linear_q runs the
down-projection. Saved for the backward: the tokens (which bl_ste_grad_weight
takes as they are) and the 8-bit checkpoints of x̂ and of max(h, 0): 2·(K + H)
bytes per token, (K + H)/16 for the checkpoints' scales and a few fp32 per token,
half of what the same four rows take in bf16.

Backward (``backward``), with the straight-through gradients of the BitLinear
layers: dW_down = mask ⊙ dyᵀ·R̂, dr = dy·Ŵ_down, dh = 2·p̂·dr, dW_up = mask ⊙
dhᵀ·Â, da = dh·Ŵ_up, and layer norm's backward of da.

Decoding (``decode``): the same calls without the checkpoints.

Every arithmetic step runs in the CUDA library; this module sequences the calls
and adds the residual (in the output's type: the block's output and the sum are
rounded to it once each). A call runs on its input's device, on that
device's current stream.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (_on, bl_layernorm_grad_q8, bl_layernorm_quant, bl_linear_q, bl_relu2_grad_q8,
               bl_relu2_requant_q8, bl_ste_grad_input, bl_ste_grad_weight, bl_zero_gemm)


@dataclass
class PreNormFFNGrads:
    """Gradients of the block: of its input, of the latent weights (masked to
    the clip range) and of the norm's parameters."""
    dX: torch.Tensor
    dW_up: torch.Tensor
    dW_down: torch.Tensor
    dweight: torch.Tensor
    dbias: torch.Tensor


@dataclass
class PreNormFFN:
    """The block's parameters: the norm's weight and bias (fp32 [K]), and the
    packed matrices and their γ as bl_quant_weights returns them."""
    weight: torch.Tensor
    bias: torch.Tensor | None
    W_up: torch.Tensor
    gamma_up: torch.Tensor
    W_down: torch.Tensor
    gamma_down: torch.Tensor
    eps: float = 1e-5

    def _block(self, X, checkpoint: bool):
        with torch.cuda.device_of(X):
            _on(X=X, W_up=self.W_up, W_down=self.W_down, gamma_down=self.gamma_down)
            return self._run(X, checkpoint)

    def _run(self, X, checkpoint: bool):
        A_q, gamma_a, _, rstd, xq, xs = bl_layernorm_quant(X, self.weight, self.bias, self.eps, self.eps,
                                                           checkpoint=checkpoint)
        acc = bl_zero_gemm(A_q, self.W_up)
        R_q, gamma_r, sums, p_q, p_s = bl_relu2_requant_q8(acc, gamma_a, self.gamma_up, self.eps,
                                                         checkpoint=checkpoint)
        Y = bl_linear_q(R_q, gamma_r, self.W_down, self.gamma_down, rowsum=sums, out_dtype=X.dtype)
        return Y.add_(X), (A_q, gamma_a, rstd, xq, xs, R_q, gamma_r, p_q, p_s)

    def decode(self, X):
        """y for a batch of tokens [M, K]; nothing is kept."""
        return self._block(X, False)[0]

    def forward(self, X):
        """(y, what ``backward`` needs)."""
        return self._block(X, True)

    def backward(self, dY, saved, latent_up, latent_down) -> PreNormFFNGrads:
        """Gradients from dY [M, K] (bf16 or fp32) and the latent weights whose
        clip range masks their gradients."""
        A_q, gamma_a, rstd, xq, xs, R_q, gamma_r, p_q, p_s = saved
        with torch.cuda.device_of(dY):
            _on(dY=dY, A_q=A_q, gamma_a=gamma_a, xhat_q=xq, R_q=R_q, gamma_r=gamma_r, P_q=p_q, W_up=self.W_up,
                gamma_up=self.gamma_up, W_down=self.W_down, gamma_down=self.gamma_down,
                latent_up=latent_up, latent_down=latent_down)
            dW_down = bl_ste_grad_weight(dY, R_q, gamma_r, latent_down, self.gamma_down, self.eps)
            dR = bl_ste_grad_input(dY, self.W_down, self.gamma_down)
            dH = bl_relu2_grad_q8(dR, p_q, p_s)
            dW_up = bl_ste_grad_weight(dH, A_q, gamma_a, latent_up, self.gamma_up, self.eps)
            dA = bl_ste_grad_input(dH, self.W_up, self.gamma_up)
            dX, dweight, dbias = bl_layernorm_grad_q8(dA, xq, xs, rstd, self.weight, out_dtype=dY.dtype)
            return PreNormFFNGrads(dX.add_(dY), dW_up, dW_down, dweight, dbias)
