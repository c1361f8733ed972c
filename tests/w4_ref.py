"""64-bit restatement of the 4-bit weight format and of layer norm, used by the
tests of bl_*_w4 and bl_layernorm* (numpy, written from the formulas)."""
from __future__ import annotations

import numpy as np
import torch

KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}


def bf16(x):
    """Round fp32 values to bf16 (nearest, ties to even), as fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().float().numpy()


def quant_w4(W, group, zeros):
    """Codes, scales and zero points (fp32 arrays) of W [N, K] (fp32 values).
    Quotients are taken in 64 bits: their distance from a border is either 0 or
    far above 2^-53, so they round as the exact ones."""
    N, K = W.shape
    G = -(-K // group)
    codes = np.empty((N, K), np.int64)
    scales = np.empty((N, G), np.float32)
    zps = np.full((N, G), 8, np.int64)
    for g in range(G):
        w = W[:, g * group:(g + 1) * group]
        hi, lo = np.maximum(w.max(1), 0).astype(np.float32), np.minimum(w.min(1), 0).astype(np.float32)
        raw = ((hi - lo).astype(np.float32) / np.float32(15) if zeros
               else np.maximum(hi, -lo) / np.float32(7))
        s = bf16(raw).astype(np.float64)
        by = np.where(s > 0, s, np.inf)
        if zeros:
            zps[:, g] = np.clip(np.rint(-lo.astype(np.float64) / by), 0, 15)
        q = np.rint(w.astype(np.float64) / by[:, None]) + zps[:, g][:, None]
        codes[:, g * group:(g + 1) * group] = np.clip(q, 0, 15)
        scales[:, g] = s
    return codes, scales, zps


def dequant(codes, scales, zps, group):
    K = codes.shape[1]
    s = np.repeat(scales.astype(np.float64), group, axis=1)[:, :K]
    z = np.repeat(zps, group, axis=1)[:, :K]
    return s * (codes - z)


def pack(codes, scales, zps, group, zeros):
    """The packed layout, one element at a time from its definition."""
    N, K = codes.shape
    RB, KB, V = -(-N // 16), -(-K // 128), 128 // group
    words = np.zeros((RB, KB, 2, 8, 4, 4), np.uint32)
    sc = np.zeros((RB, KB, 8, V, 2), np.float32)
    zp = np.zeros((RB, KB, 8, V, 2), np.uint8)
    for n in range(N):
        rb, h, g = n // 16, (n % 16) // 8, n % 8
        for k in range(K):
            kb, u, t, j = k // 128, (k % 128) // 32, (k % 32) // 8, k % 8
            words[rb, kb, h, g, t, u] |= np.uint32(int(codes[n, k]) << (4 * (j // 2) + 16 * (j % 2)))
            sc[rb, kb, g, (k % 128) // group, h] = scales[n, k // group]
            zp[rb, kb, g, (k % 128) // group, h] = zps[n, k // group]
    return words, sc, zp if zeros else None


def linear_bound(x, w, K, bf16_out, ref):
    """How far the product may be from the 64-bit one, for values of one scale
    (normal deviates). Activations are rounded to half of 2^-21.99 of the
    largest of 128 columns: with a largest value of up to 6.5 times the mean
    magnitude that is 13·2^-24 of the sum of magnitudes S. A group's products and
    their sum are exact, and become fp32 with a few operations (8 roundings);
    the groups' sums are added up in one chain per warp, K/32 at most (its
    roundings are relative to partial sums, well inside S), and 32 more across
    warps and digits. The bound below, 136 + K/256 + 36 units of 2^-24, covers
    these more than once over up to K = 40,000, and what a chain of K/32
    roundings of random sign adds for longer rows."""
    S = np.abs(x) @ np.abs(w).T
    tol = (8 * 17 + K / 1024 * 4 + 36) * 2.0 ** -24 * S + 1e-37
    return tol + (2.0 ** -8 * np.abs(ref) if bf16_out else 0.0)


def layernorm(x, w, b, eps):
    """(y, mean, rstd, x̂) in 64 bits."""
    x = x.astype(np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    xh = (x - mean[:, None]) * rstd[:, None]
    y = xh * w
    return (y + b if b is not None else y), mean, rstd, xh


def layernorm_grad(dy, xh, rstd, w):
    g = dy * w
    a, b = g.mean(1)[:, None], (g * xh).mean(1)[:, None]
    return rstd[:, None] * (g - a - xh * b), (dy * xh).sum(0), dy.sum(0)


def checkpoint(v, top):
    """8-bit checkpoint of fp32 rows: (codes, scales) in fp32 arithmetic."""
    M, K = v.shape
    b = v.astype(np.float32).reshape(M, K // 64, 64)
    m = np.abs(b).max(2)
    live = m >= np.float32(2.0 ** -100)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.where(live, np.float32(top) / m, np.float32(0)).astype(np.float32)
        scale = np.where(live, m / np.float32(top), np.float32(0)).astype(np.float32)
    codes = np.rint((b * inv[:, :, None]).astype(np.float32)).astype(np.int64)
    return codes.reshape(M, K), scale
