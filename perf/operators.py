"""The operators around the ternary product, as a benchmark: 4-bit weights with
group scales (quantiser, few-token product), layer norm to int8 tokens and its
backward, and ReLU² with an 8-bit activation checkpoint.

``run`` computes a case in plain torch operations, or, where ``own`` is true,
by the package's entry points.

Layout of the 4-bit weights, which both forms read: rows in blocks of 16, K in
blocks of 128; block (rb, kb) is 1024 bytes, 256 little-endian words indexed
[h, g, t, u]; word (h, g, t, u) holds the codes of row 16·rb + 8·h + g, columns
128·kb + 32·u + 8·t + (0..7), column 2·p + e of those at bit 4·p + 16·e. Scales
(bf16) and zero points (bytes) are [rb, kb, g, 128/group, h]. Rows past N and
columns past K have scale 0.

The int8 tokens that the layer norm and ReLU² return are the integers that the
INT32 contraction takes, so they are compared as whole numbers; 4-bit weights
are returned as the values they stand for, and the checkpoints only through the
gradients made from them.
"""
import math

import torch

own = False

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
EPS = 9.999999747378752e-06  # 1e-5 in fp32


def _dt(name):
    return BF16 if name == "bf16" else F32


# ---------------------------------------------------------------------------
# Cases


def listed():
    return [
        # A small projection in fp32 (the sizes of the single-layer check), where latency is all.
        {"name": "w4 4x512-256 fp32 g32", "op": "w4_linear", "M": 4, "N": 256, "K": 512, "group": 32,
         "zeros": False, "x": "fp32", "y": "fp32"},
        # One decoded token through the benchmark's decode matrix.
        {"name": "w4 1x2560-6912 g128", "op": "w4_linear", "M": 1, "N": 6912, "K": 2560, "group": 128,
         "zeros": False, "x": "bf16", "y": "bf16"},
        # A small decode batch, zero points (the benchmark's small-batch shape).
        {"name": "w4 16x4096-11008 g64 z", "op": "w4_linear", "M": 16, "N": 11008, "K": 4096, "group": 64,
         "zeros": True, "x": "bf16", "y": "bf16"},
        # Logits of three sequences: a language-model head kept in 4 bits.
        {"name": "w4 3x2048-128256 head", "op": "w4_linear", "M": 3, "N": 128256, "K": 2048, "group": 128,
         "zeros": False, "x": "bf16", "y": "fp32"},
        # Quantising a matrix at load time, symmetric and with zero points.
        {"name": "w4 quant 6912x2560 bf16", "op": "w4_quant", "N": 6912, "K": 2560, "group": 128,
         "zeros": False, "w": "bf16"},
        {"name": "w4 quant 4001x4160 fp32 z", "op": "w4_quant", "N": 4001, "K": 4160, "group": 32,
         "zeros": True, "w": "fp32"},
        # One decoded token: norm straight to the contraction's int8 tokens.
        {"name": "ln tokens 1x2560", "op": "ln_tokens", "M": 1, "K": 2560, "x": "bf16"},
        # A prompt of 2048 tokens, normed to bf16.
        {"name": "ln 2048x4096", "op": "ln", "M": 2048, "K": 4096, "x": "bf16", "y": "bf16"},
        # A training step's norm: tokens and an 8-bit checkpoint forward, the gradients from it.
        {"name": "ln step q8 2048x4096", "op": "ln_step_q8", "M": 2048, "K": 4096, "x": "bf16", "dy": "fp32"},
        # The backward from the kept input in fp32, odd numbers of rows and columns' blocks.
        {"name": "ln grad 8191x2560 fp32", "op": "ln_grad", "M": 8191, "K": 2560, "x": "fp32", "dy": "fp32"},
        # ReLU² of the FFN's hidden layer in training: requantised tokens forward, gradient from 8 bits.
        {"name": "relu2 step q8 2048x11008", "op": "relu2_step_q8", "M": 2048, "H": 11008, "dr": "fp32"},
        {"name": "relu2 step q8 37x2752", "op": "relu2_step_q8", "M": 37, "H": 2752, "dr": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["w4_linear", "w4_linear", "w4_quant", "ln_tokens", "ln", "ln_step_q8", "ln_grad", "relu2_step_q8"])
    types = ["bf16", "fp32"]
    if op == "w4_linear":
        M, K = _log(rng, 1, 64), 64 * _log(rng, 2, 256)
        N = min(_log(rng, 64, 128256), 128256 * 2048 // (K * max(1, M // 4)))
        return {"op": op, "M": M, "N": max(N, 16), "K": K, "group": rng.choice([32, 64, 128]),
                "zeros": rng.random() < 0.5, "x": rng.choice(types), "y": rng.choice(types)}
    if op == "w4_quant":
        K = 64 * _log(rng, 2, 256)
        return {"op": op, "N": min(_log(rng, 64, 11008), 20_000_000 // K), "K": K, "group": rng.choice([32, 64, 128]),
                "zeros": rng.random() < 0.5, "w": rng.choice(types)}
    K = 64 * _log(rng, 2, 256)
    if op == "relu2_step_q8":
        return {"op": op, "M": min(_log(rng, 1, 4096), 22_000_000 // K), "H": K, "dr": rng.choice(types)}
    M = min(_log(rng, 1, 8192), 16_000_000 // K)
    c = {"op": op, "M": M, "K": K, "x": rng.choice(types)}
    if op == "ln":
        c["y"] = rng.choice(types)
    if op in ("ln_step_q8", "ln_grad"):
        c["dy"] = rng.choice(types)
    return c


# ---------------------------------------------------------------------------
# Inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _acts(g, M, K, offset=0.0):
    """N(0, 1) activations with 1 % of the channels scaled by 20."""
    a = torch.randn(M, K, generator=g, device=DEV)
    hot = torch.rand(K, generator=g, device=DEV) < 0.01
    return (a + offset) * torch.where(hot, 20.0, 1.0)


def _w4_parts(case, seed):
    """Activations, codes [N, K], scales [N, K/group] (bf16) and zero points [N, K/group] of a w4_linear case."""
    g = _gen(seed)
    M, N, K, G = case["M"], case["N"], case["K"], case["group"]
    x = _acts(g, M, K).to(_dt(case["x"]))
    Gn = -(-K // G)
    codes = (torch.randn(N, K, generator=g, device=DEV) * 2.6 + 8.0).round_().clamp_(0, 15).to(torch.uint8)
    scales = (0.02 / 2.6 * (0.75 + 0.5 * torch.rand(N, Gn, generator=g, device=DEV))).to(BF16)
    zeros = torch.randint(5, 11, (N, Gn), generator=g, device=DEV, dtype=torch.uint8) if case["zeros"] else None
    return x, codes, scales, zeros


def _pack(codes, scales, zeros, G):
    """The packed layout from codes [N, K], scales and zero points [N, ceil(K/G)]."""
    N, K = codes.shape
    RB, KB, V = -(-N // 16), -(-K // 128), 128 // G
    c = torch.full((16 * RB, 128 * KB), 8, dtype=torch.uint8, device=DEV)
    c[:N, :K] = codes
    c = c.view(RB, 2, 8, KB, 4, 4, 4, 2).permute(0, 3, 1, 2, 5, 4, 7, 6)  # rb kb h g t u e p
    byte = c[..., 0::2] | (c[..., 1::2] << 4)                             # p pairs: bits 4p within a half-word
    w4 = byte.reshape(RB, KB, 1024).contiguous()

    def groups(v, fill):
        full = torch.full((16 * RB, KB * V), fill, dtype=v.dtype, device=DEV)
        full[:N, :v.shape[1]] = v
        return full.view(RB, 2, 8, KB, V).permute(0, 3, 2, 4, 1).contiguous()

    return w4, groups(scales, 0), None if zeros is None else groups(zeros, 8)


def prepare(case, seed):
    op, g = case["op"], _gen(seed)
    s = dict(case)
    if op == "w4_linear":
        x, codes, scales, zeros = _w4_parts(case, seed)
        w4, sc, zp = _pack(codes, scales, zeros, case["group"])
        s.update(X=x, W4=w4, scales=sc, zp=zp, out_dtype=_dt(case["y"]))
    elif op == "w4_quant":
        s["W"] = (torch.randn(case["N"], case["K"], generator=g, device=DEV) * 0.02).to(_dt(case["w"]))
    elif op == "relu2_step_q8":
        M, H = case["M"], case["H"]
        s["acc"] = (torch.randn(M, H, generator=g, device=DEV) * 1600.0).round().to(torch.int32)
        s["gamma_x"] = 3.0 + 2.0 * torch.rand(M, generator=g, device=DEV)
        s["gamma_up"] = 0.015 + 0.002 * torch.rand(1, generator=g, device=DEV)
        s["dR"] = torch.randn(M, H, generator=g, device=DEV).to(_dt(case["dr"]))
    else:
        M, K = case["M"], case["K"]
        s["X"] = _acts(g, M, K, offset=0.3).to(_dt(case["x"]))
        s["weight"] = 1.0 + 0.1 * torch.randn(K, generator=g, device=DEV)
        s["bias"] = 0.1 * torch.randn(K, generator=g, device=DEV)
        if "dy" in case:
            s["dY"] = torch.randn(M, K, generator=g, device=DEV).to(_dt(case["dy"]))
        if op == "ln_grad":  # what the forward kept
            xd = s["X"].double()
            s["mean"] = xd.mean(1).float()
            s["rstd"] = (xd.var(1, unbiased=False) + EPS).rsqrt().float()
    return s


# ---------------------------------------------------------------------------
# Plain forms


def _plain_unpack(w4, scales, zp, N, K, G):
    """The matrix [N, K] in fp32 that packed 4-bit weights stand for."""
    RB, KB, V = w4.shape[0], w4.shape[1], 128 // G
    b = w4.view(RB, KB, 2, 8, 4, 4, 2, 2, 1)  # rb kb h g t u e (byte of p pairs)
    c = torch.cat((b & 15, b >> 4), dim=8)    # ... p = 2·(byte) + (nibble)
    q = c.permute(0, 2, 3, 1, 5, 4, 7, 8, 6).reshape(16 * RB, KB * V, G)  # rb h g kb u t p p e
    sc = scales.permute(0, 4, 2, 1, 3).reshape(16 * RB, KB * V, 1).float()
    z = 8.0 if zp is None else zp.permute(0, 4, 2, 1, 3).reshape(16 * RB, KB * V, 1).float()
    return ((q.float() - z) * sc).view(16 * RB, 128 * KB)[:N, :K]


def _plain_w4_quant(W, G, with_zeros):
    """Quantised values of W [N, K]: groups of G along K (the last may be short)."""
    N, K = W.shape
    w = torch.zeros(N, -(-K // G) * G, device=DEV)
    w[:, :K] = W
    w = w.view(N, -1, G)
    # A quotient next to a border is divided in 64 bits, which rounds as the exact one does.
    if with_zeros:
        lo, hi = w.amin(2, keepdim=True).clamp(max=0), w.amax(2, keepdim=True).clamp(min=0)
        s = ((hi - lo) / torch.full_like(lo, 15.0)).to(BF16).double()
        by = torch.where(s > 0, s, torch.full_like(s, math.inf))
        z = torch.round(-lo.double() / by).clamp(0, 15)
    else:
        s = (w.abs().amax(2, keepdim=True) / torch.full((1,), 7.0, device=DEV)).to(BF16).double()
        by = torch.where(s > 0, s, torch.full_like(s, math.inf))
        z = 8.0
    q = (torch.round(w.double() / by) + z).clamp(0, 15)
    return ((q - z) * s).float().view(N, -1)[:, :K].contiguous()


def _plain_norm(X):
    """Mean and reciprocal deviation of every row (sums in 64 bits, each rounded once), and the normalised rows."""
    x = X.float()
    mean = x.double().mean(1, keepdim=True).float()
    d = x - mean
    rstd = (1.0 / torch.sqrt(d.double().square().mean(1, keepdim=True) + EPS)).float()
    return mean, rstd, d * rstd


def _plain_absmax(v):
    """AbsMax int8 tokens of fp32 rows: (tokens, scale, sums)."""
    gamma = v.abs().amax(1)
    s = torch.full_like(gamma, 127.0) / (gamma + EPS)
    q = torch.round(v * s[:, None]).clamp(-128, 127).to(torch.int8)
    return q, gamma, q.sum(1, dtype=torch.int32)


def _plain_q8(v, top):
    """v as an 8-bit checkpoint stands for it: groups of 64 columns, codes to `top`."""
    b = v.view(v.shape[0], -1, 64)
    m = b.abs().amax(2, keepdim=True)
    live = m >= 2.0 ** -100
    t = torch.full_like(m, top)
    inv = torch.where(live, t / m, torch.zeros_like(m))
    scale = torch.where(live, m / t, torch.zeros_like(m))
    return (torch.round(b * inv) * scale).view_as(v)


def _plain_ln_grad(dY, xhat, rstd, weight):
    dy = dY.float()
    gy = dy * weight
    dx = rstd * (gy - gy.mean(1, keepdim=True) - xhat * (gy * xhat).mean(1, keepdim=True))
    return dx, (dy.double() * xhat).sum(0).float(), dy.double().sum(0).float()


def _plain(s):
    op = s["op"]
    if op == "w4_linear":
        w = _plain_unpack(s["W4"], s["scales"], s["zp"], s["N"], s["K"], s["group"])
        return (s["X"].float() @ w.t()).to(s["out_dtype"])
    if op == "w4_quant":
        return _plain_w4_quant(s["W"].float(), s["group"], s["zeros"])
    if op == "relu2_step_q8":
        scale = (s["gamma_x"] * s["gamma_up"]) / torch.full_like(s["gamma_x"], 127.0)
        p = (s["acc"].float() * scale[:, None]).clamp(min=0)
        tokens, gamma_r, sums = _plain_absmax(p * p)
        dH = 2.0 * _plain_q8(p, 255.0) * s["dR"].float()
        return {"tokens": tokens, "gamma": gamma_r, "sums": sums, "dH": dH.to(BF16)}
    if op == "ln_grad":
        xhat = (s["X"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dx, dw, db = _plain_ln_grad(s["dY"], xhat, s["rstd"][:, None], s["weight"])
        return {"dX": dx.to(s["X"].dtype), "dweight": dw, "dbias": db}
    mean, rstd, xhat = _plain_norm(s["X"])
    y = xhat * s["weight"] + s["bias"]
    if op == "ln":
        return {"Y": y.to(_dt(s["y"])), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    tokens, gamma, sums = _plain_absmax(y)
    out = {"tokens": tokens, "gamma": gamma, "sums": sums, "rstd": rstd[:, 0]}
    if op == "ln_step_q8":
        dx, dw, db = _plain_ln_grad(s["dY"], _plain_q8(xhat, 127.0), rstd, s["weight"])
        out.update(dX=dx.to(s["X"].dtype), dweight=dw, dbias=db)
    return out


# ---------------------------------------------------------------------------
# The package's calls


def _own(s):
    import ternary_weight_linear_absmax_b200 as bl

    op = s["op"]
    if op == "w4_linear":
        return bl.bl_linear_w4(s["X"], s["W4"], s["scales"], s["N"], zeros=s["zp"], out_dtype=s["out_dtype"])
    if op == "w4_quant":
        w4, scales, zp = bl.bl_quant_weights_w4(s["W"], s["group"], zeros=s["zeros"])
        return bl.bl_unpack_w4(w4, scales, s["N"], s["K"], zeros=zp)
    if op == "relu2_step_q8":
        tokens, gamma_r, sums, p_q, p_scale = bl.bl_relu2_requant_q8(s["acc"], s["gamma_x"], s["gamma_up"], EPS)
        dH = bl.bl_relu2_grad_q8(s["dR"], p_q, p_scale)
        return {"tokens": tokens, "gamma": gamma_r, "sums": sums, "dH": dH}
    if op == "ln_grad":
        dx, dw, db = bl.bl_layernorm_grad(s["dY"], s["X"], s["mean"], s["rstd"], s["weight"], out_dtype=s["X"].dtype)
        return {"dX": dx, "dweight": dw, "dbias": db}
    if op == "ln":
        y, mean, rstd = bl.bl_layernorm(s["X"], s["weight"], s["bias"], EPS, out_dtype=_dt(s["y"]))
        return {"Y": y, "mean": mean, "rstd": rstd}
    step = op == "ln_step_q8"
    tokens, gamma, sums, rstd, xq, xs = bl.bl_layernorm_quant(s["X"], s["weight"], s["bias"], EPS, checkpoint=step)
    out = {"tokens": tokens, "gamma": gamma, "sums": sums, "rstd": rstd}
    if step:
        dx, dw, db = bl.bl_layernorm_grad_q8(s["dY"], xq, xs, rstd, s["weight"], out_dtype=s["X"].dtype)
        out.update(dX=dx, dweight=dw, dbias=db)
    return out


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    size = lambda name: 2 if name == "bf16" else 4  # noqa: E731
    op = case["op"]
    if op == "w4_linear":
        M, N, K = case["M"], case["N"], case["K"]
        groups = N * -(-K // case["group"])
        return {"bytes": N * K // 2 + groups * (3 if case["zeros"] else 2) + M * K * size(case["x"]) + M * N * size(case["y"]),
                "flops": 2 * M * N * K}
    if op == "w4_quant":  # read, packed, read back as values
        N, K = case["N"], case["K"]
        packed = N * K // 2 + N * -(-K // case["group"]) * (3 if case["zeros"] else 2)
        return {"bytes": N * K * (size(case["w"]) + 4) + 2 * packed, "flops": 4 * N * K}
    if op == "relu2_step_q8":
        M, H = case["M"], case["H"]
        return {"bytes": M * H * (4 + 1 + 2 * (1 + 4 / 64) + size(case["dr"]) + 2) + 12 * M, "flops": 12 * M * H}
    M, K = case["M"], case["K"]
    x = size(case["x"])
    if op == "ln_grad":
        return {"bytes": M * K * (size(case["dy"]) + 2 * x) + 8 * M + 12 * K, "flops": 12 * M * K}
    if op == "ln":
        return {"bytes": M * K * (x + size(case["y"])) + 8 * M + 8 * K, "flops": 8 * M * K}
    if op == "ln_tokens":
        return {"bytes": M * K * (x + 1) + 12 * M + 8 * K, "flops": 10 * M * K}
    return {"bytes": M * K * (x + 1 + 2 * (1 + 4 / 64) + size(case["dy"]) + x) + 16 * M + 20 * K, "flops": 24 * M * K}


# ---------------------------------------------------------------------------
# The definitions in 64 bits. Integers that a rounding decides, and what a
# checkpoint's rounding leaves, are taken as the plain types decide them:
# those have no value in 64 bits of their own.


def _exact_checkpoint(v, top):
    """What the 8-bit checkpoint of fp32 values stands for, in 64 bits."""
    N, K = v.shape
    m = v.abs().view(N, K // 64, 64).max(dim=2).values
    m = torch.where(m < 2.0 ** -100, torch.full_like(m, math.inf), m)
    per = m.repeat_interleave(64, dim=1)
    steps = torch.round(v * (torch.full_like(per, top) / per)).double()
    return steps * (per / torch.full_like(per, top)).double().nan_to_num(0.0, 0.0, 0.0) * torch.isfinite(per)


def _exact_norm(X):
    xd = X.double()
    mean = xd.sum(1) / X.shape[1]
    var = (xd * xd).sum(1) / X.shape[1] - mean * mean
    return xd, mean, torch.rsqrt(var + EPS)


def _exact_w4_quant(W, G, with_zeros):
    """Nearest codes by counting the borders passed, in 64 bits; a value on a border goes to the even side."""
    def steps(v, lo, hi):
        n = torch.full_like(v, float(lo))
        for j in range(lo, hi):
            n += (v > (j + 0.5) * s) if j % 2 == 0 else (v >= (j + 0.5) * s)
        return torch.where(s > 0, n, torch.zeros_like(n))

    out = torch.empty(W.shape, dtype=torch.float64, device=DEV)
    for c in range(0, W.shape[1], G):
        w = W[:, c:c + G].double()
        top, low = w.max(dim=1, keepdim=True).values, w.min(dim=1, keepdim=True).values
        if with_zeros:
            top, low = torch.relu(top), -torch.relu(-low)
            s = ((top.float() - low.float()) / torch.full_like(top, 15.0, dtype=F32)).to(BF16).double()
            z = steps(-low, 0, 15)
            q = torch.minimum(torch.maximum(steps(w, -16, 16), -z), 15 - z)
        else:
            s = (torch.maximum(top, -low).float() / torch.full_like(top, 7.0, dtype=F32)).to(BF16).double()
            q = steps(w, -8, 7)
        out[:, c:c + G] = q * s
    return out


def _exact_ln_grad(dY, xhat, rstd, weight):
    dy, w, K = dY.double(), weight.double(), dY.shape[1]
    a = (dy @ w) / K
    b = torch.einsum("mk,k,mk->m", dy, w, xhat) / K
    dx = rstd[:, None] * (dy * w[None, :] - a[:, None] - xhat * b[:, None])
    return dx, torch.einsum("mk,mk->k", dy, xhat), dy.sum(0)


def exact(case, seed):
    op = case["op"]
    if op == "w4_linear":
        x, codes, scales, zeros = _w4_parts(case, seed)
        G, K, N = case["group"], case["K"], case["N"]
        y = torch.zeros(case["M"], N, dtype=torch.float64, device=DEV)
        for g in range(-(-K // G)):  # one group of columns after the other
            q = codes[:, g * G:(g + 1) * G].double() - (8.0 if zeros is None else zeros[:, g:g + 1].double())
            y += (x[:, g * G:(g + 1) * G].double() @ q.t()) * scales[:, g].double()
        return y
    s = prepare(case, seed)
    if op == "w4_quant":
        return _exact_w4_quant(s["W"], case["group"], case["zeros"])
    if op == "relu2_step_q8":
        scale = (s["gamma_x"] * s["gamma_up"]) / torch.full_like(s["gamma_x"], 127.0)
        p = torch.relu(s["acc"].float() * scale[:, None])
        top = torch.relu(s["acc"].double().amax(1) * s["gamma_x"].double() * s["gamma_up"].double() / 127.0) ** 2
        return {"tokens": None, "gamma": top, "sums": None, "dH": 2.0 * _exact_checkpoint(p, 255.0) * s["dR"].double()}
    xd, mean, rstd = _exact_norm(s["X"])
    if op == "ln_grad":
        xhat = (xd - s["mean"].double()[:, None]) * s["rstd"].double()[:, None]
        dx, dw, db = _exact_ln_grad(s["dY"], xhat, s["rstd"].double(), s["weight"])
        return {"dX": dx, "dweight": dw, "dbias": db}
    y = (xd - mean[:, None]) * rstd[:, None] * s["weight"].double() + s["bias"].double()
    if op == "ln":
        return {"Y": y, "mean": mean, "rstd": rstd}
    out = {"tokens": None, "gamma": y.abs().amax(1), "sums": None, "rstd": rstd}
    if op == "ln_step_q8":
        m32, r32 = mean.float()[:, None], rstd.float()[:, None]
        kept = _exact_checkpoint((s["X"].float() - m32) * r32, 127.0)
        out["dX"], out["dweight"], out["dbias"] = _exact_ln_grad(s["dY"], kept, rstd, s["weight"])
    return out
