"""The pre-norm FFN block (prenorm_ffn.py): the layer norm, the int8 tokens, the
8-bit checkpoints and the straight-through gradients as they run together, and a
decode step through a 4-bit head."""
import numpy as np
import pytest
import torch

import oracle
import synth_inputs as si
import w4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5


@pytest.fixture(scope="module")
def bl():
    import ternary_weight_linear_absmax_b200 as m
    m.load()
    return m


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _block(bl, K, H, seed):
    from ternary_weight_linear_absmax_b200.prenorm_ffn import PreNormFFN
    Wu, Wd = si.weights(H, K, seed=seed, dtype="bf16"), si.weights(K, H, seed=seed + 1, dtype="bf16")
    lu, ld = Wu.torch(DEV), Wd.torch(DEV)
    pu, gu = bl.bl_quant_weights(lu, EPS)
    pd, gd = bl.bl_quant_weights(ld, EPS)
    rng = np.random.default_rng(seed)
    w = (1 + 0.1 * rng.standard_normal(K)).astype(np.float32)
    b = (0.1 * rng.standard_normal(K)).astype(np.float32)
    return PreNormFFN(_dev(w), _dev(b), pu, gu, pd, gd, EPS), (Wu, Wd, lu, ld, w, b)


@pytest.mark.parametrize("M,K,H", [(1, 64, 128), (4, 256, 640), (37, 512, 1408), (130, 1024, 2752)])
def test_forward(bl, M, K, H):
    """Against the oracle's integer steps on the fp32 values of the norm."""
    blk, (Wu, Wd, _, _, w, b) = _block(bl, K, H, M + K)
    X = si.activations(M, K, seed=M, outliers=True, dtype="bf16")
    y, saved = blk.forward(X.torch(DEV))
    assert torch.equal(y, blk.decode(X.torch(DEV)))
    A_q, gamma_a, rstd, xq, xs, R_q, gamma_r, p_q, p_s = saved
    x = X.f32
    mean = x.astype(np.float64).mean(1).astype(np.float32)
    r = rstd.cpu().numpy()
    v = ((((x - mean[:, None]).astype(np.float32) * r[:, None]).astype(np.float32) * w).astype(np.float32)
         + b).astype(np.float32)
    q, ga = oracle.quant_acts(v, EPS)
    np.testing.assert_array_equal(A_q.cpu().numpy(), q)
    cu, gu = oracle.quant_weights(Wu.f32, EPS)
    cd, gd = oracle.quant_weights(Wd.f32, EPS)
    rq, gr = oracle.relu2_requant(oracle.zero_gemm(q, cu), ga, gu, EPS)
    np.testing.assert_array_equal(R_q.cpu().numpy(), rq)
    np.testing.assert_array_equal(gamma_r.cpu().numpy(), gr)
    z = oracle.dequant_f32(oracle.zero_gemm(rq, cd), gr, gd).astype(np.float64)
    # the block's output and the residual sum are rounded to bf16 once each
    tol = 2.0 ** -8 * np.abs(z) + 2.0 ** -8 * (np.abs(z + x) + 2.0 ** -8 * np.abs(z)) + 1e-30
    assert np.all(np.abs(y.double().cpu().numpy() - (z + x)) <= tol * 1.001)


@pytest.mark.parametrize("M,K,H,dt", [(4, 64, 128, "f32"), (64, 512, 1408, "bf16"), (300, 1024, 2752, "bf16")])
def test_backward(bl, M, K, H, dt):
    """Every gradient against 64-bit formulas on what was saved. The two
    matrices' gradients and the values between them go through bf16 operands:
    each of the products in a gradient's chain (three at most, with the bf16
    dH between them) rounds independent operands by 2^-9 at most, so its error
    in the 2-norm stays below 2^-7 of its size for these random matrices."""
    blk, (Wu, Wd, lu, ld, w, _) = _block(bl, K, H, M + H)
    X = si.activations(M, K, seed=M, outliers=True, dtype="bf16").torch(DEV)
    dY = si.activations(M, K, seed=M + 9, dtype=dt)
    _, saved = blk.forward(X)
    got = blk.backward(dY.torch(DEV), saved, lu, ld)
    A_q, gamma_a, rstd, xq, xs, R_q, gamma_r, p_q, p_s = (t.double().cpu().numpy() for t in saved)
    dy = dY.f32.astype(np.float64)
    cu, gu = oracle.quant_weights(Wu.f32, EPS)
    cd, gd = oracle.quant_weights(Wd.f32, EPS)
    mu, md = oracle.ste_weight_mask(Wu.f32, gu, EPS), oracle.ste_weight_mask(Wd.f32, gd, EPS)
    up, down = float(gu) * cu.astype(np.float64), float(gd) * cd.astype(np.float64)
    dWd = md * (dy.T @ (R_q * (gamma_r / 127)[:, None]))
    p = p_q * np.repeat(p_s, 64, axis=1)
    dh = 2 * p * (dy @ down)
    dWu = mu * (dh.T @ (A_q * (gamma_a / 127)[:, None]))
    da = dh @ up
    dx, dw, db = ref.layernorm_grad(da, xq * np.repeat(xs, 64, axis=1), rstd, w.astype(np.float64))

    def near(t, want, products):
        d = np.linalg.norm(t.double().cpu().numpy() - want)
        assert d <= products * 2.0 ** -7 * np.linalg.norm(want), d / np.linalg.norm(want)

    near(got.dW_down, dWd, 1)
    near(got.dW_up, dWu, 2)
    near(got.dX, dx + dy, 3)
    near(got.dweight, dw, 3)
    near(got.dbias, db, 3)
    assert np.all(got.dW_up.cpu().numpy()[mu == 0] == 0) and np.all(got.dW_down.cpu().numpy()[md == 0] == 0)


def test_no_tokens(bl):
    blk, (_, _, lu, ld, _, _) = _block(bl, 64, 128, 3)
    X = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    y, saved = blk.forward(X)
    assert y.shape == (0, 64)


def test_step_in_a_graph(bl):
    """Forward and backward captured and replayed on new inputs, on a side
    stream, against the eager step."""
    M, K, H = 48, 256, 640
    blk, (_, _, lu, ld, _, _) = _block(bl, K, H, 5)
    X = [si.activations(M, K, seed=s, dtype="bf16").torch(DEV) for s in (1, 2)]
    dY = [si.activations(M, K, seed=s + 7, dtype="bf16").torch(DEV) for s in (1, 2)]

    def step(x, dy):
        y, saved = blk.forward(x)
        g = blk.backward(dy, saved, lu, ld)
        return [y, g.dX, g.dW_up, g.dW_down, g.dweight, g.dbias]

    want = [[t.clone() for t in step(x, dy)] for x, dy in zip(X, dY)]
    xin, dyin = torch.empty_like(X[0]), torch.empty_like(dY[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(xin, dyin)
    for i in (1, 0, 1):
        xin.copy_(X[i])
        dyin.copy_(dY[i])
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [1, 3, 12])
def test_decode_through_a_4bit_head(bl, M):
    """Layer norm → FFN → layer norm → 4-bit head: the logits against the
    unpacked head in 64 bits, and the greedy tokens of a short decode."""
    K, H, V = 256, 640, 1003
    blk, (*_, w, b) = _block(bl, K, H, 11)
    rng = np.random.default_rng(2)
    head = torch.from_numpy((rng.standard_normal((V, K)) * 0.05).astype(np.float32)).to(DEV)
    embed = head.bfloat16()
    W4, sc, zp = bl.bl_quant_weights_w4(head, 64, zeros=True)
    dense = bl.bl_unpack_w4(W4, sc, V, K, zeros=zp).double().cpu().numpy()
    x = embed[:M].contiguous()
    for _ in range(4):
        y = blk.decode(x)
        n, _, _ = bl.bl_layernorm(y, _dev(w), _dev(b))
        logits = bl.bl_linear_w4(n, W4, sc, V, zeros=zp, out_dtype=torch.float32)
        a = n.double().cpu().numpy()
        want = a @ dense.T
        assert np.all(np.abs(logits.double().cpu().numpy() - want)
                      <= ref.linear_bound(a, dense, K, False, want))
        x = embed[logits.argmax(1)].contiguous()
