"""Layer norm and ReLU² tokens at the edges of their arguments."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def bl():
    import ternary_weight_linear_absmax_b200 as m
    m.load()
    return m


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("M,K", [(3, 64), (4, 2560), (5, 10240), (700, 4096), (300, 12288), (2, 20480)])
def test_layernorm_tokens_where_the_scale_overflows(bl, M, K, checkpoint):
    """127/(max + eps) is infinite below max + eps = 3.7e-37: the tokens are still
    those of bl_quant_acts (the ends of the range), row sums included."""
    g = torch.Generator().manual_seed(M + K)
    X = torch.randn(M, K, generator=g).to(DEV)
    weight, bias = torch.full((K,), 1e-39, device=DEV), torch.zeros(K, device=DEV)
    weight[::7] = 0.0                                 # tokens of zeros
    y, _, _ = bl.bl_layernorm(X, weight, bias, out_dtype=torch.float32)
    for q_eps in (1e-39, 3e-37, 1e-5):
        want = bl.bl_quant_acts(y, q_eps)
        got = bl.bl_layernorm_quant(X, weight, bias, q_eps=q_eps, checkpoint=checkpoint)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert want[0].abs().max() == 0


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("M,H", [(3, 64), (4, 2752), (2, 16448), (300, 704)])
def test_relu2_tokens_where_the_scale_overflows(bl, M, H, checkpoint):
    g = torch.Generator().manual_seed(M + H)
    acc = torch.randint(-2000, 2000, (M, H), generator=g, dtype=torch.int32).to(DEV)
    gx, gu = torch.full((M,), 1e-18, device=DEV), torch.full((1,), 1e-3, device=DEV)
    sc = (gx * gu) / torch.full_like(gx, 127.0)
    r = (acc.float() * sc[:, None]).clamp(min=0).square()
    assert 0 < r.max() < 1e-37
    for eps in (1e-39, 3e-37, 1e-5):
        want = bl.bl_quant_acts(r, eps)
        got = bl.bl_relu2_requant_q8(acc, gx, gu, eps, checkpoint=checkpoint)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_no_rows_through_the_block(bl):
    """A batch without rows: outputs without rows, gradients of zero."""
    from ternary_weight_linear_absmax_b200.prenorm_ffn import PreNormFFN
    K, H = 256, 640
    lu, ld = torch.randn(H, K, device=DEV), torch.randn(K, H, device=DEV)
    (pu, gu), (pd, gd) = bl.bl_quant_weights(lu), bl.bl_quant_weights(ld)
    blk = PreNormFFN(torch.ones(K, device=DEV), None, pu, gu, pd, gd)
    X = torch.empty(0, K, device=DEV, dtype=torch.bfloat16)
    y, saved = blk.forward(X)
    assert y.shape == (0, K) and blk.decode(X).shape == (0, K)
    g = blk.backward(torch.empty_like(X), saved, lu, ld)
    assert g.dX.shape == (0, K)
    for t, shape in ((g.dW_up, (H, K)), (g.dW_down, (K, H)), (g.dweight, (K,)), (g.dbias, (K,))):
        assert t.shape == shape and torch.all(t == 0)


@pytest.mark.parametrize("M,H", [(296, 4096), (297, 4096), (297, 2752), (400, 10240), (300, 16384), (300, 13824)])
def test_relu2_rows_together_and_in_parts(bl, M, H):
    """A row's codes do not depend on how many rows come with it, on either side of
    the border between the two forms."""
    g = torch.Generator().manual_seed(M + H)
    acc = torch.randint(-3000, 3000, (M, H), generator=g, dtype=torch.int32).to(DEV)
    gx, gu = torch.rand(M, generator=g).to(DEV) + 0.5, torch.full((1,), 0.016, device=DEV)
    whole = bl.bl_relu2_requant_q8(acc, gx, gu)
    for m in range(0, M, 92):
        part = bl.bl_relu2_requant_q8(acc[m:m + 92], gx[m:m + 92], gu)
        for a, b in zip(whole, part):
            assert torch.equal(a[m:m + 92], b)


@pytest.mark.parametrize("M,K", [(443, 2560), (444, 2560), (3, 4096), (5, 5120), (9, 6912), (2, 8192), (444, 8192)])
def test_layernorm_forms(bl, M, K):
    """Rows on both sides of the borders between the forms: the tokens are those of
    bl_quant_acts on the floats, these are within the roundings of the formula, and the
    checkpoint is within half a step."""
    g = torch.Generator().manual_seed(M + K)
    X = (torch.randn(M, K, generator=g) * 2 + 0.5).to(DEV)
    w, b = (torch.rand(K, generator=g) + 0.5).to(DEV), torch.randn(K, generator=g).to(DEV)
    y, mean, rstd = bl.bl_layernorm(X, w, b, out_dtype=torch.float32)
    got = bl.bl_layernorm_quant(X, w, b, checkpoint=True)
    for a, c in zip(got, bl.bl_quant_acts(y)):
        assert torch.equal(a, c)
    xh = (X.double() - X.double().mean(1, keepdim=True)) * (X.double().var(1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
    # mean and rstd are rounded once, then one rounding per step: d, x̂, x̂·w, y
    tol = 2.0 ** -24 * (6 * (xh * w).abs() + 2 * (rstd * mean.abs())[:, None] * w + (xh * w + b).abs())
    assert torch.all((y - (xh * w + b)).abs() <= tol * 1.01)
    back = got[4].double().view(M, K // 64, 64) * got[5].double()[:, :, None]
    top = xh.abs().view(M, K // 64, 64).amax(2, keepdim=True)
    assert torch.all((back - xh.view_as(back)).abs() <= top * (0.5 / 127 + 2.0 ** -20))
