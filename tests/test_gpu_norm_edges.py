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
