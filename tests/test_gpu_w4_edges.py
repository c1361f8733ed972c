"""4-bit weights at the edges of their arguments."""
import pytest
import torch

import w4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def bl():
    import ternary_weight_linear_absmax_b200 as m
    m.load()
    return m


@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,group", [(16, 128, 128), (37, 320, 64), (33, 1088, 32)])
def test_broken_weights_stay_broken(bl, N, K, group, zeros, dt, value):
    """A NaN or an infinity in a group makes the whole group NaN or infinite when it
    is read back, and the row's results with it; other groups are not touched."""
    g = torch.Generator().manual_seed(N + K)
    W = (torch.randn(N, K, generator=g) * 0.02).to(ref.KINDS[dt])
    at = [(0, 3), (N - 1, K - 1), (N // 2, group + 5 if K > group else 5)]
    bad = W.clone()
    groups = torch.zeros(N, K, dtype=torch.bool)
    for n, k in at:
        bad[n, k] = float(value)
        groups[n, k // group * group:(k // group + 1) * group] = True
    W4, sc, zp = bl.bl_quant_weights_w4(bad.to(DEV), group, zeros=zeros)
    if zeros:
        assert zp.max() <= 15
    got = bl.bl_unpack_w4(W4, sc, N, K, zeros=zp).cpu()
    good = bl.bl_quant_weights_w4(W.to(DEV), group, zeros=zeros)
    want = bl.bl_unpack_w4(good[0], good[1], N, K, zeros=good[2]).cpu()
    assert torch.equal(got[~groups], want[~groups])
    assert not got[groups].isfinite().any()
    if value == "nan":
        assert got[groups].isnan().all()
    rows = groups.any(1)
    for M, xdt in ((2, "bf16"), (7, "bf16"), (7, "f32")):
        X = torch.randn(M, K, generator=g).to(ref.KINDS[xdt]).to(DEV)
        y = bl.bl_linear_w4(X, W4, sc, N, zeros=zp, out_dtype=torch.float32).cpu()
        assert not y[:, rows].isfinite().any()
        assert torch.equal(y[:, ~rows], bl.bl_linear_w4(X, good[0], good[1], N, zeros=good[2],
                                                        out_dtype=torch.float32).cpu()[:, ~rows])
