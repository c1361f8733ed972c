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


@pytest.mark.parametrize("M,K,group", [(20, 2048, 64), (7, 512, 32), (16, 4096, 128)])
def test_calls_that_share_a_workspace(bl, M, K, group):
    """fp32 calls of more than five tokens, issued back to back with programmatic
    dependent launch and one workspace: nothing runs between them, so a call's
    digits are written as soon as the call before has read its own. Eagerly, and
    captured and replayed; every call has activations of its own."""
    N, calls = K, 8
    g = torch.Generator().manual_seed(K)
    W = torch.randn(N, K, generator=g).to(DEV)
    W4, sc, zp = bl.bl_quant_weights_w4(W, group, zeros=True)
    X = [torch.randn(M, K, generator=g).to(DEV) for _ in range(calls)]
    want = [bl.bl_linear_w4(x, W4, sc, N, zeros=zp, out_dtype=torch.float32) for x in X]
    ws = torch.empty(int(bl.load().bl_linear_w4_workspace_bytes(M, K, group)), dtype=torch.uint8, device=DEV)
    out = [torch.zeros_like(w) for w in want]

    def run():
        for x, y in zip(X, out):
            bl.bl_linear_w4(x, W4, sc, N, zeros=zp, out=y, workspace=ws, pdl=True)

    for _ in range(3):
        run()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for y in out:
            y.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    # a chain: each call reads what the one before wrote
    sc2 = (sc.float() * 0.02).bfloat16()
    h, chain = X[0], []
    for _ in range(calls):
        h = bl.bl_linear_w4(h, W4, sc2, N, zeros=zp, out_dtype=torch.float32)
        chain.append(h)
    h = X[0]
    for y in out:
        bl.bl_linear_w4(h, W4, sc2, N, zeros=zp, out=y, workspace=ws, pdl=True)
        h = y
    assert all(torch.equal(a, b) for a, b in zip(out, chain)) and chain[-1].isfinite().all()


def test_memory_of_a_side_streams_inputs_is_kept(bl):
    """A temporary that a call on a side stream reads may be dropped right after
    the call: its memory is not handed out before the call has run."""
    g = torch.Generator(device=DEV).manual_seed(1)
    W4, sc, zp = bl.bl_quant_weights_w4(torch.randn(512, 4096, generator=g, device=DEV), 64, zeros=True)
    side = torch.cuda.Stream()
    base = torch.randn(64, 4096, generator=g, device=DEV)
    want = bl.bl_linear_w4(base, W4, sc, 512, zeros=zp, out_dtype=torch.float32)
    X = base.clone()
    side.wait_stream(torch.cuda.current_stream())
    # twice: the first call leaves its output's and workspace's memory to the second,
    # which then allocates nothing anew (an allocation waits for the device)
    for _ in range(2):
        y = bl.bl_linear_w4(X, W4, sc, 512, zeros=zp, out_dtype=torch.float32, stream=side)
        side.synchronize()
    del y
    where, shape = X.data_ptr(), X.shape
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)          # about 50 ms of work ahead of the call
    y = bl.bl_linear_w4(X, W4, sc, 512, zeros=zp, out_dtype=torch.float32, stream=side)
    del X
    fresh = torch.empty(shape, device=DEV)
    assert fresh.data_ptr() != where or side.query()     # handed out again only once the call has run
    fresh.fill_(7.0)
    side.synchronize()
    assert torch.equal(y, want)
