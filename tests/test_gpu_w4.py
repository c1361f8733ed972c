"""4-bit weights with group scales through the C ABI: the quantiser and the
packing bit for bit, the product against 64 bits."""
import numpy as np
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


def _weights(N, K, seed, dt):
    rng = np.random.default_rng(seed)
    W = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    W[0, :min(K, 32)] = 0.0                       # an empty group
    if N > 2:
        W[2] = np.abs(W[2])                       # one sign only
    return torch.from_numpy(W).to(ref.KINDS[dt])


def _unpacked(bl, W4, scales, zp, N, K):
    return bl.bl_unpack_w4(W4, scales, N, K, zeros=zp).cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,K,group", [(1, 64, 32), (16, 128, 128), (37, 192, 128), (50, 320, 64),
                                       (33, 1088, 32)])
def test_quantiser_bit_exact(bl, N, K, group, zeros, dt):
    W = _weights(N, K, N + K, dt)
    W4, scales, zp = bl.bl_quant_weights_w4(W.to(DEV), group, zeros=zeros)
    codes, s, z = ref.quant_w4(W.float().numpy(), group, zeros)
    words, sc, zpr = ref.pack(codes, s, z, group, zeros)
    got = W4.cpu().numpy().view(np.uint32).reshape(words.shape)
    rows = np.zeros((words.shape[0] * 16, words.shape[1] * 128), bool)
    rows[:N, :K] = True
    inside = rows.reshape(words.shape[0], 2, 8, words.shape[1], 4, 4, 8).all(-1).transpose(0, 3, 1, 2, 5, 4)
    np.testing.assert_array_equal(got[inside], words[inside])
    np.testing.assert_array_equal(_unpacked(bl, W4, scales, zp, N, K), ref.dequant(codes, s, z, group))
    # what lies outside the matrix has scale 0
    full = scales.float().cpu().numpy()
    np.testing.assert_array_equal(full, sc)
    assert (zp is None) == (not zeros)
    # the same codes through bl_pack_w4
    nib = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    P4, psc, pzp = bl.bl_pack_w4(torch.from_numpy(nib).to(DEV), torch.from_numpy(s).bfloat16().to(DEV), group,
                                 zeros=torch.from_numpy(z.astype(np.uint8)).to(DEV) if zeros else None)
    np.testing.assert_array_equal(P4.cpu().numpy().view(np.uint32).reshape(words.shape)[inside], words[inside])
    np.testing.assert_array_equal(psc.float().cpu().numpy(), sc)
    np.testing.assert_array_equal(_unpacked(bl, P4, psc, pzp, N, K), ref.dequant(codes, s, z, group))
    half = bl.bl_unpack_w4(W4, scales, N, K, zeros=zp, out_dtype=torch.bfloat16).float().cpu().numpy()
    np.testing.assert_array_equal(half, ref.bf16(ref.dequant(codes, s, z, group)))


def test_quantiser_borders(bl):
    """Values on, just below and just above (k + 1/2)·s, and scales from the
    smallest bf16 up: ties go to the even code, neighbours to their side."""
    rows = []
    for s in (np.float32(2.0 ** -7), np.float32(0.0078735352), np.float32(2.0 ** -126), np.float32(2.0 ** -132)):
        b = ((np.arange(-7, 7) + 0.5) * np.float64(s)).astype(np.float32)
        row = np.concatenate([b, np.nextafter(b, np.float32(np.inf)), np.nextafter(b, np.float32(-np.inf)),
                              [7 * s, -7 * s], np.zeros(20, np.float32)]).astype(np.float32)
        rows.append(row[:64])
    rows.append(np.full(64, 2.0 ** -149, np.float32))   # below every bf16: scale 0
    W = np.stack(rows)
    for zeros in (False, True):
        codes, s, z = ref.quant_w4(W, 64, zeros)
        W4, scales, zp = bl.bl_quant_weights_w4(torch.from_numpy(W).to(DEV), 64, zeros=zeros)
        np.testing.assert_array_equal(_unpacked(bl, W4, scales, zp, *W.shape), ref.dequant(codes, s, z, 64))


def _problem(bl, M, N, K, group, zeros, dt, seed):
    rng = np.random.default_rng(seed)
    G = -(-K // group)
    codes = rng.integers(0, 16, (N, K))
    s = ref.bf16(rng.uniform(0.002, 0.01, (N, G)).astype(np.float32))
    z = rng.integers(0, 16, (N, G)) if zeros else np.full((N, G), 8)
    nib = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    packed = bl.bl_pack_w4(torch.from_numpy(nib).to(DEV), torch.from_numpy(s).bfloat16().to(DEV), group,
                           zeros=torch.from_numpy(z.astype(np.uint8)).to(DEV) if zeros else None)
    X = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(ref.KINDS[dt])
    return X, packed, ref.dequant(codes, s, z, group)


def _check(bl, M, N, K, group, zeros, xdt, ydt, seed=0):
    X, (W4, sc, zp), w = _problem(bl, M, N, K, group, zeros, xdt, seed)
    Y = bl.bl_linear_w4(X.to(DEV), W4, sc, N, zeros=zp, out_dtype=ref.KINDS[ydt])
    x = X.double().numpy()
    want = x @ w.T
    got = Y.double().cpu().numpy()
    tol = ref.linear_bound(x, w, K, ydt == "bf16", want)
    assert got.shape == want.shape
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("M,N,K,group,zeros,xdt,ydt", [
    (1, 1, 64, 32, False, "bf16", "f32"), (1, 16, 128, 128, True, "f32", "f32"),
    (2, 17, 192, 64, True, "bf16", "bf16"), (3, 250, 512, 32, False, "f32", "bf16"),
    (4, 256, 512, 32, True, "f32", "f32"), (5, 129, 448, 128, False, "f32", "f32"),
    (7, 100, 1088, 64, False, "bf16", "f32"), (8, 333, 2560, 128, True, "bf16", "bf16"),
    (9, 64, 4096, 32, True, "bf16", "f32"), (11, 48, 704, 32, False, "f32", "f32"),
    (16, 555, 1024, 64, True, "bf16", "bf16"), (17, 40, 640, 128, False, "bf16", "f32"),
    (33, 70, 576, 64, True, "f32", "bf16"), (64, 96, 1280, 128, True, "bf16", "f32"),
    (65, 31, 320, 32, False, "bf16", "f32"), (130, 20, 192, 64, True, "f32", "f32")])
def test_linear(bl, M, N, K, group, zeros, xdt, ydt):
    _check(bl, M, N, K, group, zeros, xdt, ydt, seed=M * N)


@pytest.mark.parametrize("M,N,K,group", [(1, 6912, 2560, 128), (2, 300, 37440, 64), (1, 40, 262144, 128),
                                         (16, 11008, 1024, 64), (1, 20011, 512, 32)])
def test_linear_long(bl, M, N, K, group):
    """The decode matrix, long rows and many rows."""
    _check(bl, M, N, K, group, True, "bf16", "f32", seed=K)


@pytest.mark.parametrize("M,N,K,group", [(1, 60000, 128, 128), (3, 50000, 256, 64), (2, 47360, 384, 32),
                                         (5, 128256, 192, 64), (7, 80000, 256, 128), (16, 40000, 320, 32)])
def test_linear_runs_of_whole_row_blocks(bl, M, N, K, group):
    """Short rows, many of them: a warp's run holds whole row blocks between
    the ones that it shares with its neighbours. Twice, with another call's
    leftovers in shared memory between."""
    _check(bl, M, N, K, group, False, "bf16", "f32", seed=N)
    _check(bl, 4, 1000, 2048, 32, True, "f32", "f32", seed=1)
    _check(bl, M, N, K, group, True, "f32", "bf16", seed=N + 1)


def test_linear_seeded_shapes(bl):
    rng = np.random.default_rng(7)
    for i in range(24):
        M, N, K = int(rng.integers(1, 40)), int(rng.integers(1, 700)), 64 * int(rng.integers(1, 40))
        _check(bl, M, N, K, int(rng.choice([32, 64, 128])), bool(rng.integers(2)),
               ["bf16", "f32"][rng.integers(2)], ["bf16", "f32"][rng.integers(2)], seed=i)


def test_fp32_values_of_all_sizes(bl):
    """An fp32 activation keeps its 24 bits, from the smallest values to the
    largest that the sum allows."""
    K, N = 64, 16
    X, (W4, sc, zp), w = _problem(bl, 4, N, K, 32, False, "f32", 3)
    x = X.numpy() * np.array([1e-30, 1.0, 1e30, 3e37], np.float32)[:, None]
    x[0, 0], x[1, 1], x[3] = 1.17549435e-38, 1 + 2.0 ** -23, 0
    x[3, 5] = 3.4e38
    got = bl.bl_linear_w4(torch.from_numpy(x).to(DEV), W4, sc, N, out_dtype=torch.float32)
    want = x.astype(np.float64) @ w.T
    tol = ref.linear_bound(x.astype(np.float64), w, K, False, want)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)


def test_empty_and_outputs_untouched(bl):
    X, (W4, sc, zp), w = _problem(bl, 3, 21, 192, 64, True, "bf16", 5)
    Xd = X.to(DEV)
    assert bl.bl_linear_w4(Xd[:0], W4, sc, 21, zeros=zp).shape == (0, 21)
    # the buffer behind the output stays as it was
    buf = torch.full((3 * 21 + 64,), 7.0, device=DEV)
    out = buf[:63].view(3, 21)
    bl.bl_linear_w4(Xd, W4, sc, 21, zeros=zp, out=out)
    assert torch.all(buf[63:] == 7.0)
    assert torch.equal(out, bl.bl_linear_w4(Xd, W4, sc, 21, zeros=zp, out_dtype=torch.float32))


def test_nan_outside_the_matrix_is_not_read(bl):
    """Rows past N and columns past K never reach a result, whatever their
    codes; scales there are 0 by construction."""
    N, K = 5, 64
    X, (W4, sc, zp), w = _problem(bl, 2, N, K, 32, False, "bf16", 6)
    base = bl.bl_linear_w4(X.to(DEV), W4, sc, N, out_dtype=torch.float32)
    words = W4.view(-1, 2, 8, 4, 4, 4)
    words[:, :, :, :, 2:] = 0xFF                   # columns 64..127
    words[:, 1] = 0xFF                             # rows 8..15
    assert torch.equal(base, bl.bl_linear_w4(X.to(DEV), W4, sc, N, out_dtype=torch.float32))


def test_streams_graph_and_repeat(bl):
    """On a side stream, in a captured and replayed graph, and with programmatic
    dependent launch in a chain: the same bits as the plain call."""
    N, K = 4096, 4096
    X, (W4, sc, zp), w = _problem(bl, 2, N, K, 128, True, "bf16", 8)
    X = X.to(DEV)
    base = bl.bl_linear_w4(X, W4, sc, N, zeros=zp)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = bl.bl_linear_w4(X, W4, sc, N, zeros=zp, stream=side)
    side.synchronize()
    assert torch.equal(base, other)
    out = torch.empty_like(base)
    chain = [torch.empty_like(base) for _ in range(4)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h = X
        for c in chain:
            bl.bl_linear_w4(h, W4, sc, N, zeros=zp, out=c, pdl=True)
            h = c
        bl.bl_linear_w4(X, W4, sc, N, zeros=zp, out=out, pdl=True)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(base, out) and torch.equal(base, chain[0])
    h = X
    for c in chain:
        h = bl.bl_linear_w4(h, W4, sc, N, zeros=zp)
        assert torch.equal(h, c)


def test_keyword_calls_run_on_their_stream(bl, monkeypatch):
    """The stream that a call names is the one it runs on, also where its first
    argument is not a tensor."""
    W = torch.randn(64, 256, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    seen, on = [], bl._on
    monkeypatch.setattr(bl, "_on", lambda **t: seen.append(on(**t)) or seen[-1])
    W4, sc, zp = bl.bl_quant_weights_w4(group=32, zeros=True, W=W, stream=side)
    Y = bl.bl_linear_w4(zeros=zp, N=64, X=W[:3], W4=W4, scales=sc, stream=side)
    assert seen == [side.cuda_stream] * 2
    side.synchronize()
    a, b, c = bl.bl_quant_weights_w4(W, 32, zeros=True)
    assert torch.equal(a, W4) and torch.equal(b, sc) and torch.equal(c, zp)
    assert torch.equal(bl.bl_linear_w4(W[:3], a, b, 64, zeros=c), Y)


def test_many_tokens_share_a_workspace_in_order(bl):
    """Calls of more than five tokens with one caller-owned workspace, chained
    with programmatic dependent launch: each overwrites what the one before
    read, in order."""
    N = K = 2048
    X, (W4, sc, zp), w = _problem(bl, 20, N, K, 64, True, "f32", 12)
    X = X.to(DEV)
    L = bl.load()
    ws = torch.empty(int(L.bl_linear_w4_workspace_bytes(20, K, 64)), dtype=torch.uint8, device=DEV)
    want, h = [], X
    for _ in range(6):
        h = (bl.bl_linear_w4(h, W4, sc, N, zeros=zp, out_dtype=torch.float32) * 0.1).contiguous()
        want.append(h)
    h = X
    for i in range(6):
        h = (bl.bl_linear_w4(h, W4, sc, N, zeros=zp, out_dtype=torch.float32, workspace=ws, pdl=True)
             * 0.1).contiguous()
        assert torch.equal(h, want[i])
    with pytest.raises(bl.BitLinearError, match="WORKSPACE"):
        bl.bl_linear_w4(X, W4, sc, N, zeros=zp, workspace=ws[:64])


def test_weights_past_two_to_the_32(bl):
    """5.4e9 weights (2.7 GB of codes): the last rows equal those of a slice."""
    N, K = 164000, 32768
    W4 = torch.randint(0, 256, (N // 16, K // 128, 1024), dtype=torch.uint8, device=DEV)
    sc = torch.rand((N // 16, K // 128, 8, 1, 2), device=DEV).mul_(0.01).bfloat16()
    X = torch.randn(2, K, device=DEV).bfloat16()
    y = bl.bl_linear_w4(X, W4, sc, N, out_dtype=torch.float32)
    tail = bl.bl_linear_w4(X, W4[-4:].contiguous(), sc[-4:].contiguous(), 64, out_dtype=torch.float32)
    # the runs of a slab, and so the order of a row's fp32 sums, are the shape's
    assert torch.allclose(y[:, -64:], tail, rtol=0, atol=float(2.0 ** -20 * y.abs().max()))
    dense = bl.bl_unpack_w4(W4, sc, N, K, out_dtype=torch.bfloat16)
    assert torch.equal(dense[-16:], bl.bl_unpack_w4(W4[-1:].contiguous(), sc[-1:].contiguous(), 16, K,
                                                    out_dtype=torch.bfloat16))


def test_long_rows_in_clusters(bl):
    """The longest rows with every group size, and with more row blocks than a
    cluster keeps sums of."""
    for M, N, K, group in ((1, 48, 262144, 32), (2, 33, 262144, 64), (3, 20, 131072, 128), (9, 40, 65536, 32),
                           (1, 9000, 65536, 32)):
        _check(bl, M, N, K, group, True, "f32", "f32", seed=M + N)


def test_nan_and_infinity_reach_their_token_only(bl):
    X, (W4, sc, zp), w = _problem(bl, 4, 80, 512, 64, True, "f32", 9)
    base = bl.bl_linear_w4(X.to(DEV), W4, sc, 80, zeros=zp, out_dtype=torch.float32)
    X[1, 300], X[3, 5] = float("nan"), float("inf")
    got = bl.bl_linear_w4(X.to(DEV), W4, sc, 80, zeros=zp, out_dtype=torch.float32)
    assert torch.isnan(got[1]).all() and torch.isnan(got[3]).all()
    assert torch.equal(got[[0, 2]], base[[0, 2]])


@pytest.mark.parametrize("M,N,K,group", [(6, 33, 64, 32), (8, 200, 704, 64), (13, 100, 4096, 128),
                                         (16, 70, 8192, 32), (23, 48, 1024, 64)])
def test_bf16_tokens_exact(bl, M, N, K, group):
    """Whole numbers and scales that are powers of two: every product and sum is a
    multiple of the smallest scale and below 2^24 of it, so the result is the exact one."""
    rng = np.random.default_rng(M)
    G = -(-K // group)
    codes, z = rng.integers(0, 16, (N, K)), rng.integers(0, 16, (N, G))
    s = 2.0 ** rng.integers(-2, 2, (N, G))      # |sum| <= 8192·15·15·8 quarters < 2^24
    nib = torch.from_numpy((codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)).to(DEV)
    W4, sc, zp = bl.bl_pack_w4(nib, torch.from_numpy(s).bfloat16().to(DEV), group,
                               zeros=torch.from_numpy(z.astype(np.uint8)).to(DEV))
    x = rng.integers(-15, 16, (M, K))
    X = torch.from_numpy(x).bfloat16().to(DEV)
    want = x @ ref.dequant(codes, s, z, group).T
    np.testing.assert_array_equal(bl.bl_linear_w4(X, W4, sc, N, zeros=zp, out_dtype=torch.float32).cpu().numpy(),
                                  want)


@pytest.mark.parametrize("M", [7, 20])
def test_bf16_nan_and_infinity_reach_their_token_only(bl, M):
    X, (W4, sc, zp), w = _problem(bl, M, 80, 576, 64, True, "bf16", 9)
    base = bl.bl_linear_w4(X.to(DEV), W4, sc, 80, zeros=zp, out_dtype=torch.float32)
    X[1, 570], X[M - 1, 5] = float("nan"), float("inf")
    got = bl.bl_linear_w4(X.to(DEV), W4, sc, 80, zeros=zp, out_dtype=torch.float32)
    assert torch.isnan(got[1]).all() and not got[M - 1].isfinite().any()
    rest = [m for m in range(M) if m not in (1, M - 1)]
    assert torch.equal(got[rest], base[rest])


def test_bf16_rows_too_long_for_sixteen(bl):
    """Rows whose 16 or 8 bf16 tokens do not fit in a cluster's shared memory."""
    for M, N, K, group in ((16, 40, 65536, 32), (9, 33, 131072, 64), (6, 20, 262144, 128)):
        _check(bl, M, N, K, group, True, "bf16", "f32", seed=M)


def test_wide_range_within_a_block(bl):
    """Values of very different size in one 128-column block: off by at most half
    of 2^-22 of the block's largest value per column, and the sums' own error."""
    X, (W4, sc, zp), w = _problem(bl, 3, 64, 384, 128, True, "f32", 10)
    x = X.numpy() * np.exp(np.random.default_rng(1).uniform(-12, 6, X.shape)).astype(np.float32)
    got = bl.bl_linear_w4(torch.from_numpy(x).to(DEV), W4, sc, 64, zeros=zp, out_dtype=torch.float32)
    want = x.astype(np.float64) @ w.T
    top = np.abs(x).reshape(3, 3, 128).max(2)
    cols = np.abs(w).reshape(64, 3, 128).sum(2)
    tol = ref.linear_bound(x.astype(np.float64), w, 384, False, want) + 2.0 ** -23 * 2 * (top @ cols.T)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
