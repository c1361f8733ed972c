"""Layer norm (floats, int8 tokens, backward) and the 8-bit activation
checkpoints through the C ABI against 64-bit formulas."""
import numpy as np
import pytest
import torch

import oracle
import w4_ref as ref
from parity_helpers import assert_acts_match

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = float(np.float32(1e-5))
U = 2.0 ** -24
SHAPES = [(1, 64), (3, 192), (2, 2048), (5, 2560), (37, 4096), (4, 11008), (301, 320), (700, 64), (2, 16448)]


@pytest.fixture(scope="module")
def bl():
    import ternary_weight_linear_absmax_b200 as m
    m.load()
    return m


def _rows(M, K, seed, dt):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) + 0.3
    x *= np.where(rng.random(K) < 0.02, 20.0, 1.0)
    if M > 1:
        x[1] = 0.75                       # a row without spread
    if M > 2:
        x[2] = 1000.0 + 0.01 * x[2]       # a far mean
    if M > 3:
        x[3] = 0.0
    return torch.from_numpy(x.astype(np.float32)).to(ref.KINDS[dt])


def _affine(K, seed):
    rng = np.random.default_rng(seed + 1)
    return ((1 + 0.1 * rng.standard_normal(K)).astype(np.float32),
            (0.1 * rng.standard_normal(K)).astype(np.float32))


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _ulps(got, want):
    w = want.astype(np.float32)
    return np.max(np.abs(got.astype(np.float64) - want) / np.spacing(np.abs(w) + np.float32(1e-38)))


def _y32(x, mean, rstd, w, b):
    """The fp32 values that the kernels round: one operation each."""
    xh = ((x - mean[:, None]).astype(np.float32) * rstd[:, None]).astype(np.float32)
    y = (xh * w).astype(np.float32)
    return xh, (y + b).astype(np.float32) if b is not None else y


@pytest.mark.parametrize("xdt,ydt,bias", [("bf16", "bf16", True), ("f32", "f32", True), ("bf16", "f32", False),
                                          ("f32", "bf16", False)])
@pytest.mark.parametrize("M,K", SHAPES)
def test_layernorm(bl, M, K, xdt, ydt, bias):
    X = _rows(M, K, M + K, xdt)
    w, b = _affine(K, K)
    b = b if bias else None
    Y, mean, rstd = bl.bl_layernorm(X.to(DEV), _dev(w), _dev(b) if bias else None,
                                    out_dtype=ref.KINDS[ydt])
    x = X.float().numpy()
    mean, rstd = mean.cpu().numpy(), rstd.cpu().numpy()
    m64 = x.astype(np.float64).mean(1)
    # rounded once from a 64-bit sum: half a step, plus what 64 bits lose
    assert np.all(np.abs(mean - m64) <= U * np.abs(m64) + 1e-12 * np.abs(x).max(1))
    d = (x - mean[:, None]).astype(np.float32).astype(np.float64)
    r64 = 1 / np.sqrt((d * d).mean(1) + EPS)
    assert np.all(np.abs(rstd - r64) <= 1.001 * U * r64)
    _, y = _y32(x, mean, rstd, w, b)
    want = ref.bf16(y) if ydt == "bf16" else y
    np.testing.assert_array_equal(Y.float().cpu().numpy(), want)
    # and the definition in 64 bits: d is off by half a step of x − μ and by μ's
    # own rounding, three more fp32 operations follow
    y64, _, r, xh = ref.layernorm(x, w, b, EPS)
    tol = (6 * U * (np.abs(xh * w) + np.abs(y64) + (np.abs(b) if bias else 0))
           + 2 * U * np.abs(w) * (np.abs(m64) * r)[:, None]
           # μ's rounding also raises the mean of d² by its square
           + np.abs(xh * w) * ((U * m64 * r) ** 2)[:, None])
    got = Y.double().cpu().numpy()
    assert np.all(np.abs(got - y64) <= tol + (2.0 ** -8 * (np.abs(y64) + tol) if ydt == "bf16" else 0))


@pytest.mark.parametrize("xdt", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", SHAPES)
def test_layernorm_quant(bl, M, K, xdt):
    X = _rows(M, K, 3 * M + K, xdt)
    w, b = _affine(K, K + 1)
    _, mean, rs = bl.bl_layernorm(X.to(DEV), _dev(w), _dev(b))
    x, mean = X.float().numpy(), mean.cpu().numpy()
    for keep in (False, True):
        Aq, gA, sums, rstd, xq, xs = bl.bl_layernorm_quant(X.to(DEV), _dev(w), _dev(b), checkpoint=keep)
        assert torch.equal(rstd, rs)
        xh, y = _y32(x, mean, rstd.cpu().numpy(), w, b)
        assert_acts_match(Aq.cpu().numpy(), gA.cpu().numpy(), sums.cpu().numpy(), y, what="layernorm tokens")
        if not keep:
            assert xq is None and xs is None
            continue
        codes, scale = ref.checkpoint(xh, 127.0)
        np.testing.assert_array_equal(xs.cpu().numpy(), scale)
        np.testing.assert_array_equal(xq.cpu().numpy(), codes)
        back = xq.cpu().numpy().reshape(M, K // 64, 64) * scale[:, :, None].astype(np.float64)
        # half a step: codes and scale are quotients of the same maximum, each
        # off by U, and the product by another
        assert np.all(np.abs(back - xh.reshape(back.shape)) <= (0.5 + 127 * 4 * U) * scale[:, :, None])
    # without the optional outputs and without bias
    Aq2 = bl.bl_layernorm_quant(X.to(DEV), _dev(w))[0]
    _, y = _y32(x, mean, rs.cpu().numpy(), w, None)
    q, _ = oracle.quant_acts(y, 1e-5)
    assert np.max(np.abs(Aq2.cpu().numpy().astype(int) - q)) <= 1


def _grad_check(dX, dw, db, dy, xh, rstd, w, dx_bf16, M):
    want, ww, wb = ref.layernorm_grad(dy, xh, rstd, w)
    g = dy * w
    K = dy.shape[1]
    # row sums: at most K/256 sequential terms per thread, then 13 steps; x̂ two
    # fp32 operations, products one each; column sums: M/100 rows in sequence
    # at most (the grid has at least 100 CTAs or one per row), 512 partial sums
    n = K / 256 + 8 + 13
    a, b = np.abs(g).mean(1)[:, None], np.abs(g * xh).mean(1)[:, None]
    tol = rstd[:, None] * U * (8 * (np.abs(g) + np.abs(xh) * b + a) + n * (a + np.abs(xh) * b)) + 1e-37
    if dx_bf16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    assert np.all(np.abs(dX - want) <= tol), np.max(np.abs(dX - want) / tol)
    steps = M / 100 + 512 + 4
    assert np.all(np.abs(dw - ww) <= steps * U * np.abs(dy * xh).sum(0) + 1e-37)
    assert np.all(np.abs(db - wb) <= steps * U * np.abs(dy).sum(0) + 1e-37)


@pytest.mark.parametrize("ddt,xdt,odt", [("bf16", "bf16", "bf16"), ("f32", "f32", "f32"), ("f32", "bf16", "bf16"),
                                         ("bf16", "f32", "f32")])
@pytest.mark.parametrize("M,K", SHAPES)
def test_layernorm_grad(bl, M, K, ddt, xdt, odt):
    X = _rows(M, K, M + 5 * K, xdt)
    w, b = _affine(K, K + 2)
    _, mean, rstd = bl.bl_layernorm(X.to(DEV), _dev(w), _dev(b))
    dY = torch.from_numpy(np.random.default_rng(K).standard_normal((M, K)).astype(np.float32)).to(ref.KINDS[ddt])
    dX, dw, db = bl.bl_layernorm_grad(dY.to(DEV), X.to(DEV), mean, rstd, _dev(w), out_dtype=ref.KINDS[odt])
    r = rstd.double().cpu().numpy()
    xh = (X.double().numpy() - mean.double().cpu().numpy()[:, None]) * r[:, None]
    _grad_check(dX.double().cpu().numpy(), dw.double().cpu().numpy(), db.double().cpu().numpy(),
                dY.double().numpy(), xh, r, w.astype(np.float64), odt == "bf16", M)
    again = bl.bl_layernorm_grad(dY.to(DEV), X.to(DEV), mean, rstd, _dev(w), out_dtype=ref.KINDS[odt])
    for p, q in zip((dX, dw, db), again):
        assert torch.equal(p, q)   # no order that depends on timing


@pytest.mark.parametrize("ddt,odt", [("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("M,K", SHAPES)
def test_layernorm_grad_q8(bl, M, K, ddt, odt):
    X = _rows(M, K, M + 7 * K, "bf16")
    w, b = _affine(K, K + 3)
    _, _, _, rstd, xq, xs = bl.bl_layernorm_quant(X.to(DEV), _dev(w), _dev(b), checkpoint=True)
    dY = torch.from_numpy(np.random.default_rng(K).standard_normal((M, K)).astype(np.float32)).to(ref.KINDS[ddt])
    dX, dw, db = bl.bl_layernorm_grad_q8(dY.to(DEV), xq, xs, rstd, _dev(w), out_dtype=ref.KINDS[odt])
    xh = (xq.double() * xs.double().repeat_interleave(64, 1)).cpu().numpy()
    _grad_check(dX.double().cpu().numpy(), dw.double().cpu().numpy(), db.double().cpu().numpy(),
                dY.double().numpy(), xh, rstd.double().cpu().numpy(), w.astype(np.float64), odt == "bf16", M)


# Many rows: the shapes that take other units per thread than a few rows do.
MANY = [(297, 704), (300, 2560), (310, 4096), (296, 8256), (300, 11008), (298, 16384), (299, 16448)]


@pytest.mark.parametrize("M,K", MANY)
def test_many_rows(bl, M, K):
    """Rows of a large call against the same rows in small calls (other
    kernels), bit for bit; gradients against the formulas."""
    X = _rows(M, K, K, "bf16")
    w, b = _affine(K, K + 5)
    Xd, wd, bd = X.to(DEV), _dev(w), _dev(b)
    big, mean, rstd = bl.bl_layernorm(Xd, wd, bd)
    tok = bl.bl_layernorm_quant(Xd, wd, bd, checkpoint=True)
    plain = bl.bl_layernorm_quant(Xd, wd, bd)
    assert torch.equal(plain[0], tok[0]) and torch.equal(plain[1], tok[1])
    for r in (0, 1, M // 2, M - 3):
        part = Xd[r:r + 3].contiguous()
        y, m3, r3 = bl.bl_layernorm(part, wd, bd)
        # the order of a row's 64-bit sums is the shape's: far below an fp32 step
        assert torch.equal(m3, mean[r:r + 3]) and torch.equal(r3, rstd[r:r + 3])
        assert torch.equal(y, big[r:r + 3])
        for p, q in zip(bl.bl_layernorm_quant(part, wd, bd, checkpoint=True), tok):
            assert torch.equal(p, q[r:r + 3])
    dY = torch.from_numpy(np.random.default_rng(K).standard_normal((M, K)).astype(np.float32))
    xq, xs = tok[4], tok[5]
    got = bl.bl_layernorm_grad_q8(dY.to(DEV), xq, xs, rstd, wd)
    xh = (xq.double() * xs.double().repeat_interleave(64, 1)).cpu().numpy()
    r = rstd.double().cpu().numpy()
    _grad_check(*(t.double().cpu().numpy() for t in got), dY.double().numpy(), xh, r, w.astype(np.float64), True, M)
    got = bl.bl_layernorm_grad(dY.bfloat16().to(DEV), Xd, mean, rstd, wd, out_dtype=torch.float32)
    xh = (X.double().numpy() - mean.double().cpu().numpy()[:, None]) * r[:, None]
    _grad_check(*(t.double().cpu().numpy() for t in got), dY.bfloat16().double().numpy(), xh, r,
                w.astype(np.float64), False, M)


@pytest.mark.parametrize("M,H", [(300, 704), (296, 11008)])
def test_relu2_many_rows(bl, M, H):
    acc, gx, gu = _acc(M, H, H)
    a, x, u = _dev(acc), _dev(gx), _dev(gu)
    big = bl.bl_relu2_requant_q8(a, x, u)
    none = bl.bl_relu2_requant_q8(a, x, u, checkpoint=False)
    assert none[3] is None and none[4] is None
    for p, q in zip(none[:3], big[:3]):
        assert torch.equal(p, q)
    for r in (0, 2, M - 2):
        part = bl.bl_relu2_requant_q8(a[r:r + 2].contiguous(), x[r:r + 2].clone(), u)
        small = bl.bl_relu2_requant_q8(a[r:r + 2].contiguous(), x[r:r + 2].clone(), u, checkpoint=False)
        for p, q in zip(part, big):
            assert torch.equal(p, q[r:r + 2])
        for p, q in zip(small[:3], big[:3]):
            assert torch.equal(p, q[r:r + 2])


def test_rows_past_two_to_the_31_elements(bl):
    M, K = 528000, 4096
    X = torch.empty((M, K), dtype=torch.bfloat16, device=DEV).normal_()
    w, b = (_dev(t) for t in _affine(K, 8))
    y, mean, rstd = bl.bl_layernorm(X, w, b)
    tail = X[-5:].contiguous()
    assert torch.equal(y[-5:], bl.bl_layernorm(tail, w, b)[0])
    del y
    tok = bl.bl_layernorm_quant(X, w, b, checkpoint=True)
    want = bl.bl_layernorm_quant(tail, w, b, checkpoint=True)
    for p, q in zip(tok, want):
        assert torch.equal(p[-5:], q)
    dX, _, _ = bl.bl_layernorm_grad(X, X, mean, rstd, w)
    assert torch.equal(dX[-5:], bl.bl_layernorm_grad(tail, tail, mean[-5:].clone(), rstd[-5:].clone(), w)[0])


def test_two_calls_at_once(bl):
    """The same calls on two streams at once, each with its own buffers."""
    M, K = 256, 2048
    w, b = (_dev(t) for t in _affine(K, 6))
    X = [_rows(M, K, s, "bf16").to(DEV) for s in (1, 2)]
    dY = [torch.randn(M, K, device=DEV) for _ in X]

    def step(x, dy, stream=None):
        t = bl.bl_layernorm_quant(x, w, b, checkpoint=True, stream=stream)
        return list(t) + list(bl.bl_layernorm_grad_q8(dy, t[4], t[5], t[3], w, stream=stream))

    want = [step(x, dy) for x, dy in zip(X, dY)]
    streams = [torch.cuda.Stream() for _ in X]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i] = step(X[i], dY[i], s)
    torch.cuda.synchronize()
    for g, v in zip(got, want):
        for p, q in zip(g, v):
            assert torch.equal(p, q)


def test_layernorm_grad_against_differences(bl):
    """Directional derivatives of Σ dY·LN(x) in 64 bits against the kernels' gradients."""
    M, K = 6, 320
    rng = np.random.default_rng(0)
    x, dy = (rng.standard_normal((M, K)).astype(np.float32) for _ in range(2))
    w, b = _affine(K, 9)
    X, wd, bd = _dev(x), _dev(w), _dev(b)
    _, mean, rstd = bl.bl_layernorm(X, wd, bd)
    dX, dw, db = (t.double().cpu().numpy() for t in
                  bl.bl_layernorm_grad(_dev(dy), X, mean, rstd, wd, out_dtype=torch.float32))

    def loss(xx, ww, bb):
        return float((dy.astype(np.float64) * ref.layernorm(xx, ww, bb, EPS)[0]).sum())

    h = 1e-5
    for _ in range(4):
        v, vw, vb = rng.standard_normal((M, K)), rng.standard_normal(K), rng.standard_normal(K)
        x64, w64, b64 = (t.astype(np.float64) for t in (x, w, b))
        # central differences: off by h² times third derivatives (of order 10³ here) and 1e-13/h
        for got, up, down in (((dX * v).sum(), loss(x64 + h * v, w64, b64), loss(x64 - h * v, w64, b64)),
                              ((dw * vw).sum(), loss(x64, w64 + h * vw, b64), loss(x64, w64 - h * vw, b64)),
                              ((db * vb).sum(), loss(x64, w64, b64 + h * vb), loss(x64, w64, b64 - h * vb))):
            assert abs(got - (up - down) / (2 * h)) <= 1e-4 * (1 + abs(got))


@pytest.mark.parametrize("M,K", [(4, 64), (4, 2560), (300, 4096), (4, 16448)])
def test_nan_and_infinity(bl, M, K):
    """Rows with a NaN or an infinity give the tokens that bl_quant_acts makes of
    them, a checkpoint that says so, and leave the other rows alone."""
    X = _rows(M, K, M + K, "f32")
    w, b = _affine(K, K)
    clean = bl.bl_layernorm_quant(X.to(DEV), _dev(w), _dev(b), checkpoint=True)
    X[1, K - 1] = float("nan")
    X[2, 3] = float("inf")
    X = X.to(DEV)
    Aq, gA, sums, rstd, xq, xs = bl.bl_layernorm_quant(X, _dev(w), _dev(b), checkpoint=True)
    Y = bl.bl_layernorm(X, _dev(w), _dev(b), out_dtype=torch.float32)[0]
    q, g, qs = bl.bl_quant_acts(Y)[:3]
    assert torch.equal(Aq, q) and torch.equal(gA, g) and torch.equal(sums, qs)
    rest = [m for m in range(M) if m not in (1, 2)]
    for got, want in zip((Aq, gA, sums, rstd, xq, xs), clean):
        assert torch.equal(got[rest], want[rest])
    assert xs[1:3].isnan().all()
    dY = torch.ones(M, K, device=DEV)
    dX, dw, db = bl.bl_layernorm_grad_q8(dY, xq, xs, rstd, _dev(w), out_dtype=torch.float32)
    assert dX[1:3].isnan().all() and dX[rest].isfinite().all()
    assert dw.isnan().all() and torch.equal(db, torch.full_like(db, M))
    # an infinite weight: one column of every row
    w[5] = np.inf
    Aq, gA = bl.bl_layernorm_quant(X, _dev(w), _dev(b))[:2]
    q, g = bl.bl_quant_acts(bl.bl_layernorm(X, _dev(w), _dev(b), out_dtype=torch.float32)[0])[:2]
    assert torch.equal(Aq, q) and torch.equal(gA, g)


@pytest.mark.parametrize("M,H", [(4, 64), (4, 2752), (300, 704), (4, 33024)])
def test_relu2_nan_and_infinity(bl, M, H):
    """Scales of a token that are infinite or NaN: what the requantisation of the
    FFN does with them, by its formulas (a NaN passes no maximum)."""
    acc, gx, gu = _acc(M, H, M + H)
    gx[0], gx[2] = np.inf, np.nan
    Rq, gr, sums, Pq, ps = (t.cpu().numpy() for t in bl.bl_relu2_requant_q8(_dev(acc), _dev(gx), _dev(gu)))
    with np.errstate(all="ignore"):
        h = acc.astype(np.float32) * ((gx * gu[0]) / np.float32(127))[:, None]
        p = np.fmax(h, np.float32(0))
        r = p * p
        top = r.max(1)
        v = np.rint(r * (np.float32(127) / (top + np.float32(1e-5)))[:, None])
    want = np.where(np.isnan(v), -128, v).astype(np.int64)
    np.testing.assert_array_equal(gr, top)
    np.testing.assert_array_equal(Rq, want)
    np.testing.assert_array_equal(sums, want.sum(1))
    inf = np.isinf(p[0])
    assert np.all(Pq[0][inf] == 255) and np.all(np.isinf(ps[0]) == inf.reshape(-1, 64).any(1))
    assert np.all(Pq[2] == 0) and np.all(ps[2] == 0)


def test_layernorm_no_rows(bl):
    K = 128
    w, b = (_dev(t) for t in _affine(K, 1))
    X = torch.empty((0, K), device=DEV)
    Y, mean, rstd = bl.bl_layernorm(X, w, b)
    assert Y.shape == (0, K) and mean.shape == (0,)
    dX, dw, db = bl.bl_layernorm_grad(X, X, mean, rstd, w)
    assert dX.shape == (0, K) and not dw.any() and not db.any()
    assert bl.bl_layernorm_quant(X, w, b, checkpoint=True)[0].shape == (0, K)


# ---------------------------------------------------------------------------


def _acc(M, H, seed):
    rng = np.random.default_rng(seed)
    acc = np.rint(rng.standard_normal((M, H)) * 1600).astype(np.int32)
    if M > 1:
        acc[1] = -np.abs(acc[1])              # nothing passes the ReLU
    acc[0, :64] = np.minimum(acc[0, :64], 0)  # an empty group
    if M > 2:
        acc[2, 5] = 127 * H                   # the largest sum
    return acc, (3 + 2 * rng.random(M)).astype(np.float32), np.array([0.0153], np.float32)


@pytest.mark.parametrize("M,H", [(1, 64), (3, 192), (5, 2752), (4, 11008), (130, 512), (2, 16448)])
def test_relu2_requant_q8(bl, M, H):
    acc, gx, gu = _acc(M, H, M + H)
    Rq, gr, sums, Pq, ps = bl.bl_relu2_requant_q8(_dev(acc), _dev(gx), _dev(gu))
    q, g = oracle.relu2_requant(acc, gx, gu[0], 1e-5)
    np.testing.assert_array_equal(Rq.cpu().numpy(), q)
    np.testing.assert_array_equal(gr.cpu().numpy(), g)
    np.testing.assert_array_equal(sums.cpu().numpy(), q.astype(np.int64).sum(1))
    p = np.maximum(oracle.dequant_f32(acc, gx, gu[0]), np.float32(0))
    codes, scale = ref.checkpoint(p, 255.0)
    np.testing.assert_array_equal(ps.cpu().numpy(), scale)
    np.testing.assert_array_equal(Pq.cpu().numpy(), codes)


@pytest.mark.parametrize("ddt,odt", [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("M,H", [(1, 64), (3, 192), (5, 2752), (130, 512), (9, 11008)])
def test_relu2_grad_q8(bl, M, H, ddt, odt):
    acc, gx, gu = _acc(M, H, M + 2 * H)
    Pq, ps = bl.bl_relu2_requant_q8(_dev(acc), _dev(gx), _dev(gu))[3:]
    dR = torch.from_numpy(np.random.default_rng(H).standard_normal((M, H)).astype(np.float32)).to(ref.KINDS[ddt])
    dH = bl.bl_relu2_grad_q8(dR.to(DEV), Pq, ps, out_dtype=ref.KINDS[odt]).double().cpu().numpy()
    want = 2 * Pq.double().cpu().numpy() * ps.double().repeat_interleave(64, 1).cpu().numpy() * dR.double().numpy()
    tol = 3 * U * np.abs(want)
    tol = tol + (2.0 ** -8 * (np.abs(want) + tol) if odt == "bf16" else 0)
    assert np.all(np.abs(dH - want) <= tol)
    # against the derivative of ReLU² itself: half a step of the checkpoint
    p = np.maximum(acc * (gx.astype(np.float64) * gu[0] / 127)[:, None], 0)
    half = 0.5 * ps.double().repeat_interleave(64, 1).cpu().numpy()
    true = 2 * p * dR.double().numpy()
    assert np.all(np.abs(dH - true) <= 2 * (half * (1 + 255 * 8 * U)) * np.abs(dR.double().numpy())
                  + tol + 8 * U * np.abs(true) + (2.0 ** -8 * np.abs(true) if odt == "bf16" else 0))


def test_side_stream_and_graph(bl):
    """A whole step on a side stream and in a replayed graph, against the plain calls."""
    M, K = 64, 1024
    X, (w, b) = _rows(M, K, 1, "bf16").to(DEV), (_dev(t) for t in _affine(K, 4))
    dY = torch.randn(M, K, device=DEV)

    def step(stream=None):
        Aq, gA, sums, rstd, xq, xs = bl.bl_layernorm_quant(X, w, b, checkpoint=True, stream=stream)
        return (Aq, gA, sums, rstd, xq, xs) + bl.bl_layernorm_grad_q8(dY, xq, xs, rstd, w, stream=stream)

    base = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step(side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for p, q, r in zip(base, other, captured):
        assert torch.equal(p, q) and torch.equal(p, r)
