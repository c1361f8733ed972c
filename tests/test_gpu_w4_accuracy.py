"""bl_linear_w4 where the zero point matters: activations with a mean, codes that
mostly equal their zero point, whole numbers whose product is exact. A term s·(q − z)·x
with q = z is nothing, so results may be off in proportion to the terms that are
there, not to s·z·|x|."""
import numpy as np
import pytest
import torch

import w4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24            # half a step of fp32, relative
FIXED = 1.2016e-7         # half a step of the fixed-point activations: of the largest of 128 columns


@pytest.fixture(scope="module")
def bl():
    import ternary_weight_linear_absmax_b200 as m
    m.load()
    return m


def _packed(bl, codes, s, z, group, zeros):
    nib = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    return bl.bl_pack_w4(torch.from_numpy(nib).to(DEV), torch.from_numpy(s).bfloat16().to(DEV), group,
                         zeros=torch.from_numpy(z.astype(np.uint8)).to(DEV) if zeros else None)


def _run(bl, x, codes, s, z, group, zeros, xdt):
    """(x as its type holds it, weights, the product in 64 bits, what the library makes of it)."""
    W4, sc, zp = _packed(bl, codes, s, z, group, zeros)
    X = torch.from_numpy(x.astype(np.float32)).to(ref.KINDS[xdt])
    got = bl.bl_linear_w4(X.to(DEV), W4, sc, codes.shape[0], zeros=zp, out_dtype=torch.float32)
    x = X.double().numpy()
    w = ref.dequant(codes, s, z, group)
    return x, w, x @ w.T, got.double().cpu().numpy()


def _scales(rng, N, G):
    return ref.bf16(rng.uniform(0.002, 0.01, (N, G)).astype(np.float32))


def _activations(rng, kind, M, K):
    x = rng.standard_normal((M, K))
    return {"normal": x, "rectified": np.maximum(x, 0), "mean 1": x + 1, "mean 30": x + 30}[kind]


def _blocks(a, size):
    """[rows, K] → [rows, ceil(K/size), size], zeros behind column K."""
    pad = -a.shape[1] % size
    return np.pad(a, ((0, 0), (0, pad))).reshape(a.shape[0], -1, size)


FORMS = [(1, "bf16"), (2, "f32"), (3, "bf16"), (4, "f32"), (5, "bf16"), (5, "f32"),     # digits, packed columns
         (7, "f32"), (16, "f32"), (20, "f32"),                                          # digits of a launch
         (6, "bf16"), (16, "bf16")]                                                     # bf16 as it is


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,xdt", FORMS)
@pytest.mark.parametrize("N,K,group", [(40, 64, 32), (300, 4096, 128), (33, 11008, 64), (2400, 512, 32)])
def test_codes_at_their_zero_point_give_zero(bl, M, xdt, N, K, group, zeros):
    rng = np.random.default_rng(M + K)
    z = rng.integers(0, 16, (N, -(-K // group))) if zeros else np.full((N, -(-K // group)), 8)
    codes = np.repeat(z, group, 1)[:, :K]
    x = _activations(rng, "mean 30", M, K)
    *_, got = _run(bl, x, codes, _scales(rng, N, z.shape[1]), z, group, zeros, xdt)
    assert np.all(got == 0.0), np.abs(got).max()


@pytest.mark.parametrize("M,xdt", FORMS[:9])
@pytest.mark.parametrize("N,K,group,kind", [(100, 4096, 128, "rectified"), (33, 11008, 128, "mean 1"),
                                            (64, 2560, 32, "mean 30"), (16, 65536, 64, "mean 1"),
                                            (40, 1088, 64, "normal")])
def test_one_code_per_group(bl, M, xdt, N, K, group, kind):
    """One code per group differs from its zero point. A result passes through one
    rounding per group (ceil(K/group) of them), at most 16 shares of three
    digits, 8 CTAs, and a few when a group's digits are joined; each is of at most half a
    step of the sum of magnitudes S. To that comes the fixed point of the activations."""
    rng = np.random.default_rng(K + M)
    G = -(-K // group)
    z = rng.integers(0, 16, (N, G))
    codes = np.repeat(z, group, 1)[:, :K]
    first = np.arange(G) * group
    width = np.minimum(group, K - first)
    at = first + (rng.random((N, G)) * width).astype(int)
    codes[np.arange(N)[:, None], at] = rng.integers(0, 16, (N, G))
    x, w, want, got = _run(bl, _activations(rng, kind, M, K), codes, _scales(rng, N, G), z, group, True, xdt)
    fixed = FIXED * _blocks(np.abs(x), 128).max(2) @ _blocks(np.abs(w), 128).sum(2).T
    tol = (G + 64) * U * (np.abs(x) @ np.abs(w).T) + fixed
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("M,xdt", FORMS[:9])
@pytest.mark.parametrize("N,K,group,zeros,kind", [
    (64, 4096, 32, False, "rectified"), (64, 11008, 128, True, "rectified"), (48, 16384, 32, True, "mean 1"),
    (32, 65536, 64, False, "mean 1"), (500, 2560, 128, False, "normal"), (4000, 512, 64, True, "mean 30")])
def test_error_over_many_results(bl, M, xdt, N, K, group, zeros, kind):
    """Root mean square over all results. Roundings are independent and each is
    off by at most U of what it rounds, U/√3 in the root mean square: one per group
    on a partial sum (at most P, the largest partial sum from the row's
    start), three on the group's own sum g, and FIXED/√3 of the block's largest
    value per activation. Twice the root of their squares' sum."""
    rng = np.random.default_rng(K + N + M)
    G = -(-K // group)
    codes = rng.integers(0, 16, (N, K))
    z = rng.integers(0, 16, (N, G)) if zeros else np.full((N, G), 8)
    x, w, want, got = _run(bl, _activations(rng, kind, M, K), codes, _scales(rng, N, G), z, group, zeros, xdt)
    g = np.einsum("mgk,ngk->mng", _blocks(x, group), _blocks(w, group), optimize=True)
    P = np.abs(np.cumsum(g, 2)).max(2)
    fixed = (_blocks(np.abs(x), 128).max(2) ** 2) @ (_blocks(w, 128) ** 2).sum(2).T
    var = (U ** 2 * (G * P ** 2 + 3 * (g ** 2).sum(2)) + FIXED ** 2 * fixed) / 3
    assert np.sqrt(((got - want) ** 2).mean()) <= 2 * np.sqrt(var.mean()), np.sqrt(((got - want) ** 2).mean() / var.mean())


@pytest.mark.parametrize("M,xdt", FORMS)
@pytest.mark.parametrize("N,K,group", [(33, 64, 32), (200, 704, 64), (100, 4096, 128), (20, 32768, 64)])
def test_whole_numbers_exact(bl, M, xdt, N, K, group):
    """Whole activations of up to 127·2^5, one of 2^18 per block whose weight is 0,
    eight weights per row that are not, scales 1/4 to 2: all terms and their
    partial sums are multiples of 1/4 below 2^24 quarters (8·4064·15·2·4 < 2^22),
    and so are their digits' (an activation is a multiple of the fixed-point step
    at 2^18, 2^-4), so the result is the exact one."""
    rng = np.random.default_rng(M + N)
    G = -(-K // group)
    z = rng.integers(0, 16, (N, G))
    codes = np.repeat(z, group, 1)[:, :K]
    for n in range(N):
        at = 1 + rng.choice(K - 1, 8, replace=False)
        codes[n, at[at % 128 != 0]] = rng.integers(0, 16, (at % 128 != 0).sum())
    s = 2.0 ** rng.integers(-2, 2, (N, G))
    x = rng.integers(-127, 128, (M, K)) * 2 ** rng.integers(0, 6, (M, K))
    x[:, ::128] = 2 ** 18
    *_, want, got = _run(bl, x, codes, s.astype(np.float32), z, group, True, xdt)
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("M", [1, 2, 5, 9])
def test_large_values_do_not_overflow_on_the_way(bl, M):
    """Activations near fp32's largest value whose weights are 0 but for one per
    row: nothing on the way to a finite result may be infinite. One term, its
    fixed-point rounding and two additions of its digits."""
    N, K, group = 48, 256, 64
    rng = np.random.default_rng(M)
    z = np.full((N, K // group), 15)
    codes = np.repeat(z, group, 1)
    codes[:, 3] = 14
    s = np.full((N, K // group), 0.5, np.float32)
    x = np.full((M, K), 3.0e38)
    _, _, want, got = _run(bl, x, codes, s, z, group, True, "f32")
    assert np.all(np.abs(got - want) <= (FIXED + 4 * U) * np.abs(want))
