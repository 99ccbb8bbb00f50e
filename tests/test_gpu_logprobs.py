"""GPU parity of log probabilities: tokens exactly, values against fp64."""
import numpy as np
import pytest

from oracle import rows as oracle
from tests.gpu_util import dev, host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


def _dev(x, bf16, ld, skip):
    import torch
    t = torch.full((skip + x.shape[0] * ld,), 1e30, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    v = t[skip:skip + x.shape[0] * ld].view(x.shape[0], ld)[:, :x.shape[1]]
    v.copy_(torch.from_numpy(x.astype(np.float32)))
    return v


def _check(nv, x, tokens, k, scale, bf16, pad=0, skip=0, what=""):
    """Every term of S is off by 2^-23 (the exponential) and by |z - max| 2^-23 (its argument: a product
    and a rounded constant), and 24 additions in fp32 by 2^-24 each; taking a unit's reference back is
    another exponential and product, 3 2^-24: eps = (29 + 2 E) 2^-24 of S, E the mean of |z - max|.  So is a log probability, with its own rounding; and the entropy's mean, E, by eps E,
    by E2 2^-23 (E2 the mean square) and by eps E once more for its division by S."""
    import torch
    rows, V = x.shape
    y, H, top, top_lp, lp, E, E2 = oracle.logprobs(x, tokens, k, scale)
    got = nv.logprobs(_dev(x, bf16, V + pad, skip), dev(np.asarray(tokens, np.int32)), k=k, scale=scale)
    torch.cuda.synchronize()
    if k == 0:
        assert got[2] is None and got[3] is None
        got = got[:2] + (torch.zeros((rows, 0)),) * 2
    glp, gH, gtop, gtop_lp = (host(t).astype(np.float64) for t in got)
    assert np.array_equal(gtop, top), (what, np.argwhere(gtop != top)[:3], gtop[gtop != top][:3], top[gtop != top][:3])
    eps = (29 + 2 * E) * 2.0 ** -24

    def near(a, b, tol, name):
        b = np.where(b < -3.4028235677973366e38, -np.inf, b)  # rounds to -inf: half a step past the largest fp32
        inf = np.isneginf(b)
        assert np.array_equal(np.isneginf(a), inf), (what, name)
        a, b = np.where(inf, 0, a), np.where(inf, 0, b)
        bad = ~((np.abs(a - b) <= tol + 2.0 ** -24 * np.abs(b)) | (np.isnan(a) & np.isnan(b)))
        assert not bad.any(), (what, name, np.argwhere(bad)[:3], a[bad][:3], b[bad][:3])
    near(glp.reshape(rows, -1), y, eps[:, None], "logprob")
    near(gtop_lp, top_lp, eps[:, None], "top")
    near(gH, H, eps * (1 + 2 * E) + 2.0 ** -23 * E2, "entropy")


SIZES = [1, 2, 3, 7, 8, 9, 31, 505, 511, 512, 513, 1000, 4089, 4095, 4096, 4097, 4104, 8191, 20000, 99991, 152064]


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("bf16", [False, True])
def test_sizes(nv, V, bf16):
    rng = np.random.default_rng(V)
    for rows, pad, skip, k, n, scale in ((3, 0, 0, min(V, 20), 1, 1.0), (5, 3, 1, min(V, 64), 3, 0.7), (2, 8, 3, 0, 8, 1.25), (4, 1, 0, 1, 0, 2.0)):
        x = oracle.to_type(rng.standard_normal((rows, V)) * 4, "bf16" if bf16 else "f32")
        _check(nv, x, rng.integers(0, V, (rows, n)), k, scale, bf16, pad, skip, (V, bf16, rows, k))


@pytest.mark.parametrize("k", [1, 2, 5, 20, 63, 64])
@pytest.mark.parametrize("V", [64, 600, 5000, 152064])
def test_ties_and_orders(nv, V, k):
    """Few distinct values, all alike, both zeros, rising and falling rows, masked rows, a peak of neighbours."""
    rng = np.random.default_rng(V + k)
    n = np.arange(V, dtype=np.float64)
    masked = np.full(V, -np.inf)
    masked[rng.choice(V, 3, replace=False)] = [1.0, 2.0, 2.0]
    zeros = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    peak = np.full(V, -5.0)
    peak[V // 2:V // 2 + 70] = np.arange(len(peak[V // 2:V // 2 + 70])) / 8
    third = rng.standard_normal(V)
    third[:V // 3] = -np.inf
    x = np.stack([rng.integers(0, 3, V), np.full(V, 2.5), zeros, n / 1024, -n / 1024, masked, np.full(V, -np.inf), peak, third])
    for bf16 in (False, True):
        y = oracle.to_type(x, "bf16" if bf16 else "f32")
        _check(nv, y, rng.integers(0, V, (len(x), 2)), k, 1.0, bf16, 1, 1, (V, k, bf16))


def test_tokens_outside_the_vocabulary(nv):
    x = np.random.default_rng(1).standard_normal((3, 1000))
    x = oracle.to_type(x, "f32")
    _check(nv, x, [[-1, 5], [1000, 2 ** 31 - 1], [-2 ** 31, 999]], 3, 1.0, False)


def test_large_logits(nv):
    """Magnitudes up to the type's largest, and rows where some pass it: differences are rounded before they
    are scaled."""
    rng = np.random.default_rng(2)
    for mid, spread in ((1e4, 3.0), (-3e5, 1.0), (0.0, 1e30), (1e38, 1e38), (-2e38, 1e38)):
        x = oracle.to_type(mid + spread * rng.standard_normal((3, 3000)), "f32")
        _check(nv, x, rng.integers(0, 3000, (3, 4)), 10, 1.0, False, what=(mid, spread))


def test_nan_and_infinity_stay_in_their_row(nv):
    import torch
    x = torch.randn((6, 5000), device="cuda")
    x[1, 77], x[3, 4999], x[4, 0] = float("nan"), float("inf"), float("-inf")
    x[5] = float("nan")
    clean = x.clone()
    clean[1, 77] = clean[3, 4999] = 0
    clean[5] = 0
    tokens = torch.tensor([3, 4, 5, 6, 7, 8], dtype=torch.int32, device="cuda")
    want, got = nv.logprobs(clean, tokens, k=9), nv.logprobs(x, tokens, k=9)
    for w, g in zip(want, got):
        for r in (0, 2, 4):
            assert torch.equal(w[r], g[r])
    for r in (1, 3, 5):
        assert torch.isnan(got[0][r]) and torch.isnan(got[1][r])
    assert ((got[2] >= 0) & (got[2] < 5000)).all()


def test_wide_rows(nv):
    """Over half a million logits: more groups than one list ranks."""
    rng = np.random.default_rng(3)
    V = 2_000_003
    x = np.stack([rng.standard_normal(V), np.zeros(V), np.arange(V) / 65536.0])
    _check(nv, oracle.to_type(x, "f32"), rng.integers(0, V, (3, 2)), 64, 1.0, False)
    _check(nv, oracle.to_type(x, "bf16"), rng.integers(0, V, (3, 2)), 5, 1.0, True, 1, 1)


def test_scales_at_the_ends_of_their_range(nv):
    """From the smallest fp32 to the largest: the best logits (several alike) against all others, and nearly
    uniform rows with masked places."""
    rng = np.random.default_rng(4)
    apart = 2.0 * rng.integers(-2, 3, (4, 5000))
    for scale in (1e18, 1e25, 3.4e38):
        _check(nv, apart, rng.integers(0, 5000, (4, 3)), 12, scale, False, what=scale)
    for scale, spread in ((1e-45, 1e38), (1e-40, 1e36), (2.0 ** -70, 2.0 ** 58)):
        x = spread * rng.standard_normal((4, 5000))
        x[:, ::7] = -np.inf
        _check(nv, oracle.to_type(x, "f32"), rng.integers(0, 5000, (4, 3)), 12, scale, False, what=scale)
