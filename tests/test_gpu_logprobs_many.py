"""GPU parity of log probabilities on both sides of the number of rows that chooses the second kernel: few distinct rows,
repeated, against fp64."""
import numpy as np
import pytest

from oracle import rows as oracle
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


def _check(nv, x, tokens, ks, bf16, rows, scale=1.0, pad=0, skip=0):
    """Every term of S is off by 2^-23 (the exponential) and by |z - max| 2^-23 (its argument), 24 additions in fp32 by 2^-24
    each, and a unit's reference taken back by 3 2^-24: eps = (29 + 2 E) 2^-24 of S, E the mean of |z - max|.  So is a log
    probability, with its own rounding; and the entropy's mean, E, by eps E, by E2 2^-23 (E2 the mean square) and by eps E
    once more for its division by S."""
    import torch
    kinds, V = x.shape
    most = max(ks)
    y, H, top, top_lp, _, E, E2 = oracle.logprobs(x, tokens, most, scale)
    eps = (29 + 2 * E) * 2.0 ** -24
    put = lambda v: torch.from_numpy(np.array(v)).cuda()  # noqa: E731
    at = torch.arange(rows, device="cuda") % kinds
    base = put(x.astype(np.float32)).to(torch.bfloat16 if bf16 else torch.float32)
    buf = torch.full((skip + rows * (V + pad),), 1e30, dtype=base.dtype, device="cuda")
    logits = buf[skip:].view(rows, V + pad)[:, :V]
    logits.copy_(base[at])
    asked = put(np.asarray(tokens, np.int32))[at]

    def near(got, want, tol, name):
        want, tol, got = put(want)[at], put(np.broadcast_to(tol, want.shape))[at], got.double()
        inf = want.isneginf()
        assert torch.equal(got.isneginf(), inf), name
        bad = ~inf & ~((got - want).abs() <= tol + 2.0 ** -24 * want.abs())
        assert not bad.any(), (name, bad.nonzero()[:3].tolist(), got[bad][:3], want[bad][:3])
    for k in ks:
        what = (rows, V, bf16, k)
        lp, entropy, token, best = nv.logprobs(logits, asked, k=k, scale=scale)
        near(lp, y, eps[:, None], what + ("logprob",))
        near(entropy, H, eps * (1 + 2 * E) + 2.0 ** -23 * E2, what + ("entropy",))
        if k:
            want = put(top[:, :k].astype(np.int32))[at]
            assert torch.equal(token, want), what + ((token != want).nonzero()[:3].tolist(),)
            near(best, top_lp[:, :k], eps[:, None], what + ("top",))


def _kinds(V, bf16):
    """Ordinary rows, a masked third, few distinct values, all alike, rising and falling, masked but for three, masked whole, a
    peak of neighbours, and a group of 512 in 64 without any of the large ones."""
    rng = np.random.default_rng(V)
    n = np.arange(V, dtype=np.float64)
    third = 3 * rng.standard_normal(V)
    third[:V // 3] = -np.inf
    few = np.full(V, -np.inf)
    few[rng.choice(V, 3, replace=False)] = [1.0, 2.0, 2.0]
    peak = np.full(V, -5.0)
    peak[V // 2:V // 2 + 70] = np.arange(70) / 8
    low = rng.standard_normal(V)
    low[np.arange(V) // 512 % 64 == 5] = -10.0
    x = np.stack([3 * rng.standard_normal(V), 3 * rng.standard_normal(V), third, rng.integers(0, 3, V), np.full(V, 2.5), n / 65536, -n / 65536, few,
                  np.full(V, -np.inf), peak, low])
    return oracle.to_type(x, "bf16" if bf16 else "f32"), rng.integers(0, V, (len(x), 3))


@pytest.mark.parametrize("V", [5003, 99991, 152064, 300001])
@pytest.mark.parametrize("bf16", [False, True])
def test_both_sides_of_the_rule(nv, V, bf16):
    x, tokens = _kinds(V, bf16)
    for rows in (256, 257):
        _check(nv, x, tokens, (0, 1, 8, 20, 64), bf16, rows)


@pytest.mark.parametrize("rows", [3, 256, 257, 300])
def test_rows_off_16_bytes(nv, rows):
    for bf16 in (False, True):
        x, tokens = _kinds(50021, bf16)
        _check(nv, x, tokens, (0, 5, 64), bf16, rows, 0.7, 3, 1)
        _check(nv, x, tokens, (13,), bf16, rows, 1.25, 1, 0)


@pytest.mark.parametrize("rows", [2, 257])
@pytest.mark.parametrize("bf16", [False, True])
def test_more_groups_than_a_list_holds(nv, rows, bf16):
    """Of 64 sets of groups all but one have many of the best: over 1024 groups pass the bar of k = 64."""
    V = 700001
    rng = np.random.default_rng(9)
    x = rng.standard_normal((2, V))
    x[:, np.arange(V) // 512 % 64 == 5] = -10.0
    x = oracle.to_type(x, "bf16" if bf16 else "f32")
    _check(nv, x, rng.integers(0, V, (2, 2)), (64, 63, 1), bf16, rows)


def test_many_tokens_of_many_rows(nv):
    """More given tokens than the second kernel has threads, some outside the vocabulary."""
    x, _ = _kinds(3001, False)
    tokens = np.random.default_rng(2).integers(-2, 3004, (len(x), 1024))
    for rows in (256, 257):
        _check(nv, x, tokens, (0, 4), False, rows)
