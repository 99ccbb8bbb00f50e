"""Beam selection at the ends of its range: logits of large magnitude (masks of a type's lowest
value among them), against the fp64 oracle."""
import numpy as np
import pytest

from oracle import cache as oc
from tests.gpu_util import dev, host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


def _check(nv, x, beams, score, k):
    """Every listed score within its bound of the oracle's for that candidate, none of the others above
    the last one by more than both bounds.

    x - max is rounded once (2^-24 of it); the log-sum is off by at most 2^-21 of 20, the most that a
    log of 2^28 terms can be; so are the two last sums of what they add: 2^-21 (|x - max| + |c| + 20)."""
    import torch
    score = np.asarray(score, np.float32)
    got = nv.beam_select(x, beams, dev(score), k)
    torch.cuda.synchronize()
    s, parent, token = (host(g) for g in got[:3])
    vals = x.double().cpu().numpy()
    exact = oc.beam_scores(vals, score.astype(np.float64), None, -1)
    tol = 2.0 ** -21 * (vals.max(1, keepdims=True) - vals + np.abs(score[:, None]) + 20)
    batch, V = len(vals) // beams, vals.shape[1]
    assert np.isfinite(s).all()
    assert ((token >= 0) & (token < V)).all() and (parent // beams == np.arange(batch)[:, None]).all()
    for b in range(batch):
        flat = (parent[b] - b * beams).astype(np.int64) * V + token[b]
        e, t = (a[b * beams:(b + 1) * beams].ravel().copy() for a in (exact, tol))
        assert len(set(flat)) == k and (s[b][:-1] >= s[b][1:]).all()
        assert (np.abs(e[flat] - s[b]) <= t[flat]).all(), (s[b], e[flat])
        low = s[b][-1] + t[flat].max()
        e[flat] = -np.inf
        assert (e - t <= low).all(), (e.max(), low)
    return s, parent, token


def _lowest(dtype):
    import torch
    return torch.finfo(dtype).min


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("value", [-65504.0, -3e9, -1e10, -1e12, -1e30, "lowest"])
def test_blocks_masked_with_a_large_number(nv, dtype, value):
    """Whole blocks of the vocabulary at one large negative number, parts of others, a whole row."""
    import torch
    dtype = getattr(torch, dtype)
    value = _lowest(dtype) if value == "lowest" else value
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (4 * torch.randn((8, 6000), generator=g, device="cuda")).to(dtype)
    x[:, 1024:3072] = value
    x[1, :5000] = value
    x[2, torch.rand(6000, generator=g, device="cuda") < 0.4] = value
    x[5] = value  # everything masked: an even spread
    _, parent, token = _check(nv, x, 4, [-1.0, -2.0, -0.5, -3.0, -1.0, 0.0, -2.5, -40.0], 12)
    for p, t in zip(parent.ravel(), token.ravel()):
        assert p == 5 or float(x[p, t]) > -100


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("size", [1e5, 1e10, 1e30, 3e38])
def test_large_logits(nv, dtype, size):
    """Rows around a large number, both signs in one row, and ordinary rows beside them."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(4)
    x = (4 * torch.randn((6, 3500), generator=g, device="cuda"))
    unit = size * 2.0 ** -7  # bf16's step there
    x[0] = size - unit * torch.randint(0, 4, (3500,), generator=g, device="cuda")
    x[1] = -size + unit * torch.randint(0, 4, (3500,), generator=g, device="cuda")
    x[3, ::7] = -size
    x[3, 77] = size / 4
    _check(nv, x.to(getattr(torch, dtype)), 2, [0.0, -1.0, -2.0, 0.0, -3.0, -1.5], 8)


@pytest.mark.parametrize("dtype,V", [("bfloat16", 2 ** 31 - 1032), ("bfloat16", 2 ** 31 - 1025), ("float32", 2 ** 31 - 1028)])
def test_largest_vocabulary(nv, dtype, V):
    """Token numbers up to the documented limit, rows read in vectors and by element.  The sum of 2^21
    groups' sums takes 2^15 additions a lane: off by at most (2^15 + 64) 2^-24 of it."""
    import torch
    x = torch.zeros((1, V), dtype=getattr(torch, dtype), device="cuda")
    x[0, V - 1], x[0, 5], x[0, V - 1000], x[0, 1 << 30] = 8.0, 7.0, 6.0, 5.0
    s, parent, token, _ = (host(t) for t in nv.beam_select(x, 1, dev(np.zeros(1, np.float32)), 6))
    assert token[0].tolist() == [V - 1, 5, V - 1000, 1 << 30, 0, 1] and not parent.any()
    v = np.array([8.0, 7.0, 6.0, 5.0, 0.0, 0.0])
    want = v - np.log(V - 4 + np.exp(v[:4]).sum())
    assert (np.abs(s[0] - want) <= (2 ** 15 + 64) * 2.0 ** -24 + 2.0 ** -21 * 42).all(), (s, want)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_more_groups_than_are_ranked_at_once(nv, dtype):
    """64 rows of 128 blocks, the same two far below the others in each row: the bar that the k-th best of 64
    shares of the blocks sets is theirs, and nearly all 8192 blocks pass it."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((64, 131072), generator=g, device="cuda")
    x[:, 9 * 1024:10 * 1024] -= 50
    x[:, (9 + 64) * 1024:(10 + 64) * 1024] -= 50
    s, parent, token = _check(nv, x.to(getattr(torch, dtype)), 64, -3 * np.random.default_rng(1).random(64), 64)
    flat = parent[0].astype(np.int64) * 131072 + token[0]
    assert (flat[:-1] < flat[1:])[s[0][:-1] == s[0][1:]].all()
