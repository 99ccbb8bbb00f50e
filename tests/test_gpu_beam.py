"""GPU parity of beam selection over beams and vocabulary, against the fp64 oracle."""
import numpy as np
import pytest

from oracle import cache as oc
from tests.gpu_util import dev, host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


def _check(nv, x, beams, score, k, done=None, eos=-1, what=""):
    """Scores within their bound of the oracle's; the choice right wherever exact scores differ by
    more than two bounds; equal exact scores (identical arithmetic) by row, then token."""
    import torch
    t = dev(x) if isinstance(x, np.ndarray) else x
    vals = t.float().cpu().numpy().astype(np.float64)
    got = nv.beam_select(t, beams, dev(score.astype(np.float32)), k, done=None if done is None else dev(done), eos=eos)
    torch.cuda.synchronize()
    s, parent, token, ended = (host(g) for g in got)
    exact = oc.beam_scores(vals, score.astype(np.float32).astype(np.float64), done, eos)
    batch, V = len(vals) // beams, vals.shape[1]
    want, _, _ = oc.beam_select(exact, batch, beams, k)
    # x - max, the log-sum (64 partial sums of exponentials, each off by 2^-22), and the two sums
    finite = np.where(np.isfinite(vals), np.abs(vals), 0).max() + np.where(np.isfinite(score), np.abs(score), 0).max() + 20
    tol = 2.0 ** -21 * finite
    assert np.array_equal(np.isneginf(s), np.isneginf(want)), what
    f = np.isfinite(want)
    assert (np.abs(s - want)[f] <= tol).all(), what
    assert ((token >= 0) & (token < V)).all()
    assert (parent // beams == np.arange(batch)[:, None]).all()
    flat = (parent % beams).astype(np.int64) * V + token
    for b in range(batch):
        assert len(set(flat[b])) == k, what
        e = exact[b * beams:(b + 1) * beams].ravel()
        mine = e[flat[b]]
        assert (np.abs(mine - s[b])[f[b]] <= tol).all() and np.isneginf(mine[~f[b]]).all(), what
        assert (s[b][:-1] >= s[b][1:]).all(), what
        tie = s[b][:-1] == s[b][1:]
        assert (flat[b][:-1] < flat[b][1:])[tie].all(), what
        e = e.copy()
        e[flat[b]] = -np.inf
        if f[b].all():
            assert e.max() <= mine.min() + 2 * tol, what
        else:
            assert np.isneginf(e).all(), what
            rest = flat[b][~f[b]]  # -inf candidates: the lowest
            other = np.setdiff1d(np.arange(beams * V), flat[b][f[b]])[:len(rest)]
            assert np.array_equal(rest, other), what
    full = np.zeros(len(vals), bool) if done is None else done.astype(bool)
    assert np.array_equal(ended.astype(bool), full[parent] | (token == eos)), what
    return s, parent, token


@pytest.mark.parametrize("batch,beams,V,k", [(1, 1, 1, 1), (1, 1, 5, 5), (2, 3, 1000, 6), (1, 4, 1024, 8), (3, 2, 1025, 4),
                                             (1, 8, 32003, 16), (4, 4, 152064, 8), (1, 64, 5000, 64), (2, 16, 70001, 32), (1, 1, 300000, 64)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_beam_select(nv, batch, beams, V, k, dtype):
    import torch
    rng = np.random.default_rng(V + k)
    x = torch.from_numpy((rng.standard_normal((batch * beams, V)) * 4).astype(np.float32)).cuda()
    if dtype == "bf16":
        x = x.to(torch.bfloat16)
    _check(nv, x, beams, -5 * rng.random(batch * beams), k, what="%d x %d x %d, k %d, %s" % (batch, beams, V, k, dtype))


@pytest.mark.parametrize("V,k", [(3000, 8), (20000, 64)])
def test_ties(nv, V, k):
    """Few distinct logits, identical rows: equal scores go by row, then token."""
    rng = np.random.default_rng(V)
    row = rng.integers(0, 3, V).astype(np.float32)
    s, parent, token = _check(nv, np.stack([row] * 4), 4, np.zeros(4), k)
    top = np.flatnonzero(row == 2)[:k]
    assert (parent == 0).all() and np.array_equal(token[0], top)
    s, parent, token = _check(nv, np.zeros((2, V), np.float32), 2, np.zeros(2), k)
    assert np.array_equal(token[0], np.arange(k))
    # rows that differ by their score alone
    s, parent, token = _check(nv, np.stack([row] * 3), 3, np.array([-3.0, 0.0, -3.0]), k)
    assert (parent == 1).all()


def test_finished_dead_and_masked(nv):
    """Finished rows offer their end token alone, rows at -inf nothing, masked logits nothing."""
    rng = np.random.default_rng(4)
    V = 2500
    x = rng.standard_normal((8, V)).astype(np.float32)
    x[0, 5:] = -np.inf
    x[1] = -np.inf
    x[2, rng.random(V) < 0.9] = -np.inf
    done = np.array([0, 0, 0, 1, 0, 1, 1, 1], np.uint8)
    score = np.array([-1.0, -0.5, -9.0, -2.0, -np.inf, -3.0, -np.inf, 0.0])
    _check(nv, x, 4, score, 12, done=done, eos=7)
    _check(nv, x, 8, score, 16, done=done, eos=2499)
    _check(nv, x[4:], 4, score[4:], 6, done=done[4:], eos=0)  # fewer candidates than k
    _check(nv, x[:1], 1, np.array([-np.inf]), 9)
    # the first step of a search: one live beam
    s, parent, _ = _check(nv, x[2:6], 4, np.array([0.0, -np.inf, -np.inf, -np.inf]), 8)
    assert (parent == 0).all()


@pytest.mark.parametrize("dtype,cut", [("f32", 1), ("f32", 4), ("bf16", 3), ("bf16", 8)])
def test_strided_and_unaligned_rows(nv, dtype, cut):
    """Rows inside wider ones, starting off 16 bytes; what lies past V is never taken."""
    import torch
    rng = np.random.default_rng(cut)
    V = 3001
    wide = torch.full((6, V + 2 * cut + 11), float("nan"), device="cuda")
    wide[:, cut:cut + V] = torch.from_numpy(rng.standard_normal((6, V)).astype(np.float32)).cuda()
    if dtype == "bf16":
        wide = wide.to(torch.bfloat16)
    _check(nv, wide[:, cut:cut + V], 3, -rng.random(6), 7)


def test_repeats_and_graph(nv):
    import torch
    x = torch.randn((8, 40000), device="cuda")
    score = torch.zeros(8, device="cuda")
    first = nv.beam_select(x, 4, score, 8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = nv.beam_select(x, 4, score, 8)
    for i in range(3):
        x.copy_(torch.randn((8, 40000), device="cuda")) if i else None
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = nv.beam_select(x, 4, score, 8)
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
        if i == 0:
            assert all(torch.equal(a, b) for a, b in zip(out, first))
