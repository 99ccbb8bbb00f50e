"""Pins of the paged-cache oracle: closed forms, hand-worked cases and invariants (CPU)."""
import numpy as np
import pytest

from oracle import cache as oc


def _cache(rng, layers, pages, heads, page, dim):
    return rng.standard_normal((layers, pages, heads, page, dim)), rng.standard_normal((layers, pages, heads, page // 16, dim, 16))


def test_layout_of_a_token():
    k, v = np.arange(2 * 3 * 2 * 32 * 4.0).reshape(2, 3, 2, 32, 4), np.arange(2 * 3 * 2 * 32 * 4.0).reshape(2, 3, 2, 2, 4, 16)
    table = [2, 0]
    t = 32 + 21  # page 0, token 21: block 1, place 5
    assert np.array_equal(oc.k_token(k, 1, table, t), k[1, 0, :, 21])
    assert np.array_equal(oc.v_token(v, 1, table, t), v[1, 0, :, 1, :, 5])


def test_rotation_closed_forms():
    x = np.zeros((1, 1, 8))
    x[0, 0, 0], x[0, 0, 1] = 3.0, 5.0
    quarter = np.array([np.pi / 2, 0.0])
    y = oc.rotate(x, np.array([[1]]), quarter)  # pairs (0, 2), (1, 3)
    assert np.allclose(y[0, 0], [0, 5, 3, 0, 0, 0, 0, 0])
    y = oc.rotate(x, np.array([[1]]), quarter, interleaved=True)  # pairs (0, 1), (2, 3)
    assert np.allclose(y[0, 0], [-5, 3, 0, 0, 0, 0, 0, 0])
    y = oc.rotate(x, np.array([[9, 1]]), quarter, axis=[1, 0], factor=2.0)
    assert np.allclose(y[0, 0], [0, 10, 6, 0, 0, 0, 0, 0])


def test_rotation_keeps_lengths_and_differences():
    rng = np.random.default_rng(0)
    x, inv = rng.standard_normal((2, 1, 16)), 1e4 ** (-np.arange(8) / 8)
    for inter in (False, True):
        a = oc.rotate(x, np.array([[7], [12]]), inv, interleaved=inter)
        b = oc.rotate(x, np.array([[107], [112]]), inv, interleaved=inter)
        assert np.allclose((a ** 2).sum(2), (x ** 2).sum(2))
        assert np.isclose((a[0] * a[1]).sum(), (b[0] * b[1]).sum())


def test_attention_closed_forms():
    """Equal scores give the mean of what is seen; one token gives its value; none gives zero."""
    rng = np.random.default_rng(1)
    k, v = _cache(rng, 1, 3, 2, 16, 8)
    q = np.zeros((3, 4 * 8))
    start, ctx, table = [0, 3], [18], np.array([[2, 0, -1]])
    mask = [1, 0b10, 0b101]
    out, lse, _, _ = oc.tree_attention(q, k, v, 0, start, ctx, table, mask, 0.3, 4)
    tok = [oc.v_token(v, 0, table[0], t) for t in range(21)]
    for r, seen in enumerate(([18], [19], [18, 20])):
        want = np.mean([tok[t] for t in list(range(18)) + seen], 0)
        assert np.allclose(out[r], np.repeat(want, 2, 0))
        assert np.allclose(lse[r], np.log(18 + len(seen)))
    out, lse, _, _ = oc.tree_attention(q[:2], k, v, 0, [0, 2], [0], table, [2, 0], 0.3, 4)
    assert np.allclose(out[0], np.repeat(tok[1], 2, 0)) and (out[1] == 0).all() and np.isneginf(lse[1]).all()


def test_attention_against_a_direct_sum():
    rng = np.random.default_rng(2)
    k, v = _cache(rng, 2, 4, 1, 16, 4)
    q = rng.standard_normal((1, 4))
    table = np.array([[3, 1]])
    out, lse, absum, _ = oc.tree_attention(q, k, v, 1, [0, 1], [20], table, [1], 0.5, 1)
    num, den, mag = 0, 0, 0
    for t in range(21):
        w = np.exp(0.5 * oc.k_token(k, 1, table[0], t)[0] @ q[0])
        vt = oc.v_token(v, 1, table[0], t)[0]
        num, den, mag = num + w * vt, den + w, mag + w * np.abs(vt)
    assert np.allclose(out[0, 0], num / den) and np.isclose(lse[0, 0], np.log(den)) and np.allclose(absum[0, 0], mag / den)


def test_append_then_compact_by_hand():
    rng = np.random.default_rng(3)
    k, v = _cache(rng, 1, 3, 1, 16, 4)
    table = np.array([[1, 2]])
    qkv = rng.standard_normal((4, 3 * 4))
    oc.append(k, v, 0, qkv, 1, [0, 4], [14], table, np.zeros((4, 1), int), np.ones(2))
    assert np.array_equal(k[0, 1, 0, 15], qkv[1, 4:8]) and np.array_equal(v[0, 2, 0, 0, :, 1], qkv[3, 8:])
    oc.compact(k, v, [14], table, np.array([[1, 3]]), [2])
    assert np.array_equal(k[0, 1, 0, 14], qkv[1, 4:8]) and np.array_equal(k[0, 1, 0, 15], qkv[3, 4:8])
    assert np.array_equal(v[0, 1, 0, 0, :, 15], qkv[3, 8:])


def test_update_invariants():
    """Counts equal the holders; a page that may be written has one; kept tokens keep their content."""
    rng = np.random.default_rng(4)
    for trial in range(50):
        page, width, pages = 16, 4, 40
        n = int(rng.integers(1, 6))
        length = rng.integers(0, width * page + 1, n)
        table = np.full((n, width), -1)
        for i in range(n):
            table[i, :-(-length[i] // page)] = rng.integers(0, 12, -(-length[i] // page))
        refs = np.bincount(table[table >= 0], minlength=pages)
        m = int(rng.integers(1, 7))
        parent, keep, room = rng.integers(-1, n, m), rng.integers(0, 70, m), rng.integers(0, 20, m)
        new, lens, left, short, copies = oc.update(table, length, refs, parent, keep, room, page)
        assert short == 0
        assert np.array_equal(left, np.bincount(new[new >= 0], minlength=pages))
        source = dict((d, s) for s, d in copies)
        for i in range(m):
            want = min(int(keep[i]), int(length[parent[i]])) if parent[i] >= 0 else 0
            assert lens[i] == want
            held = -(-want // page)
            for j in range(held):
                old = table[parent[i], j]
                assert new[i, j] == old or source.get(new[i, j]) == old and j == held - 1
            total = min(-(-(want + int(room[i])) // page), width)
            assert (new[i, :total] >= 0).all() and (new[i, total:] == -1).all()
            first = want // page  # from here on the lane may write
            assert (left[new[i, first:total]] == 1).all()


def test_beam_scores_closed_forms():
    x = np.log(np.array([[1.0, 2.0, 5.0], [4.0, 4.0, 8.0], [1.0, 1.0, 1.0], [3.0, 2.0, 1.0]]))
    s = oc.beam_scores(x, [0.0, -1.0, -2.0, -np.inf], [0, 0, 1, 0], 1)
    assert np.allclose(np.exp(s[0]), [1 / 8, 2 / 8, 5 / 8]) and np.allclose(np.exp(s[1] + 1), [0.25, 0.25, 0.5])
    assert s[2, 1] == -2.0 and np.isneginf(s[2, [0, 2]]).all() and np.isneginf(s[3]).all()
    best, parent, token = oc.beam_select(s, 2, 2, 3)
    assert parent.tolist() == [[0, 0, 1], [2, 2, 2]] and token.tolist() == [[2, 1, 2], [1, 0, 2]]


MUTANTS = {
    "bits of the mask reversed": lambda w: int("{:064b}".format(w & (2 ** 64 - 1))[::-1], 2),
    "drafts all seen": lambda w: 2 ** 64 - 1,
    "drafts never seen": lambda w: 0,
}


@pytest.mark.parametrize("name", sorted(MUTANTS))
def test_planted_mask_mistakes_show(name):
    rng = np.random.default_rng(5)
    k, v = _cache(rng, 1, 2, 1, 16, 4)
    q, table = rng.standard_normal((3, 4)), np.array([[0, 1]])
    a = oc.tree_attention(q, k, v, 0, [0, 3], [15], table, [1, 3, 5], 0.5, 1)[0]
    b = oc.tree_attention(q, k, v, 0, [0, 3], [15], table, [MUTANTS[name](w) for w in (1, 3, 5)], 0.5, 1)[0]
    assert np.abs(a - b).max() > 1e-3
