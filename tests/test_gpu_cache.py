"""GPU parity of the paged cache's append, compaction and page-table update, against the oracle."""
import numpy as np
import pytest

from oracle import cache as oc
from tests.cache_util import Lanes, bf16, cache_tensors, values
from tests.gpu_util import dev, host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


def _e4m3_tol(x, scale):
    """Half a unit of the last place of E4M3 at |x| (3 mantissa bits, subnormals of 2^-9)."""
    y = np.abs(x) / scale
    return scale * np.maximum(y * 2.0 ** -4, 2.0 ** -10)


# (contexts, rows, q heads, kv heads, dim, page, dtype, axes, pairs, interleaved)
APPENDS = [
    ([0], [1], 1, 1, 64, 16, "bf16", 1, 32, False),
    ([5, 64, 15], [8, 8, 1], 12, 2, 128, 64, "bf16", 1, 64, False),
    ([31, 0, 7], [3, 0, 70], 4, 1, 128, 16, "e4m3", 3, 64, True),
    ([1, 250], [40, 7], 6, 3, 256, 32, "bf16", 2, 32, True),
    ([100], [300], 2, 2, 64, 128, "e4m3", 1, 8, False),
    ([3, 9], [17, 2], 2, 1, 256, 256, "e4m3", 1, 128, False),
    ([12], [9], 3, 1, 64, 16, "bf16", 1, 0, False),
    ([12, 1], [9, 5], 3, 1, 128, 16, "bf16", 3, 4, True),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "-".join(str(x) for x in c))
def test_append(nv, case):
    import torch
    ctx, rows, qh, kh, dim, page, dtype, axes, pairs, inter = case
    lanes = Lanes(sum(rows), ctx, rows, page)
    total = int(lanes.start[-1])
    rng = np.random.default_rng(dim + total)
    k, v = cache_tensors(5, 2, lanes.pages, kh, page, dim, dtype)
    ks, vs = (0.05, 0.11) if dtype == "e4m3" else (1.0, 1.0)
    k0, v0 = values(k, ks), values(v, vs)
    qkv = torch.randn((total, (qh + 2 * kh) * dim), device="cuda").to(torch.bfloat16)
    pos = rng.integers(0, 300000, (total, axes)).astype(np.int32)
    inv = (1e6 ** (-np.arange(pairs) / max(pairs, 1))).astype(np.float32)
    axis = rng.integers(0, axes, pairs).astype(np.uint8)
    q = nv.PagedCache(k, v, ks, vs).append(1, qkv, qh, *lanes.dev(), dev(pos), dev(inv), pair_axis=dev(axis), interleaved=inter, factor=1.1)
    x = host(qkv)
    wk, wv = k0.copy(), v0.copy()
    want = oc.append(wk, wv, 1, x, qh, lanes.start, lanes.ctx, lanes.table, pos, inv, axis, inter, 1.1)
    # a rotated value: two fp32 products with cosines off by 2^-22, and one rounding
    size = 1.1 * 2.0 ** -20 * (np.abs(x).max() * 2)
    got = host(q).reshape(want.shape)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + size).all()
    for what, g, w, old, s in (("k", values(k, ks), wk, k0, ks), ("v", values(v, vs), wv, v0, vs)):
        written = w != old
        tol = (_e4m3_tol(w, s) if dtype == "e4m3" else 2.0 ** -8 * np.abs(w)) + size
        assert (np.abs(g - w) <= np.where(written, tol, 0)).all(), what
        if what == "v" and dtype == "bf16":
            assert np.array_equal(g, w)


def test_append_in_place_and_strided(nv):
    """q written over the qkv rows; rows inside wider ones; no axis map."""
    import torch
    lanes = Lanes(1, [20, 3], [5, 2], 16)
    qh, kh, dim = 3, 1, 64
    qkv = torch.randn((7, (qh + 2 * kh) * dim + 12), device="cuda").to(torch.bfloat16)
    x = host(qkv)[:, :(qh + 2 * kh) * dim]
    k, v = cache_tensors(1, 1, lanes.pages, kh, 16, dim, "bf16")
    wk, wv = values(k), values(v)
    pos = np.arange(7, dtype=np.int32)[:, None] * 11
    inv = (1e4 ** (-np.arange(32) / 32)).astype(np.float32)
    tail = qkv[:, qh * dim:].clone()
    cache = nv.PagedCache(k, v)
    cache.append(0, qkv, qh, *lanes.dev(), dev(pos), dev(inv), out=qkv)
    want = oc.append(wk, wv, 0, x, qh, lanes.start, lanes.ctx, lanes.table, pos, inv)
    got = host(qkv)[:, :qh * dim].reshape(want.shape)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * np.abs(x).max()).all()
    assert torch.equal(qkv[:, qh * dim:], tail)
    assert np.array_equal(values(v), wv)
    assert (np.abs(values(k) - wk) <= 2.0 ** -8 * np.abs(wk) + 2.0 ** -19 * np.abs(x).max()).all()


def test_append_without_pages(nv):
    """Tokens past the table, and in entries outside the pool, are stored nowhere; q is whole."""
    import torch
    lanes = Lanes(2, [10, 30], [40, 4], 16)
    lanes.table = np.ascontiguousarray(lanes.table[:, :3])  # lane 0 needs four
    lanes.table[0, 1], lanes.table[1, 2] = lanes.pages + 5, -9
    k, v = cache_tensors(2, 1, lanes.pages, 1, 16, 64, "bf16")
    wk, wv = values(k), values(v)
    qkv = torch.randn((44, 4 * 64), device="cuda").to(torch.bfloat16)
    pos = np.zeros((44, 1), np.int32)
    inv = np.ones(32, np.float32)
    q = nv.PagedCache(k, v).append(0, qkv, 2, *lanes.dev(), dev(pos), dev(inv))
    oc.append(wk, wv, 0, host(qkv), 2, lanes.start, lanes.ctx, lanes.table, pos, inv)
    assert np.array_equal(values(k), wk) and np.array_equal(values(v), wv)
    assert torch.equal(q, qkv[:, :128])  # position 0 turns nothing


def test_append_saturates(nv):
    import torch
    lanes = Lanes(3, [0], [8], 16)
    k, v = cache_tensors(2, 1, lanes.pages, 1, 16, 64, "e4m3")
    qkv = torch.full((8, 3 * 64), 1000.0, device="cuda").to(torch.bfloat16)
    qkv[:, 1::2] = -1000.0
    nv.PagedCache(k, v, 2.0, 0.5).append(0, qkv, 1, *lanes.dev(), dev(np.zeros((8, 1), np.int32)), dev(np.ones(32, np.float32)))
    page = int(lanes.table[0, 0])
    assert sorted(set(values(k)[0, page, 0, :8].ravel())) == [-448.0, 448.0]
    assert sorted(set(values(v)[0, page, 0, 0, :, :8].ravel())) == [-448.0, 448.0]


# (contexts, rows, accepted paths, kv heads, dim, page, dtype, layers)
COMPACTS = [
    ([10], [8], [[0, 2, 5, 7]], 2, 128, 64, "bf16", 3),
    ([13, 0, 31], [8, 3, 5], [[1, 2, 3, 6], [2], []], 1, 64, 16, "e4m3", 2),
    ([5, 60], [64, 64], [list(range(0, 64, 2)), list(range(64))], 2, 256, 32, "bf16", 1),
    ([5], [64], [[63, 0, 1, 2, 40]], 1, 128, 128, "e4m3", 2),
]


@pytest.mark.parametrize("case", COMPACTS, ids=lambda c: "-".join(str(x) for x in c[:2] + c[3:]))
def test_compact(nv, case):
    ctx, rows, paths, kh, dim, page, dtype, layers = case
    lanes = Lanes(dim, ctx, rows, page)
    k, v = cache_tensors(7, layers, lanes.pages, kh, page, dim, dtype)
    wk, wv = values(k), values(v)
    width = max(max(len(p) for p in paths), 1) + 2
    path = np.full((len(ctx), width), -5, np.int32)
    for i, p in enumerate(paths):
        path[i, :len(p)] = p
    accepted = np.array([len(p) for p in paths], np.int32)
    _, c, t = lanes.dev()
    nv.PagedCache(k, v).compact(c, t, dev(path), dev(accepted))
    oc.compact(wk, wv, lanes.ctx, lanes.table, path, accepted)
    assert np.array_equal(values(k), wk) and np.array_equal(values(v), wv)


def test_compact_skips_what_does_not_exist(nv):
    """Entries outside [0, 64), counts outside the row, tokens past the table or in missing pages."""
    lanes = Lanes(8, [14, 20], [8, 8], 16)
    lanes.table[1, 1] = -1
    k, v = cache_tensors(8, 1, lanes.pages, 1, 16, 64, "bf16")
    wk, wv = values(k), values(v)
    path = np.array([[3, -1, 64, 200, 5], [1, 2, 3, 4, 5]], np.int32)
    accepted = np.array([99, 5], np.int32)
    _, c, t = lanes.dev()
    nv.PagedCache(k, v).compact(c, t, dev(path), dev(accepted))
    oc.compact(wk, wv, lanes.ctx, lanes.table, path, accepted)
    assert np.array_equal(values(k), wk) and np.array_equal(values(v), wv)


def _check_update(nv, table, length, refs, parent, keep, reserve, page, layers=1, kh=1, dim=64, dtype="bf16"):
    import torch
    pages = len(refs)
    k, v = cache_tensors(9, layers, pages, kh, page, dim, dtype)
    wk, wv = values(k), values(v)
    i32 = lambda a: None if a is None else dev(np.asarray(a, np.int32))  # noqa: E731
    got = nv.PagedCache(k, v).update(i32(table), i32(length), i32(refs), i32(parent), i32(keep), i32(reserve))
    torch.cuda.synchronize()
    want = oc.update(np.asarray(table), length, refs, parent, keep, reserve, page)
    for name, g, w in zip(("table", "length", "refs", "short"), got, want):
        assert np.array_equal(host(g).ravel(), np.asarray(w).ravel()), name
    for a, b in want[4]:
        wk[:, b], wv[:, b] = wk[:, a], wv[:, a]
    assert np.array_equal(values(k), wk) and np.array_equal(values(v), wv)
    return want


def test_update_reorders_and_copies(nv):
    """Two beams continue lane 0, one lane 2, one starts empty; lane 1 ends and is freed."""
    table = [[4, 7, -1, -1], [4, 2, 5, -1], [9, -1, -1, -1]]
    refs = np.zeros(12, int)
    for p in (4, 7, 4, 2, 5, 9):
        refs[p] += 1
    new, lens, left, short, copies = _check_update(nv, table, [20, 40, 16], refs, [0, 0, 2, -1], None, [1, 1, 1, 17], 16, layers=3, kh=2)
    # by hand: 7 stays lane 0's, lane 1 copies it to page 0; lane 2 (a whole page) gets page 1 as room,
    # and lane 3 two of the next free ones
    assert new.tolist() == [[4, 7, -1, -1], [4, 0, -1, -1], [9, 1, -1, -1], [2, 3, -1, -1]]
    assert copies == [(7, 0)] and short == 0 and left.tolist() == [1, 1, 1, 1, 2, 0, 0, 1, 0, 1, 0, 0]


def test_update_truncates_and_runs_out(nv):
    """keep cuts a page that another lane holds whole; too few pages; reserve past the table's width."""
    table = [[0, 1, 2], [0, 1, -1], [3, -1, -1]]
    refs = [2, 2, 1, 1]
    _check_update(nv, table, [48, 32, 5], refs, [0, 1, 2, 2, 0], [20, 32, 99, 3, 0], [100, 1, 0, 0, 33], 16)
    _check_update(nv, table, [48, 32, 5], refs, [-1, 7, -1], None, None, 16)  # everything is freed
    # page 1 held by someone outside too
    _check_update(nv, table, [48, 20, 5], [2, 3, 1, 1, 0, 0], [1, 2], None, [0, 0], 16)


@pytest.mark.parametrize("lanes_in,lanes_out,width,page,pages", [(1, 1, 1, 16, 1), (8, 8, 9, 16, 90), (64, 80, 33, 32, 2500), (5, 1500, 7, 16, 6000), (300, 257, 12, 256, 1500)])
def test_update_random(nv, lanes_in, lanes_out, width, page, pages):
    rng = np.random.default_rng(lanes_in + pages)
    table = np.full((lanes_in, width), -1, np.int64)
    length = rng.integers(0, width * page + 1, lanes_in)
    for i in range(lanes_in):
        n = -(-int(length[i]) // page)
        table[i, :n] = rng.integers(0, pages, n)  # shared pages all over
        if rng.random() < 0.1:
            table[i, rng.integers(0, width)] = rng.choice([-3, pages, 1 << 29])
    refs = np.bincount(table[(table >= 0) & (table < pages)], minlength=pages) + (rng.random(pages) < 0.1)
    parent = rng.integers(-1, lanes_in + 1, lanes_out)
    keep = rng.integers(0, width * page + 20, lanes_out)
    reserve = rng.integers(0, 3 * page, lanes_out)
    _check_update(nv, table, length, refs, parent, keep, reserve, page)


def test_update_in_a_graph(nv):
    """Replays follow the inputs and give the eager results."""
    import torch
    page, pages = 16, 40
    k, v = cache_tensors(3, 2, pages, 1, page, 64, "bf16")
    cache = nv.PagedCache(k, v)
    table = dev(np.array([[0, 1, 2, -1], [0, 3, -1, -1]], np.int32))
    length, refs = dev(np.array([40, 20], np.int32)), dev(np.array([2, 1, 1, 1] + [0] * 36, np.int32))
    parent, reserve = dev(np.array([1, 1], np.int32)), dev(np.array([5, 30], np.int32))
    cache.update(table, length, refs, parent, None, reserve)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cache.update(table, length, refs, parent, None, reserve)
    for p in ([1, 1], [0, 1], [0, 0], [-1, 0]):
        parent.copy_(torch.tensor(p, dtype=torch.int32))
        for x in out:
            x.fill_(-77)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, cache.update(table, length, refs, parent, None, reserve)):
            assert torch.equal(a, b), p


def test_compact_and_update_offsets_past_32_bits(nv):
    import torch
    page, dim, kh = 256, 256, 8
    pages = (5 << 30) // (page * dim * kh * 2)
    k = torch.zeros((1, pages, kh, page, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((1, pages, kh, page // 16, dim, 16), dtype=torch.bfloat16, device="cuda")
    cache = nv.PagedCache(k, v)
    last = pages - 1
    k[0, last] = torch.randn(k[0, last].shape, device="cuda").to(torch.bfloat16)
    v[0, last] = torch.randn(v[0, last].shape, device="cuda").to(torch.bfloat16)
    table = torch.tensor([[last]], dtype=torch.int32, device="cuda")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    kk, vv = k[0, last, :, 9].clone(), v[0, last, :, 0, :, 9].clone()
    cache.compact(i32(4), table, torch.tensor([[5]], dtype=torch.int32, device="cuda"), i32(1))
    assert torch.equal(k[0, last, :, 4], kk) and torch.equal(v[0, last, :, 0, :, 4], vv)
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    refs[pages - 2] = 0
    new, _, _, _ = cache.update(table, i32(10), refs, i32(0, 0))
    assert new.flatten().tolist() == [last, pages - 2]
    assert torch.equal(k[0, last], k[0, pages - 2]) and torch.equal(v[0, last], v[0, pages - 2])


def test_bf16_rounding_of_v_is_the_input():
    """The oracle's V is the input itself: bf16 values stay what they are."""
    x = np.array([1.0, -0.0, 3.140625, 2.0 ** -130])
    assert np.array_equal(bf16(x), x)
