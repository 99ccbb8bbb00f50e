"""GPU parity of the attention of drafted tokens over a paged cache, against the fp64 oracle."""
import numpy as np
import pytest

from oracle import cache as oc
from tests.cache_util import Lanes, cache_tensors, chain, check_attention, values
from tests.gpu_util import CANARY_ELEMS, canary_out, dev, host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


def _queries(seed, rows, width, std=2.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + 77)
    return (std * torch.randn((rows, width), generator=g, device="cuda")).to(torch.bfloat16)


def _random_masks(seed, lanes):
    rng = np.random.default_rng(seed + 5)
    words = []
    for n in lanes.rows:
        for t in range(n):
            w = int(rng.integers(0, 2 ** 62)) & ((1 << (t + 1)) - 1) | (1 << t)
            words.append(w - (1 << 64) if w >> 63 else w)
    return np.array(words, np.int64)


def _run(nv, lanes, q_heads, kv_heads, dim, page, dtype, masks=None, seed=0, k=None, v=None, layers=1, layer=0, q=None, scale=None, k_scale=0.07, v_scale=0.055,
         max_rows=None):
    import torch
    if k is None:
        k, v = cache_tensors(seed, layers, lanes.pages, kv_heads, page, dim, dtype)
    if dtype != "e4m3":
        k_scale = v_scale = 1.0
    elif k_scale == 0.07:
        k, v = (k.float() / k_scale).to(k.dtype), (v.float() / v_scale).to(v.dtype)
    rows = int(lanes.start[-1])
    q = _queries(seed, rows, q_heads * dim) if q is None else q
    masks = np.concatenate([chain(n) for n in lanes.rows]) if masks is None else masks
    out, canary = canary_out(rows, q_heads * dim, torch.bfloat16)
    cache = nv.PagedCache(k, v, k_scale, v_scale)
    start, ctx, table = lanes.dev()
    scale = dim ** -0.5 if scale is None else scale
    _, lse = cache.attend(layer, q, start, ctx, table, dev(masks), max_rows or max(lanes.rows), scale, out=out, with_lse=True)
    torch.cuda.synchronize()
    canary("attention")
    want = oc.tree_attention(host(q)[:, :q_heads * dim], values(k, k_scale), values(v, v_scale), layer, lanes.start, lanes.ctx, lanes.table, masks, scale, q_heads)
    what = "lanes %s + %s, heads %d/%d, dim %d, page %d, %s" % (list(lanes.ctx), lanes.rows, q_heads, kv_heads, dim, page, dtype)
    n = int(max(c + r for c, r in zip(lanes.ctx, lanes.rows)))
    check_attention(out, lse, want, n, dim, what)
    return out, lse


# (contexts, rows, q heads, kv heads, dim, page, dtype): one token and none of context; contexts
# and pages that end inside a tile; every block shape (rows x heads per kv head up to 16, 32, 64, 128,
# above), head dim, page size and type.
CASES = [
    ([0], [1], 1, 1, 64, 16, "bf16"),
    ([1], [1], 4, 4, 128, 16, "e4m3"),
    ([300], [1], 24, 2, 256, 64, "bf16"),
    ([63, 64, 65, 0], [1, 1, 1, 1], 12, 4, 128, 64, "bf16"),
    ([1000, 17, 513], [1, 1, 1], 16, 1, 64, 32, "e4m3"),
    ([129, 640], [2, 1], 12, 1, 128, 128, "bf16"),
    ([500, 3], [2, 2], 12, 1, 256, 256, "e4m3"),
    ([200, 77], [5, 3], 8, 1, 256, 16, "bf16"),
    ([321, 0, 90], [7, 8, 0], 16, 2, 128, 32, "bf16"),
    ([320, 15], [8, 5], 12, 1, 64, 64, "bf16"),
    ([700], [8], 48, 4, 128, 64, "e4m3"),
    ([255, 100], [64, 33], 12, 2, 128, 64, "bf16"),
    ([100], [64], 16, 1, 128, 16, "e4m3"),
    ([130], [64], 6, 1, 256, 128, "bf16"),
    ([90, 31], [64, 17], 10, 2, 64, 256, "e4m3"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_trees(nv, case):
    ctx, rows, qh, kh, dim, page, dtype = case
    lanes = Lanes(len(ctx) + dim, ctx, rows, page)
    _run(nv, lanes, qh, kh, dim, page, dtype, masks=_random_masks(dim, lanes), seed=sum(ctx))


@pytest.mark.parametrize("ctx,dim,dtype", [(5000, 128, "bf16"), (9001, 64, "e4m3"), (3333, 256, "bf16")])
def test_context_split_over_workers(nv, ctx, dim, dtype):
    """One lane whose context many workgroups share, and a short one beside it."""
    lanes = Lanes(3, [ctx, 70], [2, 1], 64)
    _run(nv, lanes, 6, 1, dim, 64, dtype, seed=ctx)


def test_many_lanes(nv):
    """More lanes than a wave has threads, empty ones among them."""
    rng = np.random.default_rng(8)
    rows = [int(x) for x in rng.integers(0, 3, 150)]
    ctx = [int(x) for x in rng.integers(0, 200, 150)]
    lanes = Lanes(4, ctx, rows, 16)
    _run(nv, lanes, 4, 2, 64, 16, "bf16", seed=9)


def test_rows_that_see_nothing(nv):
    """No context and an empty mask word: zeros and -inf; beside rows that see something."""
    lanes = Lanes(5, [0, 0, 40], [3, 2, 2], 32)
    masks = np.array([0, 2, 0, 0, 0, 0, 1], np.int64)
    out, lse = _run(nv, lanes, 4, 2, 128, 32, "bf16", masks=masks, seed=3)
    assert (host(out)[[0, 2, 3, 4]] == 0).all() and np.isneginf(host(lse)[[0, 2, 3, 4]]).all()


@pytest.mark.parametrize("dtype,fill", [("bf16", 0xFF), ("e4m3", 0xFF), ("bf16", 0x7F)])
def test_unused_memory_is_not_seen(nv, dtype, fill):
    """Pages full of NaN (or of the largest values) except where the lanes' tokens are."""
    import torch
    page, dim, kh = 32, 128, 2
    lanes = Lanes(6, [45, 7, 100], [3, 2, 1], page)
    k, v = cache_tensors(1, 1, lanes.pages, kh, page, dim, dtype)
    bad_k, bad_v = cache_tensors(1, 1, lanes.pages, kh, page, dim, dtype, fill=fill)
    kb, vb, ks, vs = (t.view(torch.uint8 if dtype == "e4m3" else torch.int16) for t in (bad_k, bad_v, k, v))
    for b, n in enumerate(lanes.ctx + np.array(lanes.rows)):
        for t in range(int(n)):
            p, o = int(lanes.table[b, t // page]), t % page
            kb[0, p, :, o] = ks[0, p, :, o]
            vb[0, p, :, o // 16, :, o % 16] = vs[0, p, :, o // 16, :, o % 16]
    a = _run(nv, lanes, 4, kh, dim, page, dtype, k=bad_k, v=bad_v, k_scale=1.0, v_scale=1.0, seed=2)
    b = _run(nv, lanes, 4, kh, dim, page, dtype, k=k, v=v, k_scale=1.0, v_scale=1.0, seed=2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_missing_pages_are_not_seen(nv):
    """Table entries outside the pool: their tokens do not exist."""
    lanes = Lanes(7, [200, 90], [2, 2], 16)
    lanes.table[0, 3], lanes.table[0, 7], lanes.table[1, 0] = -1, lanes.pages, 1 << 30
    _run(nv, lanes, 4, 1, 64, 16, "bf16", seed=5)


def test_large_scores(nv):
    """Scores of several hundred: the running maximum moves far and often."""
    lanes = Lanes(9, [700, 64], [4, 4], 64)
    _run(nv, lanes, 8, 2, 64, 64, "bf16", seed=6, scale=4.0)


def test_strides_and_layers(nv):
    """Rows inside wider ones, a layer of several, pages and layers with gaps."""
    import torch
    lanes = Lanes(10, [150, 20], [3, 1], 32)
    qh, kh, dim, page = 6, 3, 128, 32
    n = kh * page * dim
    big = torch.randn((2, lanes.pages, 2, n + 64), device="cuda").to(torch.bfloat16)
    k, v = big[:, :, 0, :n].view(2, lanes.pages, kh, page, dim), big[:, :, 1, :n].view(2, lanes.pages, kh, page // 16, dim, 16)
    rows = int(lanes.start[-1])
    q = _queries(11, rows, qh * dim + 24)
    masks = np.concatenate([chain(x) for x in lanes.rows])
    out = torch.full((rows, qh * dim + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    cache = nv.PagedCache(k, v)
    start, ctx, table = lanes.dev()
    _, lse = cache.attend(1, q[:, :qh * dim], start, ctx, table, dev(masks), 3, 0.1, out=out, with_lse=True)
    want = oc.tree_attention(host(q)[:, :qh * dim], values(k), values(v), 1, lanes.start, lanes.ctx, lanes.table, masks, 0.1, qh)
    check_attention(out[:, :qh * dim].contiguous(), lse, want, 160, dim, "strides")
    assert (out[:, qh * dim:] == 7.0).all()


def test_page_offsets_past_32_bits(nv):
    """Pages more than 4 GiB into the pool."""
    import torch
    page, dim, kh = 256, 256, 8
    pages = (5 << 30) // (page * dim * kh * 2)
    k = torch.zeros((1, pages, kh, page, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((1, pages, kh, page // 16, dim, 16), dtype=torch.bfloat16, device="cuda")
    lanes = Lanes(12, [300], [2], page)
    lanes.pages = pages
    lanes.table[0, :2] = [pages - 1, pages - 2]
    g = torch.Generator(device="cuda").manual_seed(4)
    for x in (k, v):
        x[0, -2:] = torch.randn(x[0, -2:].shape, generator=g, device="cuda").to(torch.bfloat16)
    small = Lanes(12, [300], [2], page)
    small.table[0, :2], small.pages = [1, 0], 2
    masks = chain(2)
    q = _queries(1, 2, kh * dim)
    start, ctx, table = lanes.dev()
    out, lse = nv.PagedCache(k, v).attend(0, q, start, ctx, table, dev(masks), 2, 0.05, with_lse=True)
    want = oc.tree_attention(host(q), values(k[:, -2:]), values(v[:, -2:]), 0, small.start, small.ctx, small.table, masks, 0.05, kh)
    check_attention(out, lse, want, 302, dim, "offsets")


def test_repeats_and_other_streams(nv):
    """The same bits again, on another stream, and in replays of a graph between eager calls."""
    import torch
    lanes = Lanes(13, [2000, 900, 30], [4, 2, 1], 64)
    k, v = cache_tensors(3, 1, lanes.pages, 2, 64, 128, "bf16")
    cache = nv.PagedCache(k, v)
    start, ctx, table = lanes.dev()
    q = _queries(2, 7, 8 * 128)
    masks = dev(np.concatenate([chain(x) for x in lanes.rows]))
    args = (0, q, start, ctx, table, masks, 4, 0.09)
    first = cache.attend(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = cache.attend(*args)
    torch.cuda.synchronize()
    assert torch.equal(first, other)
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend(*args, out=out)
    for i in range(4):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first), i
        assert torch.equal(cache.attend(*args), first), i
    # the graph follows the lengths that are there when it runs
    ctx.copy_(torch.tensor([100, 2, 29], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, cache.attend(*args)) and not torch.equal(out, first)


def test_rows_past_max_rows_are_left(nv):
    """A lane with more rows than max_rows: the others are computed, the rest left alone."""
    import torch
    lanes = Lanes(14, [50], [6], 16)
    k, v = cache_tensors(4, 1, lanes.pages, 1, 16, 64, "bf16")
    start, ctx, table = lanes.dev()
    q = _queries(3, 6, 64)
    masks = dev(chain(6))
    out = torch.full((6, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    nv.PagedCache(k, v).attend(0, q, start, ctx, table, masks, 4, 0.1, out=out)
    assert (out[4:] == 5.0).all() and not (out[:4] == 5.0).all(1).any()


def test_lanes_outside_the_rows_are_left(nv):
    """Lanes whose rows start or end outside the call's rows are not computed; the others are."""
    import torch
    lanes = Lanes(15, [40, 20, 30], [2, 2, 2], 16)
    k, v = cache_tensors(5, 1, lanes.pages, 1, 16, 64, "bf16")
    _, ctx, table = lanes.dev()
    q = _queries(4, 4, 64)
    cache, masks = nv.PagedCache(k, v), dev(chain(2).repeat(2).reshape(2, 2).T.copy().ravel())
    out = torch.full((4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    cache.attend(0, q, dev(np.array([0, 2, 4, 6], np.int32)), ctx, table, masks, 2, 0.1, out=out)
    assert not (out == 5.0).all(1).any()  # the third lane's rows 4 and 5 do not exist
    out.fill_(5.0)
    cache.attend(0, q, dev(np.array([-2, 0, 2, 9], np.int32)), ctx, table, masks, 2, 0.1, out=out)
    assert not (out[:2] == 5.0).all(1).any() and not (out[2:4] == 5.0).all(1).any()
