"""Attention over the paged cache: scores that are no numbers, and contexts shared out among many lanes."""
import numpy as np
import pytest

from oracle import cache as oc
from tests.cache_util import Lanes, cache_tensors, chain, check_attention, values
from tests.gpu_util import dev, host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


@pytest.mark.parametrize("ctx", [130, 5000])  # walked by one workgroup, and shared out and joined
@pytest.mark.parametrize("dim,group,rows", [(64, 4, 3), (128, 12, 8), (256, 2, 2)])
def test_nan_in_what_a_row_sees(nv, ctx, dim, group, rows):
    """A NaN score makes the row's output and log-sum NaN (-inf is for rows that see nothing), and leaves
    the rows that do not see it to the bit as they were."""
    import torch
    nan = float("nan")
    lanes = Lanes(dim, [ctx, 70], [rows, 1], 64)
    k, v = cache_tensors(1, 1, lanes.pages, 1, 64, dim, "bf16")
    start, c, table = lanes.dev()
    masks = dev(np.concatenate([chain(n) for n in lanes.rows]))
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((rows + 1, group * dim), generator=g, device="cuda").to(torch.bfloat16)
    cache = nv.PagedCache(k, v)

    def run(x):
        out, lse = cache.attend(0, x, start, c, table, masks, rows, 0.1, with_lse=True)
        return host(out).reshape(rows + 1, group, dim), host(lse)

    out, lse = run(q)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    # one head's query
    bad = q.clone()
    bad[1, dim + 3] = nan
    o, z = run(bad)
    hit = np.zeros((rows + 1, group), bool)
    hit[1, 1] = True
    assert np.isnan(o[hit]).all() and np.isnan(z[hit]).all()
    assert np.array_equal(o[~hit], out[~hit]) and np.array_equal(z[~hit], lse[~hit])
    # a key of the first lane's context: all of its rows
    t = ctx // 2
    k[0, int(lanes.table[0, t // 64]), 0, t % 64, 5] = nan
    o, z = run(q)
    assert np.isnan(o[:rows]).all() and np.isnan(z[:rows]).all()
    assert np.array_equal(o[rows], out[rows]) and np.array_equal(z[rows], lse[rows])


@pytest.mark.parametrize("kv_heads", [1, 4])  # 100 items, fewer than workers; 400, more than workers
def test_shared_contexts_of_many_lanes(nv, kv_heads):
    """More lanes than a wave has threads, long contexts among them that several workgroups share."""
    import torch
    rng = np.random.default_rng(8)
    rows = [int(x) for x in rng.integers(0, 3, 120)]
    ctx = [int(x) for x in rng.integers(0, 200, 120)]
    for b, n in ((3, 3001), (63, 1500), (64, 2000), (70, 5000), (118, 777), (119, 4000)):
        rows[b], ctx[b] = 2, n
    lanes = Lanes(4, ctx, rows, 16)
    k, v = cache_tensors(9, 1, lanes.pages, kv_heads, 16, 64, "bf16")
    g = torch.Generator(device="cuda").manual_seed(6)
    total, qh = int(lanes.start[-1]), 2 * kv_heads
    q = (2 * torch.randn((total, qh * 64), generator=g, device="cuda")).to(torch.bfloat16)
    masks = np.concatenate([chain(n) for n in rows])
    start, c, table = lanes.dev()
    out, lse = nv.PagedCache(k, v).attend(0, q, start, c, table, dev(masks), 2, 0.125, with_lse=True)
    want = oc.tree_attention(host(q), values(k), values(v), 0, lanes.start, lanes.ctx, lanes.table, masks, 0.125, qh)
    check_attention(out, lse, want, 5002, 64, "%d kv heads" % kv_heads)
