"""The paged cache's append, compaction and page-table update at the ends of their ranges."""
import numpy as np
import pytest

from oracle import cache as oc
from tests.cache_util import Lanes, cache_tensors, values
from tests.gpu_util import dev, host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_append_to_a_lane_of_negative_length(nv, dtype):
    """Stores neither k nor v of it; other lanes are whole, and so is q."""
    import torch
    lanes = Lanes(2, [5, 5, 9], [4, 3, 2], 16)
    k, v = cache_tensors(2, 1, lanes.pages, 1, 16, 64, dtype)
    wk, wv = values(k), values(v)
    qkv = torch.randn((9, 4 * 64), device="cuda").to(torch.float8_e4m3fn).to(torch.bfloat16)  # (exact in either type)
    pos = np.zeros((9, 1), np.int32)
    inv = np.ones(32, np.float32)
    start, ctx, table = lanes.dev()
    ctx[0], ctx[2] = -2, -(2 ** 31)
    q = nv.PagedCache(k, v).append(0, qkv, 2, start, ctx, table, dev(pos), dev(inv))
    lanes.table[0], lanes.table[2] = -1, -1
    oc.append(wk, wv, 0, host(qkv), 2, lanes.start, lanes.ctx, lanes.table, pos, inv)
    assert np.array_equal(values(k), wk) and np.array_equal(values(v), wv)
    assert torch.equal(q, qkv[:, :128])


def _update_case(seed, lanes_in, lanes_out, width, page, pages):
    """Tables with shared pages all over, and what a call makes of them."""
    rng = np.random.default_rng(seed)
    table = np.full((lanes_in, width), -1, np.int64)
    length = rng.integers(0, width * page + 1, lanes_in)
    for i in range(lanes_in):
        n = -(-int(length[i]) // page)
        table[i, :n] = rng.integers(0, pages, n)
    refs = np.bincount(table[table >= 0], minlength=pages) + (rng.random(pages) < 0.1)
    return (table, length, refs, rng.integers(-1, lanes_in + 1, lanes_out), rng.integers(0, width * page + 20, lanes_out),
            rng.integers(0, 3 * page, lanes_out))


# pages at and past what the one-workgroup kernel holds in LDS (32768; past 16384 more than 64 KiB), its most
# lanes, long tables, more lanes than a workgroup has threads, and both sides of the sum of the three that chooses
# it (2 (lanes_in + lanes_out) width + pages + 256 lanes_out = 81920); 8-bit page copies in every case
@pytest.mark.parametrize("lanes_in,lanes_out,width,pages", [
    (1, 120, 150, 14900), (1, 120, 150, 14901), (4, 300, 4, 2000), (1, 316, 1, 390), (1, 320, 1, 700), (20, 30, 40, 16385), (20, 30, 40, 32768), (20, 30, 40, 32769), (64, 64, 512, 32768), (64, 65, 512, 20000), (3, 1024, 8, 9000), (3, 1025, 8, 9000)])
@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
def test_update_at_the_limits_of_its_kernels(nv, lanes_in, lanes_out, width, pages, dtype):
    import torch
    page, dim = 16, 64
    case = _update_case(pages + lanes_out, lanes_in, lanes_out, width, page, pages)
    g = torch.Generator(device="cuda").manual_seed(3)
    t = torch.uint8 if dtype == "e4m3" else torch.int16
    k, v = (torch.randint(0, 120, s, generator=g, device="cuda", dtype=t)
            for s in ((2, pages, 1, page, dim), (2, pages, 1, page // 16, dim, 16)))
    wk, wv = k.clone(), v.clone()
    f = torch.float8_e4m3fn if dtype == "e4m3" else torch.bfloat16
    cache = nv.PagedCache(k.view(f), v.view(f), *((0.1, 0.2) if dtype == "e4m3" else ()))
    got = cache.update(*(dev(np.asarray(x, np.int32)) for x in case))
    table, length, refs, short, copies = oc.update(*case, page)
    for name, a, b in zip(("table", "length", "refs", "short"), got, (table, length, refs, short)):
        assert np.array_equal(host(a).ravel(), np.asarray(b).ravel()), name
    assert copies
    for a, b in copies:
        wk[:, b], wv[:, b] = wk[:, a], wv[:, a]
    assert torch.equal(k, wk) and torch.equal(v, wv)
