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
