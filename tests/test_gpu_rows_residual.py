"""GPU parity of the norm where the residual stream is some columns of a wide buffer."""
import numpy as np
import pytest

from oracle import rows as oracle
from tests.gpu_util import host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


@pytest.mark.parametrize("K,width,at", [(64, 1000, 8), (1001, 4003, 1), (5120, 40960, 5120), (640, 1280, 0), (640, 1288, 0)])
def test_a_stream_of_a_wide_buffer(nv, K, width, at):
    """Eager, and captured and replayed with new values in the buffer, which keeps them."""
    import torch
    rng = np.random.default_rng(K + width)
    x, w = oracle.bf16(rng.standard_normal((7, K))), oracle.bf16(rng.standard_normal(K))
    xd, wd = (torch.from_numpy(v.astype(np.float32)).cuda().to(torch.bfloat16) for v in (x, w))
    wide = torch.empty((7, width), dtype=torch.bfloat16, device="cuda")
    fill = lambda: wide.copy_(torch.from_numpy(oracle.bf16(rng.standard_normal((7, width))).astype(np.float32)))  # noqa: E731

    def check(got, stream):
        torch.cuda.synchronize()
        y, h = oracle.rms_norm(x, w, 1e-6, 0.0, host(wide.float())[:, at:at + K], "bf16")
        assert np.array_equal(host(stream.float()), h) and np.array_equal(host(got.float()), oracle.bf16(y))

    fill()
    before = wide.clone()
    check(*nv.rms_norm(xd, wd, 1e-6, residual=wide[:, at:at + K]))
    assert torch.equal(wide, before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = nv.rms_norm(xd, wd, 1e-6, residual=wide[:, at:at + K])
    for _ in range(4):
        fill()
        before = wide.clone()
        graph.replay()
        check(*out)
        assert torch.equal(wide, before)
