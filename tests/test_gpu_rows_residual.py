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


@pytest.mark.parametrize("K", [40, 1001, 1536, 5120, 7001, 17408, 24584, 30001])
@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_streams_in_place(nv, K, name):
    """The new stream in place of x, of the residual, and of both where they are one; the norm in place of x."""
    import torch
    rng = np.random.default_rng(K)
    types = {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8}
    x, r = (oracle.to_type(rng.standard_normal((5, K)) * 3, name) for _ in range(2))
    w = oracle.to_type(rng.standard_normal(K), "bf16")
    put = lambda v, t: torch.from_numpy(v.astype(np.float32)).cuda().to(types[t])  # noqa: E731
    wd = put(w, "bf16")
    for out in ("bf16", "f32", "int8"):
        for place in ("x", "residual", "one"):
            xd = put(x, name)
            rd = xd if place == "one" else put(r, name)
            y, h = oracle.rms_norm(x, w, 1e-6, 0.0, x if place == "one" else r, name)
            got = nv.rms_norm(xd, wd, 1e-6, residual=rd, residual_out=rd if place == "residual" else xd, dtype=types[out])
            assert got[-1].data_ptr() == (rd if place == "residual" else xd).data_ptr()
            assert np.array_equal(host(got[-1].float()), h), (K, out, place)
            if out == "int8":
                q, s = oracle.codes(y)
                assert np.array_equal(host(got[1]), s) and np.array_equal(host(got[0]), q), (K, out, place)
            else:
                assert np.array_equal(host(got[0].float()), oracle.to_type(y, out)), (K, out, place)
    xd = put(x, name)
    y, _ = oracle.rms_norm(x, w, 1e-6)
    nv.rms_norm(xd, wd, 1e-6, dtype=types[name], out=xd)
    assert np.array_equal(host(xd.float()), oracle.to_type(y, name)), K
