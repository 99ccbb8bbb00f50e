"""CPU tests of the norm, the 8-bit calls and their binding at the ends of what they take."""
import os

import pytest


@pytest.fixture(scope="module")
def nv():
    import nvfp4_weight_streaming_amd as nv
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_weight_streaming_amd import build as b
        b.build()
    nv.lib()
    return nv


@pytest.mark.parametrize("M", [(1 << 22) + 1, 2 ** 31 - 129, 2 ** 31 - 100, 2 ** 31 - 1])
@pytest.mark.parametrize("K,N", [(64, 64), (5120, 7168), (131056, 16), (131056, 1 << 30)])
def test_workspace_of_more_rows_than_a_product_takes(nv, M, K, N):
    assert nv.nvfp4_int8_gemm_workspace_bytes(M, K, N) == 0


def test_a_weight_keeps_nothing_of_the_callers(nv, monkeypatch):
    """What the caller writes into the scales' buffer afterwards is not the weight's."""
    import torch

    from tests.test_rows_binding import _gpu_class, _recorded
    OnGpu = _gpu_class()
    seen = _recorded(nv, monkeypatch)
    codes, scale = torch.zeros((48, 64), dtype=torch.int8).as_subclass(OnGpu), torch.arange(48.0).as_subclass(OnGpu)
    w = nv.Int8Weight.from_canonical(codes, scale)
    scale.zero_()
    assert torch.equal(w.scale, torch.arange(48.0)) and w.scale.get_device() == 0
    w.packed = w.packed.as_subclass(OnGpu)
    nv.int8_gemm(codes[:3], scale[:3], w)
    assert seen["nvfp4_int8_gemm"][4] == w.scale.data_ptr() != scale.data_ptr()


@pytest.mark.parametrize("rows,ld,alike", [(3, 64, True), (3, 128, True), (3, 129, False), (3, 100000, False), (1, 100000, False)])
def test_the_new_stream_takes_memory_for_its_rows(nv, monkeypatch, rows, ld, alike):
    """A residual of a few columns of a wide buffer: the new one is not as wide."""
    import struct

    import torch

    from tests.test_rows_binding import _gpu_class, _recorded
    OnGpu = _gpu_class()
    seen = _recorded(nv, monkeypatch)
    r = torch.arange(rows * ld, dtype=torch.float32).view(rows, ld).as_subclass(OnGpu)[:, :64]
    was = r.clone()
    _, stream = nv.rms_norm(torch.zeros(rows, 64).as_subclass(OnGpu), torch.zeros(64).as_subclass(OnGpu), 1e-6, residual=r)
    d = struct.unpack("PiqPPiqPiffPiqP", seen["nvfp4_rms_norm"][0])
    assert stream.shape == r.shape and stream.untyped_storage().nbytes() <= 2 * rows * 64 * 4
    assert d[4] == stream.data_ptr() != r.data_ptr() and d[6] == (ld if alike else 64)
    assert (d[3] == r.data_ptr()) == (alike or rows == 1)
    if d[3] == d[4]:
        assert torch.equal(stream, was)  # what the call reads is the residual's values
    assert torch.equal(r, was)
