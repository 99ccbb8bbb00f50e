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
