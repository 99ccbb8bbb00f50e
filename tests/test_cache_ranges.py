"""CPU tests of the paged cache's entry points at the ends of their arguments' ranges."""
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


P = 0x1000  # a well-aligned pointer that is never followed


def _cache(nv, **kw):
    d = dict(k_dev=P, v_dev=P, layers=2, pages=10, kv_heads=4, page_tokens=64, head_dim=128, dtype=0, k_scale=1.0,
             v_scale=1.0, page_stride=0, layer_stride=0)
    d.update(kw)
    return nv.Cache(**d)


@pytest.mark.parametrize("scale,k_scale,ok", [(0.1, 1.0, True), (1e-30, 1e-20, False), (1e30, 1e30, False), (1e-20, 1e-18, True),
                                              (1e-19, 1e-18, True), (1e30, 1e8, True)])
def test_scales_whose_product_is_no_number(nv, scale, k_scale, ok):
    """The kernel multiplies by scale x k_scale: 0 or infinity would make masked scores NaN."""
    f = lambda: nv.nvfp4_tree_attention(_cache(nv, dtype=1, k_scale=k_scale), 0, P, 1024, 8, 0, 2, 8, P, P, P, 4, P, scale, P, 1024,  # noqa: E731
                                        None, P, 1 << 40, stream=0)
    if ok:
        f()  # of no rows: nothing is launched
        return
    with pytest.raises(nv.Nvfp4Error) as e:
        f()
    assert e.value.status == nv.EINVAL and e.value.message.startswith("scale")


@pytest.mark.parametrize("lanes,width", [(65535, 32769), (1 << 15, 1 << 16), (2, 1 << 30)])
def test_updates_of_too_many_entries(nv, lanes, width):
    """Requests for pages are counted in 32 bits: tables of 2^31 entries or more are refused."""
    c = _cache(nv, page_tokens=16)
    width = min(width, 1 << 26)
    args = lambda w: (c, 2, P, P, P, w, lanes, P, None, None, 2 * P, 2 * P, 2 * P, P, P, 10)  # noqa: E731
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.nvfp4_cache_update(*args(width), stream=0)
    if lanes * width < 2 ** 31:
        assert e.value.message.startswith("workspace_bytes")  # (the next check: nothing is launched)
        return
    assert e.value.status == nv.EUNSUPPORTED and e.value.message.startswith("lanes_out")
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.nvfp4_cache_update(*args((2 ** 31 - 1) // lanes), stream=0)
    assert e.value.message.startswith("workspace_bytes")


def test_calls_of_more_threads_than_a_launch_has(nv):
    """A launch takes fewer than 2^32 threads: what needs more is refused, not cut off."""
    rot = nv.Rotary(positions_dev=P, inv_freq_dev=P, pair_axis_dev=None, axes=1, pairs=0, interleaved=0, factor=1.0)
    c = _cache(nv, head_dim=64, kv_heads=1)
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.nvfp4_cache_append(c, 0, P, 192, 1 << 24, 1, 2, P, P, P, 4, rot, P, 64, stream=0)
    assert e.value.status == nv.EUNSUPPORTED and e.value.message.startswith("rows")
    c = _cache(nv, kv_heads=1024)
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.nvfp4_cache_compact(c, 1 << 15, P, P, 4, P, 8, P, stream=0)
    assert e.value.status == nv.EUNSUPPORTED and e.value.message.startswith("lanes")
