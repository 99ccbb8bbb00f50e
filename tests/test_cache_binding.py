"""CPU tests of what the paged cache's binding refuses and accepts beyond shapes and types: memory
that is shared between layers, tensors of another device, empty calls."""
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


def _kv(layers=3, pages=5, heads=2, page=32, dim=64):
    import torch
    return (torch.zeros((layers, pages, heads, page, dim), dtype=torch.bfloat16),
            torch.zeros((layers, pages, heads, page // 16, dim, 16), dtype=torch.bfloat16))


@pytest.mark.parametrize("one", [dict(layers=1), dict(pages=1)], ids=str)
def test_expanded_layers_or_pages_are_refused(nv, one):
    """A stride of 0 would be taken for "dense": layers or pages past the first lie outside the tensors."""
    k, v = _kv(**one)
    nv.PagedCache(k, v)
    with pytest.raises(nv.Nvfp4Error, match="share memory"):
        nv.PagedCache(k.expand(3, 5, -1, -1, -1), v.expand(3, 5, -1, -1, -1, -1))


def test_layers_between_pages_are_taken(nv):
    """[pages][layers] in memory: real strides, handed on as they are."""
    k, v = _kv(layers=5, pages=3)
    c = nv.PagedCache(k.transpose(0, 1), v.transpose(0, 1))
    assert (c.desc.page_stride, c.desc.layer_stride) == (3 * 2 * 32 * 64 * 2, 2 * 32 * 64 * 2)
