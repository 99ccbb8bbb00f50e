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


def _calls(nv, put):
    """(name, function, arguments) of every call on a cache, each tensor passed through `put`."""
    import torch
    i32 = lambda *s: put(torch.zeros(s, dtype=torch.int32))  # noqa: E731
    bf16 = lambda *s: put(torch.zeros(s, dtype=torch.bfloat16))  # noqa: E731
    cache = nv.PagedCache(*(put(x) for x in _kv()))
    lanes = dict(row_start=i32(3), ctx_len=i32(2), page_table=i32(2, 4))
    logits = put(torch.zeros((4, 10)))
    return [
        ("append", cache.append, dict(layer=0, qkv=bf16(3, 512), q_heads=4, **lanes, positions=i32(3, 2), inv_freq=put(torch.zeros(32)),
                                      pair_axis=put(torch.zeros(32, dtype=torch.uint8)), out=bf16(3, 256))),
        ("attend", cache.attend, dict(layer=0, q=bf16(3, 256), **lanes, mask=put(torch.zeros(3, dtype=torch.int64)), max_rows=2, scale=0.1,
                                      out=bf16(3, 256))),
        ("compact", cache.compact, dict(ctx_len=i32(2), page_table=i32(2, 4), path=i32(2, 4), accepted=i32(2))),
        ("update", cache.update, dict(page_table=i32(2, 4), length=i32(2), refs=i32(5), parent=i32(2), keep=i32(2), reserve=i32(2))),
        ("beam_select", nv.beam_select, dict(logits=logits, beams=2, score=put(torch.zeros(4)), k=2, done=put(torch.zeros(4, dtype=torch.uint8)),
                                             eos=1)),
    ]


def _never(nv, monkeypatch):
    """No entry point may be reached: host tensors must not come as far as a kernel."""
    import types
    sizes = {n: getattr(nv.lib(), n) for n in nv.EXPORTS if n.endswith("_bytes")}
    monkeypatch.setattr(nv, "_lib", types.SimpleNamespace(**sizes))


def test_host_tensors_are_refused(nv, monkeypatch):
    """Each argument of each call left in host memory beside others on a GPU, and all of them."""
    import torch

    class OnGpu(torch.Tensor):
        def get_device(self):
            return 0

    _never(nv, monkeypatch)
    for name, f, args in _calls(nv, lambda x: x):
        with pytest.raises(nv.Nvfp4Error, match="not on a GPU"):
            f(**args)
    for name, f, args in _calls(nv, lambda x: x.as_subclass(OnGpu)):
        tensors = [n for n, x in args.items() if isinstance(x, torch.Tensor)]
        assert len(tensors) >= 3
        for n in tensors:
            with pytest.raises(nv.Nvfp4Error, match="GPU") as e:
                f(**{**args, n: args[n].as_subclass(torch.Tensor)})
            assert e.value.message.startswith(n + ":"), (name, n, e.value.message)


def test_k_and_v_on_one_device(nv):
    import torch
    k, v = _kv()
    with pytest.raises(nv.Nvfp4Error, match="not on k's device"):
        nv.PagedCache(k, torch.empty_like(v, device="meta"))


def test_calls_of_no_rows(nv):
    """Empty tensors have no address: such calls return empty outputs and launch nothing."""
    import torch

    class OnGpu(torch.Tensor):
        def get_device(self):
            return 0

    def t(*s, dtype=torch.int32):
        return torch.zeros(s, dtype=dtype).as_subclass(OnGpu)

    cache = nv.PagedCache(*(x.as_subclass(OnGpu) for x in _kv()))
    lanes = t(3), t(2), t(2, 4)
    bf16 = torch.bfloat16
    assert t(0, 512, dtype=bf16).data_ptr() == 0
    q = cache.append(0, t(0, 512, dtype=bf16), 4, *lanes, t(0, 2), t(32, dtype=torch.float32))
    assert tuple(q.shape) == (0, 256)
    for most in (0, 1, 8):
        out, lse = cache.attend(0, t(0, 256, dtype=bf16), *lanes, t(0, dtype=torch.int64), most, 0.1, with_lse=True)
        assert tuple(out.shape) == (0, 256) and tuple(lse.shape) == (0, 4)
    with pytest.raises(nv.Nvfp4Error, match="max_rows"):
        cache.attend(0, t(0, 256, dtype=bf16), *lanes, t(0, dtype=torch.int64), 65, 0.1)
    with pytest.raises(nv.Nvfp4Error, match="layer"):
        cache.append(3, t(0, 512, dtype=bf16), 4, *lanes, t(0, 2), t(32, dtype=torch.float32))


def test_single_rows_of_any_stride(nv, monkeypatch):
    """The stride of a tensor of one row is never used: rows cut from wider ones of odd width are taken."""
    import torch
    import types

    class OnGpu(torch.Tensor):
        def get_device(self):
            return 0

    seen = {}
    sizes = {n: getattr(nv.lib(), n) for n in nv.EXPORTS if n.endswith("_bytes")}
    calls = {n: (lambda *a, n=n: seen.__setitem__(n, a) or 0) for n in ("nvfp4_cache_append", "nvfp4_tree_attention")}
    monkeypatch.setattr(nv, "_lib", types.SimpleNamespace(**sizes, **calls))

    def t(*s, dtype=torch.int32):
        return torch.zeros(s, dtype=dtype).as_subclass(OnGpu)

    cache = nv.PagedCache(*(x.as_subclass(OnGpu) for x in _kv()))
    wide, bf16 = t(4, 519, dtype=torch.bfloat16), torch.bfloat16
    lanes = t(2), t(1), t(1, 4)
    for out in (None, wide[:1, :256], wide[:1]):
        cache.append(0, wide[:1, :512], 4, *lanes, t(1, 1), t(32, dtype=torch.float32), out=out)
        assert (seen["nvfp4_cache_append"][3], seen["nvfp4_cache_append"][13]) == (512, 256)
        cache.attend(0, wide[:1, :256], *lanes, t(1, dtype=torch.int64), 1, 0.1, out=out)
        assert (seen["nvfp4_tree_attention"][3], seen["nvfp4_tree_attention"][15]) == (256, 256)
    cache.append(0, wide[:2, :512], 4, t(2), t(1), t(1, 4), t(2, 1), t(32, dtype=torch.float32), out=wide[:, :256])
    assert (seen["nvfp4_cache_append"][3], seen["nvfp4_cache_append"][13]) == (519, 519)
    cache.attend(0, wide[:2, :256], *lanes, t(2, dtype=torch.int64), 1, 0.1, out=t(2, 300, dtype=bf16))
    assert (seen["nvfp4_tree_attention"][3], seen["nvfp4_tree_attention"][15]) == (519, 300)
