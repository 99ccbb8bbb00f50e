"""CPU tests of the paged-cache and beam entry points: what they refuse, naming the parameter,
before any HIP call; workspace sizes; mask words of a tree."""
import ctypes
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


def _refused(nv, word, status, f, *a):
    with pytest.raises(nv.Nvfp4Error) as e:
        f(*a)
    assert e.value.status == status and e.value.message.startswith(word), (e.value.message, word)


BAD_CACHES = [(dict(layers=0), "cache.layers", 1), (dict(pages=0), "cache.pages", 1), (dict(kv_heads=0), "cache.kv_heads", 1),
              (dict(kv_heads=2000), "cache.kv_heads", 1), (dict(head_dim=96), "cache.head_dim", 2), (dict(page_tokens=8), "cache.page_tokens", 2),
              (dict(page_tokens=48), "cache.page_tokens", 2), (dict(page_tokens=512), "cache.page_tokens", 2), (dict(dtype=2), "cache.dtype", 1),
              (dict(dtype=1, k_scale=0.0), "cache.k_scale", 1), (dict(dtype=1, v_scale=float("nan")), "cache.k_scale", 1),
              (dict(k_dev=None), "cache.k", 1), (dict(v_dev=P + 8), "cache.v", 1), (dict(page_stride=100), "cache.page_stride", 1),
              (dict(page_stride=65536 * 4 + 8), "cache.page_stride", 1), (dict(layer_stride=16), "cache.layer_stride", 1)]


def _attend(nv, c, **kw):
    d = dict(layer=0, q=P, q_ld=1024, q_heads=8, rows=8, lanes=2, max_rows=8, row_start=P, ctx_len=P, page_table=P, table_ld=4, mask=P,
             scale=0.1, out=P, out_ld=1024, lse=None, workspace=P, workspace_bytes=1 << 40)
    d.update(kw)
    return nv.nvfp4_tree_attention(c, *d.values(), stream=0)


def _append(nv, c, rot=None, **kw):
    r = dict(positions_dev=P, inv_freq_dev=P, pair_axis_dev=None, axes=1, pairs=64, interleaved=0, factor=1.0)
    r.update(rot or {})
    d = dict(layer=0, qkv=P, qkv_ld=2048, rows=8, q_heads=8, lanes=2, row_start=P, ctx_len=P, page_table=P, table_ld=4,
             rotary=nv.Rotary(**r), q_out=P, q_ld=1024)
    d.update(kw)
    return nv.nvfp4_cache_append(c, *d.values(), stream=0)


def _compact(nv, c, **kw):
    d = dict(lanes=2, ctx_len=P, page_table=P, table_ld=4, path=P, path_ld=8, accepted=P)
    d.update(kw)
    return nv.nvfp4_cache_compact(c, *d.values(), stream=0)


def _update(nv, c, **kw):
    d = dict(lanes_in=2, table_in=P, len_in=P, refs_in=P, table_ld=4, lanes_out=3, parent=P, keep=None, reserve=None,
             table_out=2 * P, len_out=2 * P, refs_out=2 * P, short=P, workspace=P, workspace_bytes=1 << 40)
    d.update(kw)
    return nv.nvfp4_cache_update(c, *d.values(), stream=0)


@pytest.mark.parametrize("bad,word,status", BAD_CACHES, ids=lambda x: str(x))
def test_caches_are_checked(nv, bad, word, status):
    for f in (_attend, _append, _compact, _update):
        _refused(nv, word, status, lambda: f(nv, _cache(nv, **bad)))


def test_null_cache(nv):
    L = nv.lib()
    assert L.nvfp4_cache_compact(None, 1, P, P, 1, P, 1, P, None) == nv.EINVAL and nv.last_error().startswith("cache")


@pytest.mark.parametrize("bad,word", [
    (dict(layer=2), "layer"), (dict(layer=-1), "layer"), (dict(q_heads=6), "q_heads"), (dict(q_heads=0), "q_heads"), (dict(max_rows=0), "max_rows"),
    (dict(max_rows=65), "max_rows"), (dict(rows=-1), "rows"), (dict(rows=1 << 25), "rows"), (dict(lanes=0), "lanes"), (dict(lanes=70000), "lanes"), (dict(table_ld=0), "table_ld"),
    (dict(table_ld=1 << 25), "table_ld"), (dict(page_table=None), "page_table"), (dict(page_table=P + 2), "page_table"),
    (dict(q_ld=1016), "q_ld"), (dict(q_ld=1028), "q_ld"), (dict(out_ld=1022), "out_ld"), (dict(out_ld=1026), "out_ld"),
    (dict(q=None), "q"), (dict(q=P + 8), "q"), (dict(out=P + 4), "out"), (dict(out=None), "out"), (dict(row_start=None), "row_start"),
    (dict(ctx_len=P + 1), "ctx_len"), (dict(mask=P + 4), "mask"), (dict(lse=P + 2), "lse"), (dict(scale=0.0), "scale"),
    (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"), (dict(workspace_bytes=1000), "workspace_bytes"),
    (dict(workspace=None), "workspace"), (dict(workspace=P + 4), "workspace")], ids=lambda x: str(x))
def test_attention_refuses(nv, bad, word):
    _refused(nv, word, nv.EINVAL, lambda: _attend(nv, _cache(nv), **bad))


@pytest.mark.parametrize("bad,rot,word", [
    (dict(layer=-1), {}, "layer"), (dict(rows=-1), {}, "rows"), (dict(q_heads=0), {}, "q_heads"), (dict(qkv_ld=2044), {}, "qkv_ld"), (dict(qkv_ld=2050), {}, "qkv_ld"),
    (dict(q_ld=1020), {}, "q_ld"), (dict(qkv=P + 4), {}, "qkv"), (dict(q_out=None), {}, "q_out"), (dict(row_start=P + 1), {}, "row_start"),
    (dict(ctx_len=None), {}, "ctx_len"), (dict(lanes=0), {}, "lanes"), (dict(table_ld=-3), {}, "table_ld"),
    ({}, dict(pairs=68), "rotary.pairs"), ({}, dict(pairs=6), "rotary.pairs"), ({}, dict(pairs=-4), "rotary.pairs"), ({}, dict(axes=0), "rotary.axes"),
    ({}, dict(axes=9), "rotary.axes"), ({}, dict(positions_dev=None), "rotary.positions"), ({}, dict(inv_freq_dev=P + 2), "rotary.inv_freq")], ids=lambda x: str(x))
def test_append_refuses(nv, bad, rot, word):
    _refused(nv, word, nv.EINVAL, lambda: _append(nv, _cache(nv), rot, **bad))


def test_append_of_no_rows_launches_nothing(nv):
    _append(nv, _cache(nv), rows=0)


@pytest.mark.parametrize("bad,word", [
    (dict(lanes=0), "lanes"), (dict(table_ld=0), "table_ld"), (dict(path_ld=0), "path_ld"), (dict(path=None), "path"), (dict(ctx_len=P + 2), "ctx_len"),
    (dict(accepted=None), "accepted")], ids=lambda x: str(x))
def test_compact_refuses(nv, bad, word):
    _refused(nv, word, nv.EINVAL, lambda: _compact(nv, _cache(nv), **bad))


@pytest.mark.parametrize("bad,word", [
    (dict(lanes_in=0), "lanes"), (dict(lanes_out=0), "lanes_out"), (dict(table_in=None), "page_table"), (dict(len_in=None), "len_in"), (dict(refs_in=P + 1), "refs_in"),
    (dict(parent=None), "parent"), (dict(keep=P + 2), "keep"), (dict(reserve=P + 2), "reserve"), (dict(table_out=None), "table_out"), (dict(table_out=P), "table_out"),
    (dict(len_out=P), "len_out"), (dict(refs_out=P), "refs_out"), (dict(short=None), "short"), (dict(workspace_bytes=10), "workspace_bytes"),
    (dict(workspace=None), "workspace")], ids=lambda x: str(x))
def test_update_refuses(nv, bad, word):
    _refused(nv, word, nv.EINVAL, lambda: _update(nv, _cache(nv), **bad))


@pytest.mark.parametrize("bad,word", [
    (dict(logits_dtype=2), "logits_dtype"), (dict(batch=0), "batch"), (dict(batch=65535), "batch"), (dict(beams=0), "beams"), (dict(beams=65), "beams"), (dict(V=0), "V"),
    (dict(V=1 << 30, ld=1 << 30), "V"), (dict(ld=999), "ld"), (dict(k=0), "k"), (dict(k=65), "k"), (dict(V=5, k=6), "k"), (dict(logits=None), "logits"),
    (dict(logits=P + 2), "logits"), (dict(score=None), "score"), (dict(score_out=P + 1), "score_out"), (dict(parent=None), "parent"), (dict(token=None), "token"),
    (dict(done=P, eos=-1), "eos"), (dict(done=P, eos=1000), "eos"), (dict(workspace_bytes=1), "workspace_bytes"), (dict(workspace=P + 8), "workspace")], ids=lambda x: str(x))
def test_beam_refuses(nv, bad, word):
    d = dict(logits=P, logits_dtype=0, ld=1000, batch=2, beams=4, V=1000, score=P, done=None, eos=-1, k=8, score_out=P, parent=P, token=P,
             done_out=None, workspace=P, workspace_bytes=1 << 40)
    d.update(bad)
    _refused(nv, word, nv.EINVAL, lambda: nv.nvfp4_beam_select(*d.values(), stream=0))


def test_workspace_sizes(nv):
    assert nv.nvfp4_beam_workspace_bytes(2, 4, 1025) == 2 * 4 * 2 * 8
    assert nv.nvfp4_beam_workspace_bytes(2, 65, 1025) == nv.nvfp4_beam_workspace_bytes(0, 1, 1) == 0
    assert nv.nvfp4_tree_attention_workspace_bytes(8, 3, 128, 1) == nv.nvfp4_tree_attention_workspace_bytes(8, 4, 100, 1) == 0
    assert nv.nvfp4_tree_attention_workspace_bytes(48, 4, 128, 64) > nv.nvfp4_tree_attention_workspace_bytes(48, 4, 128, 1) > 0
    assert nv.nvfp4_cache_update_workspace_bytes(100, 8, 10) >= 100 * 8 + 8 * 8 + 8 * 10 * 8
    assert nv.nvfp4_cache_update_workspace_bytes(0, 8, 10) == 0


def test_tree_mask(nv):
    mask, depth = nv.nvfp4_tree_mask([-1, 0, 0, 1, -1, 3])
    assert mask == [0b1, 0b11, 0b101, 0b1011, 0b10000, 0b101011] and depth == [0, 1, 1, 2, 0, 3]
    mask, depth = nv.nvfp4_tree_mask(list(range(-1, 63)))
    assert mask[:3] == [1, 3, 7] and mask[63] == -1 and depth[63] == 63
    for bad in ([], [0], [-2], [-1, 1], [-1] * 65):
        with pytest.raises(nv.Nvfp4Error):
            nv.nvfp4_tree_mask(bad)
    depth = (ctypes.c_int * 1)()
    assert nv.lib().nvfp4_tree_mask(None, 1, None, depth) == nv.EINVAL and "parent" in nv.last_error()


def test_the_binding_checks_tensors(nv):
    """Shapes, types and strides the C entry points cannot see."""
    import torch
    k, v = torch.zeros((2, 5, 4, 32, 64), dtype=torch.bfloat16), torch.zeros((2, 5, 4, 2, 64, 16), dtype=torch.bfloat16)
    nv.PagedCache(k, v)
    nv.PagedCache(k[:, ::2], v[:, ::2])
    for a, b in ((k.float(), v.float()), (k, v[:1]), (k, v.to(torch.float8_e4m3fn)), (k[:, ::2], v[:, :3]), (k.transpose(2, 3), v), (k[0], v[0])):
        with pytest.raises(nv.Nvfp4Error):
            nv.PagedCache(a, b)
    c = nv.PagedCache(k, v)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = dict(layer=0, q=torch.zeros((3, 512), dtype=torch.bfloat16), row_start=i32(3), ctx_len=i32(2), page_table=i32(2, 4), mask=torch.zeros(3, dtype=torch.int64), max_rows=2, scale=0.1)
    for bad in (dict(q=good["q"].float()), dict(q=good["q"].t()), dict(row_start=i32(2)), dict(ctx_len=torch.zeros(2)), dict(page_table=i32(3, 4)),
                dict(page_table=i32(2, 9)[:, :4]), dict(mask=i32(3)), dict(out=torch.zeros((2, 512), dtype=torch.bfloat16)), dict(out=torch.zeros((3, 256), dtype=torch.bfloat16))):
        with pytest.raises(nv.Nvfp4Error):
            c.attend(**{**good, **bad})
    for bad in (dict(refs=i32(4)), dict(parent=torch.zeros(2)), dict(keep=i32(3)), dict(length=i32(3))):
        with pytest.raises(nv.Nvfp4Error):
            c.update(**{**dict(page_table=i32(2, 4), length=i32(2), refs=i32(5), parent=i32(2)), **bad})
    for bad in (dict(path=i32(1, 4)), dict(path=torch.zeros((2, 4))), dict(accepted=i32(3))):
        with pytest.raises(nv.Nvfp4Error):
            c.compact(**{**dict(ctx_len=i32(2), page_table=i32(2, 4), path=i32(2, 4), accepted=i32(2)), **bad})
    ap = dict(layer=0, qkv=torch.zeros((3, 768), dtype=torch.bfloat16), q_heads=4, row_start=i32(3), ctx_len=i32(2), page_table=i32(2, 4), positions=i32(3, 2), inv_freq=torch.zeros(32))
    for bad in (dict(qkv=torch.zeros((3, 512), dtype=torch.bfloat16)), dict(positions=i32(2, 2)), dict(inv_freq=i32(32)), dict(pair_axis=i32(32)), dict(out=torch.zeros((2, 256), dtype=torch.bfloat16))):
        with pytest.raises(nv.Nvfp4Error):
            c.append(**{**ap, **bad})
    with pytest.raises(nv.Nvfp4Error):
        nv.beam_select(torch.zeros((4, 10), dtype=torch.float16), 2, torch.zeros(4), 2)
    with pytest.raises(nv.Nvfp4Error):
        nv.beam_select(torch.zeros((4, 10)), 3, torch.zeros(4), 2)
