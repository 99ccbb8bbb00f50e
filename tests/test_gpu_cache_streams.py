"""Calls with a stream of the caller's, not torch's current one: what a call allocates must not go to
the current stream's next allocations while its kernels run elsewhere."""
import numpy as np
import pytest

from tests.cache_util import Lanes, cache_tensors, chain
from tests.gpu_util import dev, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


def _calls(nv):
    """name -> (entry point, function): every call that allocates."""
    import torch
    lanes = Lanes(13, [2000, 900, 30], [4, 2, 1], 64)
    k, v = cache_tensors(3, 2, lanes.pages, 2, 64, 128, "bf16")
    cache = nv.PagedCache(k, v)
    start, ctx, table = lanes.dev()
    g = torch.Generator(device="cuda").manual_seed(2)
    qkv = torch.randn((7, 12 * 128), generator=g, device="cuda").to(torch.bfloat16)
    q = qkv[:, :8 * 128].contiguous()
    masks = dev(np.concatenate([chain(x) for x in lanes.rows]))
    pos, inv = dev(np.arange(7, dtype=np.int32)[:, None]), dev(np.ones(64, np.float32))
    refs = dev(np.bincount(lanes.table[lanes.table >= 0], minlength=lanes.pages).astype(np.int32))
    parent = dev(np.array([2, 2, 1], np.int32))
    logits = torch.randn((8, 40000), generator=g, device="cuda")
    score = torch.zeros(8, device="cuda")
    return {
        "append": ("nvfp4_cache_append", lambda **s: [cache.append(0, qkv, 8, start, ctx, table, pos, inv, **s)]),
        "attend": ("nvfp4_tree_attention", lambda **s: list(cache.attend(1, q, start, ctx, table, masks, 4, 0.09, with_lse=True, **s))),
        "update": ("nvfp4_cache_update", lambda **s: list(cache.update(table, ctx, refs, parent, **s))),
        "beam_select": ("nvfp4_beam_select", lambda **s: list(nv.beam_select(logits, 4, score, 8, **s))),
        "topk": ("nvfp4_topk", lambda **s: list(nv.topk(logits, 8, **s))),
    }


@pytest.mark.parametrize("kind", ["stream", "handle"])
@pytest.mark.parametrize("name", ["append", "attend", "update", "beam_select", "topk"])
def test_a_stream_of_the_callers(nv, monkeypatch, name, kind):
    import torch
    entry, call = _calls(nv)[name]
    want = call()
    torch.cuda.synchronize()
    seen = []
    through = getattr(nv.lib(), entry)
    monkeypatch.setattr(nv._lib, entry, lambda *a: seen.append(a) or through(*a))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side if kind == "stream" else side.cuda_stream)
    args, = seen
    assert args[-1] == side.cuda_stream
    held = [(t.data_ptr(), t.numel() * t.element_size()) for t in got]
    if name != "append":
        held.append((args[-3], args[-2]))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    del got
    # the next allocations of these sizes on the current stream
    for at, n in held:
        for x in [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(8)]:
            assert x.data_ptr() + n <= at or at + n <= x.data_ptr(), (name, at, n)
    assert torch.cuda.current_stream() != side


def test_quantizing_on_a_stream_of_the_callers(nv, monkeypatch):
    """The tensor scale is read once that stream has written it, and the workspace stays its own."""
    import torch
    w = torch.randn((64, 1024), device="cuda")
    want = nv.PackedWeight.quantize(w, keep_canonical=True)
    seen = []
    through = nv.lib().nvfp4_quantize
    monkeypatch.setattr(nv._lib, "nvfp4_quantize", lambda *a: seen.append(a) or through(*a))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nv.PackedWeight.quantize(w, side, keep_canonical=True)
    assert got.tensor_scale == want.tensor_scale and seen[0][-1] == side.cuda_stream
    side.synchronize()
    for a, b in zip((want.codes, want.scales, *want.canonical), (got.codes, got.scales, *got.canonical)):
        assert torch.equal(a, b)
    n = nv.nvfp4_quantize_workspace_bytes()
    for x in [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(8)]:
        assert not any(isinstance(a, int) and x.data_ptr() <= a < x.data_ptr() + n for a in seen[0][3:-1])


def test_the_default_stream_by_handle(nv):
    import torch
    for name, (_, call) in _calls(nv).items():
        want = call()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = call(stream=0)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), name
