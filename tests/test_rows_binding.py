"""CPU tests of what the binding of the norm, the 8-bit rows and product and the log probabilities refuses
and hands on: devices, shapes, types, strides, empty calls."""
import contextlib
import os
import types

import pytest


@pytest.fixture(scope="module")
def nv():
    import nvfp4_weight_streaming_amd as nv
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_weight_streaming_amd import build as b
        b.build()
    nv.lib()
    return nv


def _gpu_class():
    import torch

    class OnGpu(torch.Tensor):
        def get_device(self):
            return 0

    return OnGpu


def _calls(nv, put):
    """(name, function, arguments) of every call, each tensor passed through `put`."""
    import torch
    bf16 = lambda *s: put(torch.zeros(s, dtype=torch.bfloat16))  # noqa: E731
    f32 = lambda *s: put(torch.zeros(s))  # noqa: E731
    i8 = lambda *s: put(torch.zeros(s, dtype=torch.int8))  # noqa: E731
    w = nv.Int8Weight(i8(64 * 128), f32(48), 64, 48)
    return [
        ("rms_norm", nv.rms_norm, dict(x=bf16(3, 64), weight=bf16(64), eps=1e-6, residual=f32(3, 64), out=bf16(3, 64), residual_out=f32(3, 64))),
        ("int8_quantize", nv.int8_quantize, dict(x=bf16(3, 64), codes=i8(3, 64))),
        ("int8_gemm", nv.int8_gemm, dict(codes=i8(3, 64), scale=f32(3), weight=w, bias=f32(48), out=bf16(3, 48))),
        ("logprobs", nv.logprobs, dict(logits=f32(3, 100), tokens=put(torch.zeros((3, 2), dtype=torch.int32)), k=4)),
        ("from_canonical", nv.Int8Weight.from_canonical, dict(codes=i8(48, 64), scale=f32(48))),
    ]


def _recorded(nv, monkeypatch):
    """Entry points that note their arguments and do nothing."""
    seen = {}
    sizes = {n: getattr(nv.lib(), n) for n in nv.EXPORTS if n.endswith("_bytes")}
    calls = {n: (lambda *a, n=n: seen.__setitem__(n, a) or 0) for n in nv.EXPORTS if not n.endswith("_bytes")}
    monkeypatch.setattr(nv, "_lib", types.SimpleNamespace(**{**calls, **sizes}))
    return seen


def test_host_tensors_are_refused(nv, monkeypatch):
    """Each argument of each call left in host memory beside others on a GPU, and all of them."""
    import torch
    OnGpu = _gpu_class()
    seen = _recorded(nv, monkeypatch)
    for name, f, args in _calls(nv, lambda x: x):
        with pytest.raises(nv.Nvfp4Error, match="not a matrix on a GPU"):
            f(**args)
    for name, f, args in _calls(nv, lambda x: x.as_subclass(OnGpu)):
        f(**args)
        tensors = [n for n, x in args.items() if isinstance(x, torch.Tensor)]
        for n in tensors:
            seen.clear()
            with pytest.raises(nv.Nvfp4Error, match="GPU") as e:
                f(**{**args, n: args[n].as_subclass(torch.Tensor)})
            # (a first argument off the GPU makes the call one of no GPU, and the next is named)
            assert not seen and (e.value.message.startswith(n + ":") or n == tensors[0]), (name, n, e.value.message)
    w = nv.Int8Weight(torch.zeros(64 * 128, dtype=torch.int8), torch.zeros(48), 64, 48)
    a = dict(_calls(nv, lambda x: x.as_subclass(OnGpu))[2][2], weight=w)
    with pytest.raises(nv.Nvfp4Error, match="weight: not on the call's GPU"):
        nv.int8_gemm(**a)


def test_shapes_and_types_are_refused(nv, monkeypatch):
    import torch
    OnGpu = _gpu_class()
    seen = _recorded(nv, monkeypatch)
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype).as_subclass(OnGpu)  # noqa: E731
    calls = {n: (f, a) for n, f, a in _calls(nv, lambda x: x.as_subclass(OnGpu))}
    i8, f32, f64, f16 = torch.int8, torch.float32, torch.float64, torch.float16
    for name, word, bad in [
            ("rms_norm", "x:", dict(x=t(64))), ("rms_norm", "x:", dict(x=t(3, 64, dtype=f16))), ("rms_norm", "x:", dict(x=t(64, 3).t())),
            ("rms_norm", "weight:", dict(weight=t(63))), ("rms_norm", "weight:", dict(weight=t(64, dtype=f64))),
            ("rms_norm", "weight:", dict(weight=t(128)[::2])), ("rms_norm", "dtype:", dict(dtype=f64)),
            ("rms_norm", "out:", dict(out=t(3, 65))), ("rms_norm", "out:", dict(out=t(3, 64, dtype=f32))),
            ("rms_norm", "out:", dict(out=t(3, 64), dtype=i8)), ("rms_norm", "residual:", dict(residual=t(2, 64))),
            ("rms_norm", "residual:", dict(residual=t(3, 64, dtype=i8))), ("rms_norm", "residual_out:", dict(residual_out=t(3, 64))),
            ("rms_norm", "residual_out:", dict(residual_out=t(3, 72, dtype=f32)[:, :64])),
            ("rms_norm", "residual_out:", dict(residual=None)),
            ("int8_quantize", "x:", dict(x=t(3, 64, dtype=i8))), ("int8_quantize", "x:", dict(x=t(3, 63), swiglu=True)),
            ("int8_quantize", "codes:", dict(swiglu=True)), ("int8_quantize", "codes:", dict(codes=t(3, 64))),
            ("int8_gemm", "codes:", dict(codes=t(3, 48, dtype=i8))), ("int8_gemm", "codes:", dict(codes=t(3, 64))),
            ("int8_gemm", "scale:", dict(scale=t(2, dtype=f32))), ("int8_gemm", "bias:", dict(bias=t(48))), ("int8_gemm", "dtype:", dict(dtype=i8)),
            ("int8_gemm", "out:", dict(out=t(3, 47))), ("int8_gemm", "out:", dict(out=t(3, 48), dtype=f32)),
            ("logprobs", "logits:", dict(logits=t(3, 100, dtype=f16))), ("logprobs", "tokens:", dict(tokens=t(3, 2))),
            ("logprobs", "tokens:", dict(tokens=t(2, dtype=torch.int32))), ("logprobs", "tokens:", dict(tokens=t(3, 1, 1, dtype=torch.int32))),
            ("from_canonical", "codes:", dict(codes=t(48, 80, dtype=i8)[:, :64])), ("from_canonical", "scale:", dict(scale=t(47, dtype=f32)))]:
        f, args = calls[name]
        seen.clear()
        with pytest.raises(nv.Nvfp4Error) as e:
            f(**{**args, **bad})
        assert e.value.message.startswith(word) and not seen, (name, bad.keys(), e.value.message)


def test_strides_are_handed_on(nv, monkeypatch):
    """Rows apart by their stride; the stride of a single row, which is never used, by its columns."""
    import struct

    import torch
    OnGpu = _gpu_class()
    seen = _recorded(nv, monkeypatch)
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype).as_subclass(OnGpu)  # noqa: E731
    layout = "PiqPPiqPiffPiqP"
    for rows, lds in ((3, (80, 72, 100)), (1, (64, 64, 64))):
        x, r, o = t(rows, 80)[:, :64], t(rows, 72, dtype=torch.float32)[:, :64], t(rows, 100)[:, :64]
        nv.rms_norm(x, t(64), 0.5, residual=r, residual_out=r, out=o, weight_offset=1.0)
        d = struct.unpack(layout, seen["nvfp4_rms_norm"][0])
        assert (d[2], d[6], d[13]) == lds and d[0] == x.data_ptr() and d[3] == d[4] == r.data_ptr() and d[9:11] == (1.0, 0.5)
        _, stream = nv.rms_norm(x, t(64), 0.5, residual=r)
        d = struct.unpack(layout, seen["nvfp4_rms_norm"][0])
        assert d[6] == lds[1] and d[4] == stream.data_ptr() != r.data_ptr() and stream.shape == r.shape
        q = t(rows, 96, dtype=torch.int8)[:, :64]
        nv.int8_quantize(x, codes=q)
        a = seen["nvfp4_int8_quantize"]
        assert (a[2], a[7]) == ((80, 96) if rows > 1 else (64, 64))
        w = nv.Int8Weight(t(64 * 128, dtype=torch.int8), t(48, dtype=torch.float32), 64, 48)
        nv.int8_gemm(q, t(rows, dtype=torch.float32), w, out=t(rows, 51)[:, :48])
        a = seen["nvfp4_int8_gemm"]
        assert (a[1], a[11]) == ((96, 51) if rows > 1 else (64, 48))
        nv.logprobs(t(rows, 107)[:, :100], t(rows, dtype=torch.int32))
        assert seen["nvfp4_logprobs"][2] == (107 if rows > 1 else 100)


def test_calls_of_no_rows(nv):
    """Empty tensors have no address: such calls return empty outputs and launch nothing."""
    import torch
    OnGpu = _gpu_class()
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype).as_subclass(OnGpu)  # noqa: E731
    out, stream = nv.rms_norm(t(0, 64), t(64), 1e-6, residual=t(0, 64))
    assert tuple(out.shape) == tuple(stream.shape) == (0, 64)
    codes, scale = nv.int8_quantize(t(0, 64), swiglu=True)
    assert tuple(codes.shape) == (0, 32) and tuple(scale.shape) == (0,)
    w = nv.Int8Weight(t(64 * 128, dtype=torch.int8), t(48, dtype=torch.float32), 64, 48)
    assert tuple(nv.int8_gemm(t(0, 64, dtype=torch.int8), t(0, dtype=torch.float32), w).shape) == (0, 48)
    lp, entropy, token, top = nv.logprobs(t(0, 100), t(0, 2, dtype=torch.int32), k=3)
    assert tuple(lp.shape) == (0, 2) and tuple(entropy.shape) == (0,) and tuple(token.shape) == tuple(top.shape) == (0, 3)
    with pytest.raises(nv.Nvfp4Error, match="k"):
        nv.logprobs(t(3, 100), t(3, dtype=torch.int32), k=65)
    with pytest.raises(nv.Nvfp4Error, match="k"):
        nv.logprobs(t(3, 100), t(3, dtype=torch.int32), k=-1)


def test_the_tensors_device_is_made_current(nv, monkeypatch):
    import torch
    OnGpu = _gpu_class()
    seen, state = _recorded(nv, monkeypatch), dict(device=1, entered=[])

    @contextlib.contextmanager
    def on_device(gpu):
        was, state["device"] = state["device"], gpu
        state["entered"].append(gpu)
        yield
        state["device"] = was

    T = nv._torch()
    monkeypatch.setattr(T, "device", lambda: state["device"])
    monkeypatch.setattr(T, "on_device", on_device)
    for name, f, args in _calls(nv, lambda x: x.as_subclass(OnGpu)):
        state["entered"].clear()
        seen.clear()
        f(**args)
        assert state == dict(device=1, entered=[0]) and len(seen) == 1, name


def test_a_weight_of_other_sizes_is_refused(nv):
    import torch
    packed, scale = torch.zeros(64 * 128, dtype=torch.int8), torch.zeros(48)
    nv.Int8Weight(packed[:48 * 128], scale, 64, 48)
    nv.Int8Weight(packed, scale, 64, 48)
    for bad, word in (((packed[:47 * 128], scale, 64, 48), "packed"), ((packed[:48 * 128], scale, 144, 48), "packed"),
                      ((packed[:48 * 128].view(torch.uint8), scale, 64, 48), "packed"), ((packed[::2][:48 * 128], scale, 64, 48), "packed"),
                      ((packed[:48 * 128], scale[:47], 64, 48), "scale"), ((packed[:48 * 128], scale.double(), 64, 48), "scale"),
                      ((packed[:48 * 128], torch.zeros((48, 2))[:, 0], 64, 48), "scale"), ((packed, scale, 24, 48), "K, N"), ((packed, scale, 64, 0), "K, N")):
        with pytest.raises(nv.Nvfp4Error, match="^.*" + word):
            nv.Int8Weight(*bad)


def test_sizes_past_a_c_integer_are_refused(nv, monkeypatch):
    """Shapes alone: storage of one value, told to be larger."""
    import torch
    OnGpu = _gpu_class()
    seen = _recorded(nv, monkeypatch)
    tall = lambda t: torch.zeros(1, dtype=t).as_strided((2 ** 32 + 1, 1), (0, 1)).as_subclass(OnGpu)  # noqa: E731
    wide = lambda t: torch.zeros(1, dtype=t).as_strided((1, 2 ** 32 + 16), (0, 0)).as_subclass(OnGpu)  # noqa: E731
    put = lambda x: x.as_subclass(OnGpu)  # noqa: E731
    one = put(torch.zeros(1))
    w = nv.Int8Weight(put(torch.zeros(16 * 128, dtype=torch.int8)), one, 16, 1)
    tokens = put(torch.zeros((1, 1), dtype=torch.int32))
    for f in (lambda: nv.rms_norm(tall(torch.float32), one, 1e-6), lambda: nv.int8_quantize(tall(torch.bfloat16)),
              lambda: nv.int8_gemm(tall(torch.int8), one, w), lambda: nv.logprobs(tall(torch.float32), tokens),
              lambda: nv.Int8Weight.from_canonical(tall(torch.int8), one),
              lambda: nv.logprobs(put(torch.zeros((1, 100))), torch.zeros(1, dtype=torch.int32).as_strided((1, 2 ** 32 + 1), (0, 0)).as_subclass(OnGpu)),
              lambda: nv.logprobs(put(torch.zeros((1, 100))), tokens, k=2 ** 32 + 4)):
        with pytest.raises(nv.Nvfp4Error):
            f()
    with pytest.raises(nv.Nvfp4Error):
        nv.int8_quantize(wide(torch.float32))
    assert not seen
