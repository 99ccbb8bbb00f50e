"""CPU tests of the norm, 8-bit and log-probability entry points: what they refuse, naming the parameter,
before any HIP call; sizes; calls of no rows."""
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
NAN, INF = float("nan"), float("inf")


def _refused(nv, word, f):
    with pytest.raises(nv.Nvfp4Error) as e:
        f()
    assert e.value.status == nv.EINVAL and e.value.message.startswith(word), (e.value.message, word)


def _norm(nv, rows=4, K=64, **kw):
    d = dict(x_dev=P, x_dtype=1, x_ld=64, residual_dev=P, residual_out_dev=P, residual_dtype=1, residual_ld=64, weight_dev=P, weight_dtype=1,
             weight_offset=0.0, eps=1e-6, out_dev=P, out_dtype=1, out_ld=64, scale_dev=None)
    d.update(kw)
    return nv.nvfp4_rms_norm(nv.Norm(**d), rows, K, stream=0)


def _quantize(nv, **kw):
    d = dict(x=P, x_dtype=1, x_ld=64, rows=4, K=64, swiglu=0, codes=P, codes_ld=64, scale=P)
    d.update(kw)
    return nv.nvfp4_int8_quantize(*d.values(), stream=0)


def _gemm(nv, **kw):
    d = dict(a=P, a_ld=64, a_scale=P, w_packed=P, w_scale=P, bias=P, M=4, K=64, N=16, out=P, out_dtype=1, out_ld=16, workspace=P,
             workspace_bytes=1 << 40)
    d.update(kw)
    return nv.nvfp4_int8_gemm(*d.values(), stream=0)


def _logprobs(nv, **kw):
    d = dict(logits=P, logits_dtype=0, ld=100, rows=4, V=100, scale=1.0, tokens=P, n_tokens=1, k=3, logprob=P, entropy=P, top_token=P,
             top_logprob=P, workspace=P, workspace_bytes=1 << 40)
    d.update(kw)
    return nv.nvfp4_logprobs(*d.values(), stream=0)


@pytest.mark.parametrize("bad,word", [
    (dict(rows=-1), "rows"), (dict(rows=1 << 22), "rows"), (dict(K=0), "K"), (dict(K=(1 << 24) + 1), "K"), (dict(x_dtype=2), "x_dtype"),
    (dict(x_dev=None), "x"), (dict(x_dev=P + 1), "x"), (dict(x_ld=63), "x_ld"), (dict(x_dtype=0, x_dev=P + 2), "x"),
    (dict(weight_dtype=3), "weight_dtype"), (dict(weight_dev=None), "weight"), (dict(out_dtype=3), "out_dtype"), (dict(out_dev=None), "out"),
    (dict(out_ld=10), "out_ld"), (dict(residual_dev=None), "residual"), (dict(residual_out_dev=None), "residual_out"),
    (dict(residual_dtype=2), "residual_dtype"), (dict(residual_ld=63), "residual_ld"), (dict(eps=-1.0), "eps"), (dict(eps=NAN), "eps"),
    (dict(weight_offset=NAN), "weight_offset"), (dict(out_dtype=2), "scale"), (dict(out_dtype=2, scale_dev=P + 1), "scale")], ids=str)
def test_norm_refuses(nv, bad, word):
    _refused(nv, word, lambda: _norm(nv, **bad))


def test_null_norm(nv):
    assert nv.lib().nvfp4_rms_norm(None, 1, 1, None) == nv.EINVAL and nv.last_error().startswith("norm")


@pytest.mark.parametrize("bad,word", [
    (dict(rows=-1), "rows"), (dict(rows=1 << 22), "rows"), (dict(K=0), "K"), (dict(K=(1 << 24) + 1), "K"), (dict(x_dtype=2), "x_dtype"),
    (dict(x=None), "x"), (dict(x=P + 1), "x"), (dict(x_ld=63), "x_ld"), (dict(swiglu=1), "x_ld"), (dict(swiglu=2), "swiglu"),
    (dict(codes=None), "codes"), (dict(codes_ld=63), "codes_ld"), (dict(scale=None), "scale"), (dict(scale=P + 2), "scale")], ids=str)
def test_quantize_refuses(nv, bad, word):
    _refused(nv, word, lambda: _quantize(nv, **bad))


@pytest.mark.parametrize("bad,word", [
    (dict(M=-1), "M"), (dict(M=(1 << 22) + 1), "M"), (dict(a_ld=(1 << 22) + 16), "a_ld"), (dict(K=0), "K"), (dict(K=24), "K"), (dict(K=131072), "K"), (dict(N=0), "N"), (dict(out_dtype=2), "out_dtype"),
    (dict(a_ld=48), "a_ld"), (dict(a_ld=72), "a_ld"), (dict(out_ld=15), "out_ld"), (dict(a=None), "a"), (dict(a=P + 8), "a"),
    (dict(a_scale=None), "a_scale"), (dict(w_packed=P + 8), "w_packed"), (dict(w_scale=None), "w_scale"), (dict(bias=P + 1), "bias"),
    (dict(out=None), "out"), (dict(out=P + 1), "out"), (dict(out_dtype=0, out=P + 2), "out")], ids=str)
def test_gemm_refuses(nv, bad, word):
    _refused(nv, word, lambda: _gemm(nv, **bad))


@pytest.mark.parametrize("bad,word", [
    (dict(logits_dtype=2), "logits_dtype"), (dict(V=0), "V"), (dict(V=(1 << 30) + 1), "V"), (dict(rows=-1), "rows"),
    (dict(rows=1 << 24), "rows"), (dict(ld=99), "ld"), (dict(scale=0.0), "scale"), (dict(scale=INF), "scale"), (dict(scale=NAN), "scale"),
    (dict(scale=-1.0), "scale"), (dict(n_tokens=-1), "n_tokens"), (dict(n_tokens=1025), "n_tokens"), (dict(k=-1), "k"), (dict(k=65), "k"),
    (dict(V=2, k=3), "k"), (dict(logits=None), "logits"), (dict(logits=P + 2), "logits"), (dict(tokens=None), "tokens"),
    (dict(logprob=None), "logprob"), (dict(entropy=P + 1), "entropy"), (dict(top_token=None), "top_token"),
    (dict(top_logprob=None), "top_logprob"), (dict(workspace=P + 8), "workspace"), (dict(workspace_bytes=64), "workspace_bytes")], ids=str)
def test_logprobs_refuses(nv, bad, word):
    _refused(nv, word, lambda: _logprobs(nv, **bad))


@pytest.mark.parametrize("K,N", [(16, 1), (64, 16), (80, 17), (5120, 152064)])
def test_packed_sizes(nv, K, N):
    assert nv.nvfp4_int8_packed_bytes(K, N) == -(-K // 128) * 128 * -(-N // 16) * 16


@pytest.mark.parametrize("K,N", [(0, 16), (8, 16), (24, 16), (16, 0), (-16, 4), (131072, 16)])
def test_packed_sizes_invalid(nv, K, N):
    assert nv.nvfp4_int8_packed_bytes(K, N) == 0
    for f in (nv.nvfp4_int8_pack, nv.nvfp4_int8_unpack):
        _refused(nv, "N" if N < 1 else "K", lambda: f(P, K, N, P, stream=0) if f is nv.nvfp4_int8_pack else f(P, K, N, P, stream=0))


def test_pack_refuses_pointers(nv):
    _refused(nv, "codes", lambda: nv.nvfp4_int8_pack(None, 64, 16, P, stream=0))
    _refused(nv, "packed", lambda: nv.nvfp4_int8_pack(P, 64, 16, P + 4, stream=0))
    _refused(nv, "packed", lambda: nv.nvfp4_int8_unpack(P + 4, 64, 16, P, stream=0))
    _refused(nv, "codes", lambda: nv.nvfp4_int8_unpack(P, 64, 16, None, stream=0))


def test_calls_of_no_rows(nv):
    """They look at no pointer of a row, and launch nothing."""
    _norm(nv, rows=0, x_dev=None, residual_dev=None, residual_out_dev=None, out_dev=None, weight_dev=None)
    _quantize(nv, rows=0, x=None, codes=None, scale=None)
    _gemm(nv, M=0, a=None, a_scale=None, out=None)
    _logprobs(nv, rows=0, logits=None, tokens=None, logprob=None, top_token=None, top_logprob=None, workspace=None, workspace_bytes=0)


def test_workspace_sizes(nv):
    assert nv.nvfp4_logprobs_workspace_bytes(0, 100, 1) == 0 and nv.nvfp4_logprobs_workspace_bytes(1, 100, 65) == 0
    assert nv.nvfp4_logprobs_workspace_bytes(1, 2, 3) == 0
    assert nv.nvfp4_logprobs_workspace_bytes(2, 4089, 0) == 2 * 16  # one unit, whatever the row's offset from 16 bytes
    assert nv.nvfp4_logprobs_workspace_bytes(2, 4090, 1) == 2 * 2 * (16 + 32)
    assert nv.nvfp4_int8_gemm_workspace_bytes(0, 64, 16) == 0 and nv.nvfp4_int8_gemm_workspace_bytes(4, 24, 16) == 0
    for M in (1, 8, 16):
        assert nv.nvfp4_int8_gemm_workspace_bytes(M, 5120, 152064) == 0


def test_structure_matches_the_header(nv):
    """Field by field: offsets as a C compiler lays them out."""
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = [n for n, _ in nv.Norm._fields_]
    src = '#include <stdio.h>\n#include "nvfp4.h"\nint main(void) {\n%s\nprintf("%%zu", sizeof(nvfp4_norm)); return 0; }\n' % "\n".join(
        'printf("%%zu ", offsetof(nvfp4_norm, %s));' % n for n in names)
    with tempfile.TemporaryDirectory() as d:
        open(os.path.join(d, "t.c"), "w").write(src)
        subprocess.check_call(["gcc", "-I", os.path.join(root, "include"), "-o", os.path.join(d, "t"), os.path.join(d, "t.c")])
        got = [int(v) for v in subprocess.check_output([os.path.join(d, "t")]).split()]
    assert got == [getattr(nv.Norm, n).offset for n in names] + [ctypes.sizeof(nv.Norm)]


def test_more_columns_than_an_index_holds(nv):
    """Tiles' ends stay within 32 bits."""
    big = (1 << 30) + 1
    _refused(nv, "N", lambda: _gemm(nv, N=big, out_ld=big))
    _refused(nv, "N", lambda: _gemm(nv, M=64, N=2 ** 31 - 1, out_ld=2 ** 31))
    _refused(nv, "N", lambda: nv.nvfp4_int8_pack(P, 64, big, P, stream=0))
    assert nv.nvfp4_int8_packed_bytes(64, big) == 0 and nv.nvfp4_int8_gemm_workspace_bytes(64, 64, big) == 0
    assert nv.nvfp4_int8_packed_bytes(16, 1 << 30) == 128 << 30
