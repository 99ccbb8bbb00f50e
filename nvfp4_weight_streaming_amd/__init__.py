"""Python binding of libnvfp4 (the MI355X NVFP4 weight-streaming GEMM).

Argument marshalling only: every computation runs in the HIP kernels of
``libnvfp4.so``; torch is used for device memory and streams.  The functions
carry the names of the C entry points declared in ``include/nvfp4.h``.
Tensors are passed by device pointer; a ``stream`` argument defaults to
torch's current stream.  A failing call raises ``Nvfp4Error`` with the
library's message (which names the offending parameter).

If ``libnvfp4.so`` is missing, importing works but the first call raises: there
is no fallback path of any kind.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4.so")

OK, EINVAL, EUNSUPPORTED, EHIP, ESTATE = 0, 1, 2, 3, 4
OUT_F32, OUT_BF16, OUT_INT8 = 0, 1, 2
PREFILL_AUTO, PREFILL_PIECES, PREFILL_STREAM_K = 0, 1, 2
DECODE_MAX_M = 8
VERIFY_MAX_M = 64

# Every symbol include/nvfp4.h declares.
EXPORTS = (
    "nvfp4_status_string", "nvfp4_last_error", "nvfp4_version",
    "nvfp4_packed_code_bytes", "nvfp4_packed_scale_bytes", "nvfp4_pack", "nvfp4_unpack",
    "nvfp4_quantize_workspace_bytes", "nvfp4_quantize",
    "nvfp4_gemm_create", "nvfp4_gemm_create_ex", "nvfp4_gemm_destroy", "nvfp4_gemm_run",
    "nvfp4_gemm_run_noalloc", "nvfp4_gemm_argmax_area_bytes", "nvfp4_gemm_run_argmax",
    "nvfp4_workspace_clear",
    "nvfp4_round_workspace_bytes", "nvfp4_round_create", "nvfp4_round_run",
    "nvfp4_round_graph_nodes", "nvfp4_round_destroy",
    "nvfp4_rms_norm", "nvfp4_int8_quantize", "nvfp4_int8_packed_bytes", "nvfp4_int8_pack",
    "nvfp4_int8_unpack", "nvfp4_int8_gemm_workspace_bytes", "nvfp4_int8_gemm",
    "nvfp4_topk_workspace_bytes", "nvfp4_topk", "nvfp4_swiglu", "nvfp4_stream_read",
    "nvfp4_cache_append", "nvfp4_cache_compact", "nvfp4_cache_update",
    "nvfp4_cache_update_workspace_bytes", "nvfp4_tree_mask", "nvfp4_tree_attention",
    "nvfp4_tree_attention_workspace_bytes", "nvfp4_beam_select", "nvfp4_beam_workspace_bytes",
    "nvfp4_logprobs_workspace_bytes", "nvfp4_logprobs",
)
TOPK_MAX_K = 64
TREE_MAX_ROWS = 64
BEAM_MAX_BEAMS = 64
ROW_MAX_K = 1 << 24
INT8_MAX_K = 131056
CACHE_BF16, CACHE_E4M3 = 0, 1


class Nvfp4Error(RuntimeError):
    def __init__(self, status, message):
        super().__init__("%s (status %d): %s" % (_STATUS.get(status, "?"), status, message))
        self.status = status
        self.message = message


_STATUS = {OK: "ok", EINVAL: "EINVAL", EUNSUPPORTED: "EUNSUPPORTED", EHIP: "EHIP",
           ESTATE: "ESTATE"}


class GemmConfig(ctypes.Structure):
    _fields_ = [("split_k", ctypes.c_int), ("waves", ctypes.c_int), ("chunks", ctypes.c_int),
                ("windows", ctypes.c_int), ("verify_waves", ctypes.c_int),
                ("verify_windows", ctypes.c_int), ("tile_max_m", ctypes.c_int),
                ("tile_superblocks", ctypes.c_int), ("verify_ranges", ctypes.c_int),
                ("prefill_schedule", ctypes.c_int)]


class Layer(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int), ("N", ctypes.c_int),
                ("codes_dev", ctypes.c_void_p), ("scales_dev", ctypes.c_void_p),
                ("tensor_scale", ctypes.c_float), ("act_dev", ctypes.c_void_p),
                ("out_dev", ctypes.c_void_p), ("out_dtype", ctypes.c_int),
                ("act_op", ctypes.c_int)]


ACT_INPUT, ACT_SWIGLU_PREV = 0, 1


class Cache(ctypes.Structure):
    _fields_ = [("k_dev", ctypes.c_void_p), ("v_dev", ctypes.c_void_p),
                ("layers", ctypes.c_int), ("pages", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("page_tokens", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("dtype", ctypes.c_int), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float), ("page_stride", ctypes.c_int64),
                ("layer_stride", ctypes.c_int64)]


class Rotary(ctypes.Structure):
    _fields_ = [("positions_dev", ctypes.c_void_p), ("inv_freq_dev", ctypes.c_void_p),
                ("pair_axis_dev", ctypes.c_void_p), ("axes", ctypes.c_int),
                ("pairs", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("factor", ctypes.c_float)]


class Norm(ctypes.Structure):
    _fields_ = [("x_dev", ctypes.c_void_p), ("x_dtype", ctypes.c_int), ("x_ld", ctypes.c_int64),
                ("residual_dev", ctypes.c_void_p), ("residual_out_dev", ctypes.c_void_p),
                ("residual_dtype", ctypes.c_int), ("residual_ld", ctypes.c_int64),
                ("weight_dev", ctypes.c_void_p), ("weight_dtype", ctypes.c_int),
                ("weight_offset", ctypes.c_float), ("eps", ctypes.c_float),
                ("out_dev", ctypes.c_void_p), ("out_dtype", ctypes.c_int),
                ("out_ld", ctypes.c_int64), ("scale_dev", ctypes.c_void_p)]


_lib = None


def lib():
    """The loaded shared library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libnvfp4.so is not built (run __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        c = ctypes
        vp, sz, i = c.c_void_p, c.c_size_t, c.c_int
        L.nvfp4_status_string.argtypes = [i]
        L.nvfp4_status_string.restype = c.c_char_p
        L.nvfp4_last_error.argtypes = []
        L.nvfp4_last_error.restype = c.c_char_p
        L.nvfp4_version.restype = i
        L.nvfp4_packed_code_bytes.argtypes = [i, i]
        L.nvfp4_packed_code_bytes.restype = sz
        L.nvfp4_packed_scale_bytes.argtypes = [i, i]
        L.nvfp4_packed_scale_bytes.restype = sz
        L.nvfp4_pack.argtypes = [vp, vp, i, i, vp, vp, vp]
        L.nvfp4_unpack.argtypes = [vp, vp, i, i, vp, vp, vp]
        L.nvfp4_quantize_workspace_bytes.restype = sz
        L.nvfp4_quantize.argtypes = [vp, i, i, vp, vp, vp, vp, vp]
        L.nvfp4_gemm_create.argtypes = [c.POINTER(vp), i, i, i, i, c.POINTER(sz)]
        L.nvfp4_gemm_create_ex.argtypes = [c.POINTER(vp), i, i, i, i, c.POINTER(GemmConfig),
                                           c.POINTER(sz)]
        L.nvfp4_gemm_destroy.argtypes = [vp]
        L.nvfp4_gemm_destroy.restype = None
        L.nvfp4_gemm_run.argtypes = [vp, i, i, i, vp, vp, c.c_float, vp, vp, vp, vp]
        L.nvfp4_gemm_run_noalloc.argtypes = [vp, i, i, i, vp, vp, c.c_float, vp, vp, vp]
        L.nvfp4_gemm_run_argmax.argtypes = [vp, i, i, i, vp, vp, c.c_float, vp, vp, vp, vp, vp,
                                            sz, vp]
        L.nvfp4_gemm_argmax_area_bytes.argtypes = [vp]
        L.nvfp4_gemm_argmax_area_bytes.restype = sz
        L.nvfp4_workspace_clear.argtypes = [vp, sz, vp]
        L.nvfp4_round_workspace_bytes.argtypes = [c.POINTER(Layer), i, i, c.POINTER(sz)]
        L.nvfp4_round_create.argtypes = [c.POINTER(vp), c.POINTER(Layer), i, i, vp, sz, vp]
        L.nvfp4_round_run.argtypes = [vp, i, vp]
        L.nvfp4_round_graph_nodes.argtypes = [vp, i]
        L.nvfp4_round_destroy.argtypes = [vp]
        L.nvfp4_round_destroy.restype = None
        L.nvfp4_topk_workspace_bytes.argtypes = [i, i, i]
        L.nvfp4_topk_workspace_bytes.restype = sz
        L.nvfp4_topk.argtypes = [vp, i, i, i, i, vp, vp, vp, sz, vp]
        L.nvfp4_swiglu.argtypes = [vp, i, i, vp, vp]
        L.nvfp4_stream_read.argtypes = [vp, sz, vp, vp]
        i64, f = c.c_int64, c.c_float
        L.nvfp4_cache_append.argtypes = [c.POINTER(Cache), i, vp, i64, i, i, i, vp, vp, vp, i,
                                         c.POINTER(Rotary), vp, i64, vp]
        L.nvfp4_cache_compact.argtypes = [c.POINTER(Cache), i, vp, vp, i, vp, i, vp, vp]
        L.nvfp4_cache_update_workspace_bytes.argtypes = [i, i, i]
        L.nvfp4_cache_update_workspace_bytes.restype = sz
        L.nvfp4_cache_update.argtypes = [c.POINTER(Cache), i, vp, vp, vp, i, i, vp, vp, vp, vp,
                                         vp, vp, vp, vp, sz, vp]
        L.nvfp4_tree_mask.argtypes = [c.POINTER(i), i, c.POINTER(c.c_uint64), c.POINTER(i)]
        L.nvfp4_tree_attention_workspace_bytes.argtypes = [i, i, i, i]
        L.nvfp4_tree_attention_workspace_bytes.restype = sz
        L.nvfp4_tree_attention.argtypes = [c.POINTER(Cache), i, vp, i64, i, i, i, i, vp, vp, vp, i,
                                           vp, f, vp, i64, vp, vp, sz, vp]
        L.nvfp4_beam_workspace_bytes.argtypes = [i, i, i]
        L.nvfp4_beam_workspace_bytes.restype = sz
        L.nvfp4_beam_select.argtypes = [vp, i, i64, i, i, i, vp, vp, i, i, vp, vp, vp, vp, vp, sz,
                                        vp]
        L.nvfp4_rms_norm.argtypes = [vp, i, i, vp]  # an nvfp4_norm
        L.nvfp4_int8_quantize.argtypes = [vp, i, i64, i, i, i, vp, i64, vp, vp]
        L.nvfp4_int8_packed_bytes.argtypes = [i, i]
        L.nvfp4_int8_packed_bytes.restype = sz
        L.nvfp4_int8_pack.argtypes = [vp, i, i, vp, vp]
        L.nvfp4_int8_unpack.argtypes = [vp, i, i, vp, vp]
        L.nvfp4_int8_gemm_workspace_bytes.argtypes = [i, i, i]
        L.nvfp4_int8_gemm_workspace_bytes.restype = sz
        L.nvfp4_int8_gemm.argtypes = [vp, i64, vp, vp, vp, vp, i, i, i, vp, i, i64, vp, sz, vp]
        L.nvfp4_logprobs_workspace_bytes.argtypes = [i, i, i]
        L.nvfp4_logprobs_workspace_bytes.restype = sz
        L.nvfp4_logprobs.argtypes = [vp, i, i64, i, i, f, vp, i, i, vp, vp, vp, vp, vp, sz, vp]
        for name in EXPORTS:
            getattr(L, name)
        _lib = L
    return _lib


def _check(status):
    if status != OK:
        raise Nvfp4Error(status, lib().nvfp4_last_error().decode(errors="replace"))


def _ptr(x):
    """Device pointer of a tensor, or an int / None passed through."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def last_error() -> str:
    return lib().nvfp4_last_error().decode(errors="replace")


def status_string(status: int) -> str:
    return lib().nvfp4_status_string(status).decode()


def nvfp4_packed_code_bytes(K: int, N: int) -> int:
    return lib().nvfp4_packed_code_bytes(K, N)


def nvfp4_packed_scale_bytes(K: int, N: int) -> int:
    return lib().nvfp4_packed_scale_bytes(K, N)


def nvfp4_pack(codes, scales, K, N, codes_packed, scales_packed, stream=None):
    _check(lib().nvfp4_pack(_ptr(codes), _ptr(scales), K, N, _ptr(codes_packed),
                            _ptr(scales_packed), _stream(stream)))


def nvfp4_unpack(codes_packed, scales_packed, K, N, codes, scales, stream=None):
    _check(lib().nvfp4_unpack(_ptr(codes_packed), _ptr(scales_packed), K, N, _ptr(codes),
                              _ptr(scales), _stream(stream)))


def nvfp4_quantize_workspace_bytes() -> int:
    return lib().nvfp4_quantize_workspace_bytes()


def nvfp4_quantize(w, K, N, codes, scales, tensor_scale, workspace, stream=None):
    _check(lib().nvfp4_quantize(_ptr(w), K, N, _ptr(codes), _ptr(scales), _ptr(tensor_scale),
                                _ptr(workspace), _stream(stream)))


def nvfp4_swiglu(gate_up, M, F, out, stream=None):
    _check(lib().nvfp4_swiglu(_ptr(gate_up), M, F, _ptr(out), _stream(stream)))


def nvfp4_stream_read(buf, nbytes, sink, stream=None):
    _check(lib().nvfp4_stream_read(_ptr(buf), nbytes, _ptr(sink), _stream(stream)))


def nvfp4_gemm_argmax_area_bytes(plan) -> int:
    return lib().nvfp4_gemm_argmax_area_bytes(plan)


def nvfp4_gemm_run_argmax(plan, M, K, N, codes, scales, tensor_scale, act, logits, argmax,
                          workspace, area, area_bytes, stream=None):
    _check(lib().nvfp4_gemm_run_argmax(plan, M, K, N, _ptr(codes), _ptr(scales),
                                       tensor_scale, _ptr(act), _ptr(logits),
                                       _ptr(argmax), _ptr(workspace), _ptr(area), area_bytes,
                                       _stream(stream)))


def nvfp4_topk_workspace_bytes(M, V, k) -> int:
    return lib().nvfp4_topk_workspace_bytes(M, V, k)


def nvfp4_topk(logits, M, V, ld, k, idx, val, workspace=None, workspace_bytes=0, stream=None):
    _check(lib().nvfp4_topk(_ptr(logits), M, V, ld, k, _ptr(idx), _ptr(val), _ptr(workspace),
                            workspace_bytes, _stream(stream)))


def topk(logits, k, stream=None):
    """(indices int32 [M][k], values [M][k]) of a device fp32 [M][V] tensor.  A stream that is given is
    torch's current one during the call, so outputs belong to it."""
    import torch
    if stream is not None and logits.is_cuda:
        with _on(stream, logits.device):
            return topk(logits, k)
    M, V = logits.shape
    idx = torch.empty((M, k), dtype=torch.int32, device=logits.device)
    val = torch.empty((M, k), dtype=torch.float32, device=logits.device)
    wsb = nvfp4_topk_workspace_bytes(M, V, k)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=logits.device) if wsb else None
    nvfp4_topk(logits, M, V, logits.stride(0), k, idx, val, ws, wsb, stream)
    return idx, val


def nvfp4_cache_append(cache, layer, qkv, qkv_ld, rows, q_heads, lanes, row_start, ctx_len,
                       page_table, table_ld, rotary, q_out, q_ld, stream=None):
    _check(lib().nvfp4_cache_append(ctypes.byref(cache), layer, _ptr(qkv), qkv_ld, rows, q_heads,
                                    lanes, _ptr(row_start), _ptr(ctx_len), _ptr(page_table),
                                    table_ld, ctypes.byref(rotary), _ptr(q_out), q_ld,
                                    _stream(stream)))


def nvfp4_cache_compact(cache, lanes, ctx_len, page_table, table_ld, path, path_ld, accepted,
                        stream=None):
    _check(lib().nvfp4_cache_compact(ctypes.byref(cache), lanes, _ptr(ctx_len), _ptr(page_table),
                                     table_ld, _ptr(path), path_ld, _ptr(accepted),
                                     _stream(stream)))


def nvfp4_cache_update_workspace_bytes(pages, lanes_out, table_ld) -> int:
    return lib().nvfp4_cache_update_workspace_bytes(pages, lanes_out, table_ld)


def nvfp4_cache_update(cache, lanes_in, table_in, len_in, refs_in, table_ld, lanes_out, parent,
                       keep, reserve, table_out, len_out, refs_out, short, workspace,
                       workspace_bytes, stream=None):
    _check(lib().nvfp4_cache_update(ctypes.byref(cache), lanes_in, _ptr(table_in), _ptr(len_in),
                                    _ptr(refs_in), table_ld, lanes_out, _ptr(parent), _ptr(keep),
                                    _ptr(reserve), _ptr(table_out), _ptr(len_out),
                                    _ptr(refs_out), _ptr(short), _ptr(workspace),
                                    workspace_bytes, _stream(stream)))


def nvfp4_tree_mask(parent):
    """(mask words, depths) of a tree given by each drafted token's parent (-1: the context);
    mask words as signed 64-bit integers, the type a mask tensor has."""
    n = len(parent)
    p = (ctypes.c_int * max(n, 1))(*parent)
    mask, depth = (ctypes.c_uint64 * max(n, 1))(), (ctypes.c_int * max(n, 1))()
    _check(lib().nvfp4_tree_mask(p, n, mask, depth))
    return [m - (1 << 64) if m >> 63 else m for m in mask], list(depth)


def nvfp4_tree_attention_workspace_bytes(q_heads, kv_heads, head_dim, max_rows) -> int:
    return lib().nvfp4_tree_attention_workspace_bytes(q_heads, kv_heads, head_dim, max_rows)


def nvfp4_tree_attention(cache, layer, q, q_ld, q_heads, rows, lanes, max_rows, row_start, ctx_len,
                         page_table, table_ld, mask, scale, out, out_ld, lse, workspace,
                         workspace_bytes, stream=None):
    _check(lib().nvfp4_tree_attention(ctypes.byref(cache), layer, _ptr(q), q_ld, q_heads, rows,
                                      lanes, max_rows, _ptr(row_start), _ptr(ctx_len),
                                      _ptr(page_table), table_ld, _ptr(mask), scale, _ptr(out),
                                      out_ld, _ptr(lse), _ptr(workspace), workspace_bytes,
                                      _stream(stream)))


def nvfp4_beam_workspace_bytes(batch, beams, V) -> int:
    return lib().nvfp4_beam_workspace_bytes(batch, beams, V)


def nvfp4_beam_select(logits, logits_dtype, ld, batch, beams, V, score, done, eos, k, score_out,
                      parent, token, done_out, workspace, workspace_bytes, stream=None):
    _check(lib().nvfp4_beam_select(_ptr(logits), logits_dtype, ld, batch, beams, V, _ptr(score),
                                   _ptr(done), eos, k, _ptr(score_out), _ptr(parent),
                                   _ptr(token), _ptr(done_out), _ptr(workspace),
                                   workspace_bytes, _stream(stream)))


def beam_select(logits, beams, score, k, done=None, eos=-1, stream=None):
    """The k best continuations of each request: (score fp32, parent int32, token int32, done
    uint8), each [requests][k], of a device fp32 or bf16 logits tensor [requests * beams][V].  A
    stream that is given is torch's current one during the call, so outputs belong to it."""
    import torch
    if stream is not None and logits.is_cuda:
        with _on(stream, logits.device):
            return beam_select(logits, beams, score, k, done, eos)
    rows, V = logits.shape
    batch = rows // beams if beams > 0 else 0
    if rows != batch * beams:
        _refuse("logits: %d rows are not a multiple of %d beams" % (rows, beams))
    ld, inner = logits.stride()
    if inner != 1 and V > 1:
        _refuse("logits: rows are not contiguous")
    if logits.dtype is torch.float32:
        dtype = OUT_F32
    elif logits.dtype is torch.bfloat16:
        dtype = OUT_BF16
    else:
        _refuse("logits: not float32 or bfloat16")
    gpu = logits.get_device()
    if gpu < 0:
        _refuse("logits: not on a GPU")
    if not (score.dtype is torch.float32 and score.numel() == rows and score.is_contiguous()
            and score.get_device() == gpu):
        _refuse("score: not %d contiguous float32 values on the logits' GPU" % rows)
    if done is not None and not (done.dtype is torch.uint8 and done.numel() == rows and done.is_contiguous()
                                 and done.get_device() == gpu):
        _refuse("done: not %d contiguous uint8 values on the logits' GPU" % rows)
    L, dev = _lib or lib(), logits.device
    shape = (batch, k)
    out = score.new_empty(shape)
    parent = torch.empty(shape, dtype=torch.int32, device=dev)
    token = torch.empty_like(parent)
    ended = torch.empty(shape, dtype=torch.uint8, device=dev) if done is None else done.new_empty(shape)
    wsb = L.nvfp4_beam_workspace_bytes(batch, beams, V)
    ws = score.new_empty(wsb // 4 + 4)
    st = L.nvfp4_beam_select(logits.data_ptr(), dtype, ld if rows > 1 else max(ld, V), batch, beams, V,
                             score.data_ptr(), None if done is None else done.data_ptr(), eos, k,
                             out.data_ptr(), parent.data_ptr(), token.data_ptr(), ended.data_ptr(),
                             ws.data_ptr(), wsb, _current(dev))
    if st:
        _check(st)
    return out, parent, token, ended


def nvfp4_rms_norm(norm, rows, K, stream=None):
    _check(lib().nvfp4_rms_norm(ctypes.byref(norm), rows, K, _stream(stream)))


def nvfp4_int8_quantize(x, x_dtype, x_ld, rows, K, swiglu, codes, codes_ld, scale, stream=None):
    _check(lib().nvfp4_int8_quantize(_ptr(x), x_dtype, x_ld, rows, K, swiglu, _ptr(codes),
                                     codes_ld, _ptr(scale), _stream(stream)))


def nvfp4_int8_packed_bytes(K, N) -> int:
    return lib().nvfp4_int8_packed_bytes(K, N)


def nvfp4_int8_pack(codes, K, N, packed, stream=None):
    _check(lib().nvfp4_int8_pack(_ptr(codes), K, N, _ptr(packed), _stream(stream)))


def nvfp4_int8_unpack(packed, K, N, codes, stream=None):
    _check(lib().nvfp4_int8_unpack(_ptr(packed), K, N, _ptr(codes), _stream(stream)))


def nvfp4_int8_gemm_workspace_bytes(M, K, N) -> int:
    return lib().nvfp4_int8_gemm_workspace_bytes(M, K, N)


def nvfp4_int8_gemm(a, a_ld, a_scale, w_packed, w_scale, bias, M, K, N, out, out_dtype, out_ld,
                    workspace=None, workspace_bytes=0, stream=None):
    _check(lib().nvfp4_int8_gemm(_ptr(a), a_ld, _ptr(a_scale), _ptr(w_packed), _ptr(w_scale),
                                 _ptr(bias), M, K, N, _ptr(out), out_dtype, out_ld,
                                 _ptr(workspace), workspace_bytes, _stream(stream)))


def nvfp4_logprobs_workspace_bytes(rows, V, k) -> int:
    return lib().nvfp4_logprobs_workspace_bytes(rows, V, k)


def nvfp4_logprobs(logits, logits_dtype, ld, rows, V, scale, tokens, n_tokens, k, logprob, entropy,
                   top_token, top_logprob, workspace, workspace_bytes, stream=None):
    _check(lib().nvfp4_logprobs(_ptr(logits), logits_dtype, ld, rows, V, scale, _ptr(tokens),
                                n_tokens, k, _ptr(logprob), _ptr(entropy), _ptr(top_token),
                                _ptr(top_logprob), _ptr(workspace), workspace_bytes,
                                _stream(stream)))


_INT_MAX = 2 ** 31 - 1


class _Torch:
    """torch's types and calls that the functions below use, looked up once."""
    known = None

    def __init__(self):
        import struct

        import torch
        self.f32, self.bf16, self.i8, self.i32, self.u8 = (torch.float32, torch.bfloat16, torch.int8, torch.int32,
                                                           torch.uint8)
        self.floats = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16}
        self.outs = {None: OUT_BF16, **self.floats}
        self.normed = {**self.outs, torch.int8: OUT_INT8}
        self.empty, self.like = torch.empty, torch.empty_like
        here = torch.cuda.is_available()
        self.stream = torch._C._cuda_getCurrentRawStream if here else lambda gpu: 0
        self.device = torch._C._cuda_getDevice if here else lambda: 0
        self.on_device = torch.cuda.device
        self.norm = struct.Struct("PiqPPiqPiffPiqP").pack  # an nvfp4_norm


def _torch():
    if _Torch.known is None:
        _Torch.known = _Torch()
    return _Torch.known


def _bad_matrix(x, name, gpu, types):
    """Names what is wrong with a matrix."""
    if x.dim() != 2 or x.get_device() < 0 or x.get_device() != gpu:
        _refuse("%s: not a matrix on %s GPU" % (name, "a" if gpu < 0 else "the call's"))
    if x.dtype not in types:
        _refuse("%s: of type %s" % (name, x.dtype))
    if x.stride(1) != 1 and x.shape[1] > 1:
        _refuse("%s: rows are not contiguous" % name)


def _matrix(x, name, gpu, types):
    """(shape, row stride) of a matrix of contiguous rows on a GPU; the stride of a single row is never
    used, and is its columns."""
    if x.dim() != 2 or gpu < 0 or x.get_device() != gpu or x.dtype not in types or (x.stride(1) != 1 and x.shape[1] > 1):
        _bad_matrix(x, name, gpu, types)
    shape = x.shape
    if shape[0] > _INT_MAX or shape[1] > _INT_MAX:  # what a C int would cut off
        _refuse("%s: shape %s" % (name, tuple(shape)))
    return shape, x.stride(0) if shape[0] > 1 else shape[1]


def _vector(x, n, dtype, name, gpu):
    """Refuses anything but n contiguous values of a type on a GPU."""
    if not (x.dtype is dtype and x.numel() == n and x.is_contiguous() and x.get_device() == gpu):
        _refuse("%s: not %d contiguous %s values on the call's GPU" % (name, n, str(dtype).replace("torch.", "")))


def rms_norm(x, weight, eps, residual=None, dtype=None, weight_offset=0.0, out=None, residual_out=None,
             stream=None):
    """Root-mean-square norm of a device fp32 or bf16 matrix [rows][K], or of the residual stream it is
    added to, times ``weight + weight_offset`` ([K], fp32 or bf16).  ``dtype``: the output's, bfloat16 (as
    by default), float32, or int8 for codes with a scale each row.  Returns ``out``; ``(codes, scale)`` for
    int8; and the new residual stream as a last value if ``residual`` is given (``residual_out`` may be
    ``residual`` itself; by default it has the residual's stride, or, if that is more than 2 K, none between rows).  A stream that is given is torch's current one during the call, so outputs belong
    to it."""
    if stream is not None and x.is_cuda:
        with _on(stream, x.device):
            return rms_norm(x, weight, eps, residual, dtype, weight_offset, out, residual_out)
    T, L, gpu = _Torch.known or _torch(), _lib or lib(), x.get_device()
    if gpu != T.device() and gpu >= 0:  # launches go to the current device
        with T.on_device(gpu):
            return rms_norm(x, weight, eps, residual, dtype, weight_offset, out, residual_out)
    shape, x_ld = _matrix(x, "x", gpu, T.floats)
    rows, K = shape
    wanted = T.normed.get(dtype)
    if wanted is None:
        _refuse("dtype: %s" % dtype)
    w_type = T.floats.get(weight.dtype)
    if w_type is None:
        _refuse("weight: of type %s" % weight.dtype)
    _vector(weight, K, weight.dtype, "weight", gpu)
    if out is None:
        # (empty_like takes 0.9 us, new_empty 1.1, empty 1.5)
        dtype = dtype or T.bf16
        out = T.like(x) if x.dtype is dtype and x_ld == K else x.new_empty(shape, dtype=dtype)
        out_ld = K
    else:
        out_shape, out_ld = _matrix(out, "out", gpu, (dtype or T.bf16,))
        if out_shape != shape:
            _refuse("out: shape %s, not %s" % (tuple(out.shape), (rows, K)))
    scale = None
    if wanted == OUT_INT8:
        scale = T.empty(rows, dtype=T.f32, device=x.device)
    r = r_out = r_type = r_ld = 0
    if residual is not None:
        r_shape, r_ld = _matrix(residual, "residual", gpu, T.floats)
        if r_shape != shape:
            _refuse("residual: shape %s, not %s" % (tuple(residual.shape), (rows, K)))
        r_type = T.floats[residual.dtype]
        if residual_out is None:
            if r_ld > 2 * K:
                # (both streams have one stride: a few columns of a wide buffer would take as much memory as it has)
                residual, r_ld = residual.contiguous(), K
                residual_out = residual
            else:
                residual_out = T.like(residual) if r_ld == K else residual.new_empty((rows, r_ld))[:, :K]
        elif _matrix(residual_out, "residual_out", gpu, (residual.dtype,)) != (shape, r_ld):
            _refuse("residual_out: not of the residual's shape, type and stride")
        r, r_out = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        _refuse("residual_out: without a residual")
    st = L.nvfp4_rms_norm(T.norm(x.data_ptr(), T.floats[x.dtype], x_ld, r, r_out, r_type, r_ld, weight.data_ptr(), w_type,
                                 weight_offset, eps, out.data_ptr(), wanted, out_ld,
                                 0 if scale is None else scale.data_ptr()), rows, K, T.stream(gpu))
    if st:
        _check(st)
    if scale is None:
        return out if residual is None else (out, residual_out)
    return (out, scale) if residual is None else (out, scale, residual_out)


def int8_quantize(x, swiglu=False, codes=None, stream=None):
    """(codes int8 [rows][K], scale fp32 [rows]) of a device fp32 or bf16 matrix [rows][K], or, with
    ``swiglu``, of silu(gate) * up of one [rows][gate | up] of 2 K columns.  A stream that is given is
    torch's current one during the call, so outputs belong to it."""
    if stream is not None and x.is_cuda:
        with _on(stream, x.device):
            return int8_quantize(x, swiglu, codes)
    T, L, gpu = _Torch.known or _torch(), _lib or lib(), x.get_device()
    if gpu != T.device() and gpu >= 0:  # launches go to the current device
        with T.on_device(gpu):
            return int8_quantize(x, swiglu, codes)
    (rows, K), x_ld = _matrix(x, "x", gpu, T.floats)
    if swiglu:
        if K % 2:
            _refuse("x: %d columns are not two halves" % K)
        K //= 2
    if codes is None:
        codes, codes_ld = T.empty((rows, K), dtype=T.i8, device=x.device), K
    else:
        shape, codes_ld = _matrix(codes, "codes", gpu, (T.i8,))
        if shape != (rows, K):
            _refuse("codes: shape %s, not %s" % (tuple(shape), (rows, K)))
    scale = T.empty(rows, dtype=T.f32, device=x.device)
    st = L.nvfp4_int8_quantize(x.data_ptr(), T.floats[x.dtype], x_ld, rows, K, 1 if swiglu else 0, codes.data_ptr(),
                               codes_ld, scale.data_ptr(), T.stream(gpu))
    if st:
        _check(st)
    return codes, scale


class Int8Weight:
    """A K x N matrix of 8-bit integers with one scale for each output channel, packed on the GPU."""

    def __init__(self, packed, scale, K: int, N: int):
        T, size = _torch(), nvfp4_int8_packed_bytes(K, N)
        if not size:
            _refuse("K, N: %d x %d cannot be packed" % (K, N))
        if packed.dtype is not T.i8 or packed.numel() < size or not packed.is_contiguous():
            _refuse("packed: not %d contiguous int8 values, or more" % size)
        if scale.dtype is not T.f32 or scale.numel() != N or not scale.is_contiguous():
            _refuse("scale: not %d contiguous float32 values" % N)
        self.packed, self.scale, self.K, self.N = packed, scale, K, N

    @classmethod
    def from_canonical(cls, codes, scale, stream=None):
        """Pack a device int8 matrix [N][K] with its channels' fp32 scales [N].  Both are copied: the weight does not
        change with the tensors that it was made of."""
        if stream is not None and codes.is_cuda:
            with _on(stream, codes.device):
                return cls.from_canonical(codes, scale)
        T, gpu = _torch(), codes.get_device()
        if gpu != T.device() and gpu >= 0:
            with T.on_device(gpu):
                return cls.from_canonical(codes, scale)
        (N, K), ld = _matrix(codes, "codes", gpu, (T.i8,))
        if ld != K:
            _refuse("codes: rows are not next to each other")
        _vector(scale, N, T.f32, "scale", gpu)
        packed = T.empty(nvfp4_int8_packed_bytes(K, N), dtype=T.i8, device=codes.device)
        st = lib().nvfp4_int8_pack(codes.data_ptr(), K, N, packed.data_ptr(), T.stream(gpu))
        if st:
            _check(st)
        return cls(packed, scale.clone(), K, N)

    @classmethod
    def quantize(cls, w, stream=None):
        """Quantise a device fp32 or bf16 matrix [N][K] and pack it."""
        if stream is not None and w.is_cuda:
            with _on(stream, w.device):
                return cls.quantize(w)
        return cls.from_canonical(*int8_quantize(w))


def int8_gemm(codes, scale, weight, dtype=None, bias=None, out=None, stream=None):
    """[M][N] product, bfloat16 (as by default) or float32, of a device int8 matrix [M][K] with its rows'
    fp32 scales [M] and an ``Int8Weight``, plus ``bias`` (fp32 [N]).  A stream that is given is torch's
    current one during the call, so outputs belong to it."""
    if stream is not None and codes.is_cuda:
        with _on(stream, codes.device):
            return int8_gemm(codes, scale, weight, dtype, bias, out)
    T, L, gpu, K, N = _Torch.known or _torch(), _lib or lib(), codes.get_device(), weight.K, weight.N
    if gpu != T.device() and gpu >= 0:  # launches go to the current device
        with T.on_device(gpu):
            return int8_gemm(codes, scale, weight, dtype, bias, out)
    (M, cols), ld = _matrix(codes, "codes", gpu, (T.i8,))
    if cols != K:
        _refuse("codes: %d columns, not the weight's K = %d" % (cols, K))
    _vector(scale, M, T.f32, "scale", gpu)
    if weight.packed.get_device() != gpu or weight.scale.get_device() != gpu:
        _refuse("weight: not on the call's GPU")
    if bias is not None:
        _vector(bias, N, T.f32, "bias", gpu)
    wanted = T.outs.get(dtype)
    if wanted is None:
        _refuse("dtype: %s" % dtype)
    if out is None:
        out, out_ld = T.empty((M, N), dtype=dtype or T.bf16, device=codes.device), N
    else:
        shape, out_ld = _matrix(out, "out", gpu, (dtype or T.bf16,))
        if shape != (M, N):
            _refuse("out: shape %s, not %s" % (tuple(shape), (M, N)))
    wsb = L.nvfp4_int8_gemm_workspace_bytes(M, K, N)
    ws = T.empty(wsb, dtype=T.u8, device=codes.device) if wsb else None
    st = L.nvfp4_int8_gemm(codes.data_ptr(), ld, scale.data_ptr(), weight.packed.data_ptr(), weight.scale.data_ptr(),
                           None if bias is None else bias.data_ptr(), M, K, N, out.data_ptr(), wanted, out_ld,
                           None if ws is None else ws.data_ptr(), wsb, T.stream(gpu))
    if st:
        _check(st)
    return out


def logprobs(logits, tokens, k=0, scale=1.0, stream=None):
    """(logprob fp32 of the tokens' shape, entropy fp32 [rows], top_token int32 [rows][k], top_logprob fp32
    [rows][k]; the last two None for k = 0) of a device fp32 or bf16 logits matrix [rows][V], times
    ``scale`` (an inverse temperature), and int32 ``tokens`` [rows] or [rows][n].  A stream that is given is
    torch's current one during the call, so outputs belong to it."""
    if stream is not None and logits.is_cuda:
        with _on(stream, logits.device):
            return logprobs(logits, tokens, k, scale)
    T, L, gpu, dev = _Torch.known or _torch(), _lib or lib(), logits.get_device(), logits.device
    if gpu != T.device() and gpu >= 0:  # launches go to the current device
        with T.on_device(gpu):
            return logprobs(logits, tokens, k, scale)
    (rows, V), ld = _matrix(logits, "logits", gpu, T.floats)
    asked = tokens.shape
    if len(asked) not in (1, 2) or asked[0] != rows:
        _refuse("tokens: shape %s does not go with %d rows" % (tuple(asked), rows))
    n = asked[1] if len(asked) == 2 else 1
    if n > 1024:
        _refuse("tokens: %d of a row, more than 1024" % n)
    if k > V:
        _refuse("k: %d > V = %d" % (k, V))
    _vector(tokens, rows * n, T.i32, "tokens", gpu)
    logprob = T.empty(asked, dtype=T.f32, device=dev)
    entropy = logprob.new_empty(rows)
    top_token = top = None
    if k > 0:
        top_token, top = tokens.new_empty((rows, k)), logprob.new_empty((rows, k))
    wsb = L.nvfp4_logprobs_workspace_bytes(rows, V, k)
    ws = logprob.new_empty(wsb // 4)
    st = L.nvfp4_logprobs(logits.data_ptr(), T.floats[logits.dtype], ld, rows, V, scale, tokens.data_ptr(), n, k,
                          logprob.data_ptr(), entropy.data_ptr(), None if top is None else top_token.data_ptr(),
                          None if top is None else top.data_ptr(), ws.data_ptr(), wsb, T.stream(gpu))
    if st:
        _check(st)
    return logprob, entropy, top_token, top


def nvfp4_gemm_create(max_M, K, N, out_dtype, split_k=0, waves=0, chunks=0, windows=0,
                      verify_waves=0, verify_windows=0, tile_max_m=0, tile_superblocks=0,
                      verify_ranges=0, prefill_schedule=0):
    """Returns (plan handle, workspace bytes)."""
    h = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    if (split_k or waves or chunks or windows or verify_waves or verify_windows or tile_max_m
            or tile_superblocks or verify_ranges or prefill_schedule):
        cfg = GemmConfig(split_k, waves, chunks, windows, verify_waves, verify_windows,
                         tile_max_m, tile_superblocks, verify_ranges, prefill_schedule)
        _check(lib().nvfp4_gemm_create_ex(ctypes.byref(h), max_M, K, N, out_dtype,
                                          ctypes.byref(cfg), ctypes.byref(ws)))
    else:
        _check(lib().nvfp4_gemm_create(ctypes.byref(h), max_M, K, N, out_dtype,
                                       ctypes.byref(ws)))
    return h.value, ws.value


def nvfp4_gemm_destroy(plan):
    lib().nvfp4_gemm_destroy(plan)


def nvfp4_gemm_run(plan, M, K, N, codes, scales, tensor_scale, act, out, workspace=None,
                   stream=None):
    _check(lib().nvfp4_gemm_run(plan, M, K, N, _ptr(codes), _ptr(scales),
                                ctypes.c_float(tensor_scale), _ptr(act), _ptr(out),
                                _ptr(workspace), _stream(stream)))


def nvfp4_gemm_run_noalloc(plan, M, K, N, codes, scales, tensor_scale, act, out, stream=None):
    _check(lib().nvfp4_gemm_run_noalloc(plan, M, K, N, _ptr(codes), _ptr(scales),
                                        ctypes.c_float(tensor_scale), _ptr(act), _ptr(out),
                                        _stream(stream)))


def nvfp4_workspace_clear(workspace, nbytes, stream=None):
    _check(lib().nvfp4_workspace_clear(_ptr(workspace), nbytes, _stream(stream)))


def _layers(layers):
    arr = (Layer * len(layers))()
    for i, l in enumerate(layers):
        arr[i] = Layer(l["K"], l["N"], _ptr(l["codes"]), _ptr(l["scales"]),
                       float(l["tensor_scale"]), _ptr(l["act"]), _ptr(l["out"]),
                       int(l.get("out_dtype", OUT_BF16)), int(l.get("act_op", ACT_INPUT)))
    return arr


def nvfp4_round_workspace_bytes(layers, max_M) -> int:
    ws = ctypes.c_size_t()
    _check(lib().nvfp4_round_workspace_bytes(_layers(layers), len(layers), max_M,
                                             ctypes.byref(ws)))
    return ws.value


def nvfp4_round_create(layers, max_M, workspace, workspace_bytes, stream=None):
    h = ctypes.c_void_p()
    _check(lib().nvfp4_round_create(ctypes.byref(h), _layers(layers), len(layers), max_M,
                                    _ptr(workspace), workspace_bytes, _stream(stream)))
    return h.value


def nvfp4_round_run(plan, M, stream=None):
    _check(lib().nvfp4_round_run(plan, M, _stream(stream)))


def nvfp4_round_graph_nodes(plan, M) -> int:
    return lib().nvfp4_round_graph_nodes(plan, M)


def nvfp4_round_destroy(plan):
    lib().nvfp4_round_destroy(plan)


# ---- convenience layer (still only marshalling) -----------------------------

class PackedWeight:
    """A K x N NVFP4 matrix in the packed layout on the GPU."""

    def __init__(self, codes_packed, scales_packed, tensor_scale: float, K: int, N: int):
        self.codes = codes_packed
        self.scales = scales_packed
        self.tensor_scale = float(tensor_scale)
        self.K = K
        self.N = N

    @staticmethod
    def alloc(K, N, device="cuda"):
        import torch
        c = torch.empty(nvfp4_packed_code_bytes(K, N), dtype=torch.uint8, device=device)
        s = torch.empty(nvfp4_packed_scale_bytes(K, N), dtype=torch.uint8, device=device)
        return c, s

    @classmethod
    def from_canonical(cls, codes, scales, tensor_scale, K, N, stream=None):
        """Pack canonical planes (device tensors [N][K/2], [N][K/16])."""
        if stream is not None and codes.is_cuda:
            with _on(stream, codes.device):
                return cls.from_canonical(codes, scales, tensor_scale, K, N)
        c, s = cls.alloc(K, N, codes.device)
        nvfp4_pack(codes, scales, K, N, c, s, stream)
        return cls(c, s, tensor_scale, K, N)

    @classmethod
    def quantize(cls, w, stream=None, keep_canonical=False):
        """Quantise a device fp32 [N][K] tensor and pack it.  Reads the tensor
        scale back to the host (one synchronisation)."""
        import torch
        if stream is not None and w.is_cuda:
            with _on(stream, w.device):
                return cls.quantize(w, None, keep_canonical)
        N, K = w.shape
        dev = w.device
        codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((N, K // 16), dtype=torch.uint8, device=dev)
        ts = torch.empty(1, dtype=torch.float32, device=dev)
        ws = torch.empty(nvfp4_quantize_workspace_bytes(), dtype=torch.uint8, device=dev)
        nvfp4_quantize(w, K, N, codes, scales, ts, ws, stream)
        pw = cls.from_canonical(codes, scales, 0.0, K, N, stream)
        pw.tensor_scale = float(ts.item())
        if keep_canonical:
            pw.canonical = (codes, scales)
        return pw


def _refuse(message):
    raise Nvfp4Error(EINVAL, message)


def _current(device):
    """torch's current stream on a device, as a handle."""
    import torch
    if device.type != "cuda":
        return 0
    return torch._C._cuda_getCurrentRawStream(device.index)


def _on(stream, device):
    """Context in which a stream (torch's, or a handle of `device`) is torch's current one: what a call
    allocates is then taken from that stream's memory, and reused by it alone."""
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    if stream.device != device:
        _refuse("stream: on %s, not %s" % (stream.device, device))
    return torch.cuda.stream(stream)


class PagedCache:
    """A paged key/value cache over the caller's tensors and the operators on it.

    ``k``: [layers][pages][kv_heads][page_tokens][head_dim]; ``v``: [layers][pages][kv_heads]
    [page_tokens / 16][head_dim][16]; bfloat16, or float8_e4m3fn standing for ``scale`` times its
    value.  A page is contiguous; layers and pages may have other strides (equal ones for k and v).

    ``row_start`` (int32 [lanes + 1]), ``ctx_len`` (int32 [lanes]) and ``page_table`` (int32
    [lanes][pages of a lane], contiguous) and a call's other tensors are on k's and v's GPU, and are
    refused elsewhere; include/nvfp4.h has the rules of
    each call.  A call runs on torch's current stream, or makes the one that it is given current:
    outputs and workspaces come from that stream's memory, call by call, and tensors of other streams
    need what torch asks for there (a wait before, ``record_stream`` before they are dropped).
    (The checks are written out in each method: they run once per layer and round.)
    """

    def __init__(self, k, v, k_scale=1.0, v_scale=1.0):
        import torch
        if k.dim() != 5 or v.dim() != 6:
            _refuse("k, v: not 5 and 6 dimensions")
        layers, pages, heads, tokens, dim = k.shape
        if tuple(v.shape) != (layers, pages, heads, tokens // 16, dim, 16):
            _refuse("v: shape %s does not go with k's %s" % (tuple(v.shape), tuple(k.shape)))
        if k.device != v.device:
            _refuse("v: not on k's device")
        if k.dtype != v.dtype or k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            _refuse("k, v: not both bfloat16 or float8_e4m3fn")
        for x, want, name in ((k, (tokens * dim, dim, 1), "k"),
                              (v, (tokens * dim, 16 * dim, 16, 1), "v")):
            if any(n != 1 and a != b for n, a, b in zip(x.shape[2:], x.stride()[2:], want)):
                _refuse("%s: a page is not contiguous" % name)
            if any(n > 1 and s == 0 for n, s in zip(x.shape[:2], x.stride()[:2])):
                _refuse("%s: layers or pages share memory" % name)
        es = k.element_size()
        strides = [[0 if n == 1 else s * es for n, s in zip(x.shape[:2], x.stride()[:2])]
                   for x in (k, v)]
        if strides[0] != strides[1]:
            _refuse("k, v: layers or pages have different strides")
        self.k, self.v = k, v
        self.layers, self.pages, self.kv_heads, self.page_tokens, self.head_dim = k.shape
        self.device = k.device
        self._gpu = k.get_device()  # -1: none, and every call is refused
        self.desc = Cache(k.data_ptr(), v.data_ptr(), layers, pages, heads, tokens, dim,
                          CACHE_BF16 if es == 2 else CACHE_E4M3, float(k_scale), float(v_scale),
                          strides[0][1], strides[0][0])
        self._ref = ctypes.byref(self.desc)
        self._attend_ws = {}  # workspace bytes by (q heads, rows)
        self._update_ws = {}  # by lanes and table width

    def _bad_lanes(self, row_start, ctx_len, page_table, lanes, length="ctx_len"):
        """Names what is wrong with a call's lanes."""
        import torch
        if self._gpu < 0:
            _refuse("cache: not on a GPU")
        for x, n, name in ((row_start, lanes + 1, "row_start"), (ctx_len, lanes, length)):
            if x is not None and not (x.dtype is torch.int32 and x.numel() == n and x.is_contiguous()
                                      and x.get_device() == self._gpu):
                _refuse("%s: not %d contiguous int32 values on the cache's GPU" % (name, n))
        _refuse("page_table: not a contiguous int32 matrix of %d rows on the cache's GPU" % lanes)

    def append(self, layer, qkv, q_heads, row_start, ctx_len, page_table, positions, inv_freq,
               pair_axis=None, interleaved=False, factor=1.0, out=None, stream=None):
        """Rotates q and k of a qkv product's rows, stores k and v, returns q [rows][q_heads * dim]."""
        import torch
        if stream is not None and self._gpu >= 0:
            with _on(stream, self.device):
                return self.append(layer, qkv, q_heads, row_start, ctx_len, page_table, positions, inv_freq,
                                   pair_axis, interleaved, factor, out)
        i32, bf16 = torch.int32, torch.bfloat16
        lanes, dim, L, dev, gpu = ctx_len.numel(), self.head_dim, _lib or lib(), self.device, self._gpu
        if not (ctx_len.dtype is i32 and ctx_len.is_contiguous() and row_start.dtype is i32
                and row_start.is_contiguous() and row_start.numel() == lanes + 1
                and page_table.dtype is i32 and page_table.is_contiguous()
                and page_table.dim() == 2 and page_table.shape[0] == lanes
                and gpu >= 0 and ctx_len.get_device() == gpu and row_start.get_device() == gpu
                and page_table.get_device() == gpu):
            self._bad_lanes(row_start, ctx_len, page_table, lanes)
        width = q_heads * dim
        if qkv.dtype is not bf16 or qkv.dim() != 2 or qkv.get_device() != gpu:
            _refuse("qkv: not a bfloat16 matrix on the cache's GPU")
        rows, cols = qkv.shape
        ld, inner = qkv.stride()
        taken = width + 2 * self.kv_heads * dim
        if cols < taken or inner != 1:
            _refuse("qkv: rows are not %d contiguous values" % taken)
        pairs, axes = inv_freq.numel(), positions.shape[1] if positions.dim() == 2 else 1
        if not (inv_freq.dtype is torch.float32 and inv_freq.is_contiguous() and inv_freq.get_device() == gpu):
            _refuse("inv_freq: not contiguous float32 values on the cache's GPU")
        if not (positions.dtype is i32 and positions.is_contiguous() and positions.numel() == rows * axes
                and positions.get_device() == gpu):
            _refuse("positions: not %d contiguous int32 values on the cache's GPU" % (rows * axes))
        if pair_axis is not None and not (pair_axis.dtype is torch.uint8 and pair_axis.is_contiguous()
                                          and pair_axis.numel() == pairs and pair_axis.get_device() == gpu):
            _refuse("pair_axis: not %d contiguous uint8 values on the cache's GPU" % pairs)
        if out is None:
            out, q_ld = qkv.new_empty((rows, width)), width
        else:
            q_ld = self._out_ld(out, rows, width)
        rot = Rotary(positions.data_ptr(), inv_freq.data_ptr(),
                     None if pair_axis is None else pair_axis.data_ptr(), axes, pairs, interleaved, factor)
        st = L.nvfp4_cache_append(self._ref, layer, qkv.data_ptr(), ld if rows > 1 else taken, rows,
                                  q_heads, lanes, row_start.data_ptr(), ctx_len.data_ptr(),
                                  page_table.data_ptr(), page_table.shape[1], ctypes.byref(rot), out.data_ptr(),
                                  q_ld, _current(dev))
        if st:
            _check(st)
        return out

    def _out_ld(self, out, rows, width):
        """Leading dimension of a caller's output of at least `rows` rows."""
        import torch
        if out.dtype is not torch.bfloat16 or out.dim() != 2 or out.shape[0] < rows or out.get_device() != self._gpu:
            _refuse("out: not a bfloat16 matrix of %d rows on the cache's GPU" % rows)
        if out.shape[1] < width or out.stride(1) != 1:
            _refuse("out: rows are not %d contiguous values" % width)
        return out.stride(0) if rows > 1 else width

    def attend(self, layer, q, row_start, ctx_len, page_table, mask, max_rows, scale, out=None,
               with_lse=False, stream=None):
        """Attention of each lane's drafted rows q [rows][q_heads * dim] over its context and the
        drafts its mask words (int64 [rows]) name; max_rows: at least any lane's rows.  Returns
        out, or (out, lse fp32 [rows][q_heads])."""
        import torch
        if stream is not None and self._gpu >= 0:
            with _on(stream, self.device):
                return self.attend(layer, q, row_start, ctx_len, page_table, mask, max_rows, scale, out, with_lse)
        i32, bf16 = torch.int32, torch.bfloat16
        lanes, dim, L, dev, gpu = ctx_len.numel(), self.head_dim, _lib or lib(), self.device, self._gpu
        if not (ctx_len.dtype is i32 and ctx_len.is_contiguous() and row_start.dtype is i32
                and row_start.is_contiguous() and row_start.numel() == lanes + 1
                and page_table.dtype is i32 and page_table.is_contiguous()
                and page_table.dim() == 2 and page_table.shape[0] == lanes
                and gpu >= 0 and ctx_len.get_device() == gpu and row_start.get_device() == gpu
                and page_table.get_device() == gpu):
            self._bad_lanes(row_start, ctx_len, page_table, lanes)
        if q.dtype is not bf16 or q.dim() != 2 or q.get_device() != gpu:
            _refuse("q: not a bfloat16 matrix on the cache's GPU")
        rows, cols = q.shape
        ld, inner = q.stride()
        q_heads = cols // dim
        width = q_heads * dim
        if inner != 1:
            _refuse("q: rows are not contiguous")
        if not (mask.dtype is torch.int64 and mask.numel() == rows and mask.is_contiguous()
                and mask.get_device() == gpu):
            _refuse("mask: not %d contiguous int64 values on the cache's GPU" % rows)
        if out is None:
            out, out_ld = q.new_empty((rows, width)), width
        else:
            out_ld = self._out_ld(out, rows, width)
        lse = torch.empty((rows, q_heads), dtype=torch.float32, device=dev) if with_lse else None
        wsb = self._attend_ws.get((q_heads, max_rows))
        if wsb is None:
            wsb = L.nvfp4_tree_attention_workspace_bytes(q_heads, self.kv_heads, dim, max_rows)
            self._attend_ws[q_heads, max_rows] = wsb
        ws = q.new_empty(wsb // 2 + 8)
        st = L.nvfp4_tree_attention(self._ref, layer, q.data_ptr(), ld if rows > 1 else width, q_heads,
                                    rows, lanes, max_rows, row_start.data_ptr(), ctx_len.data_ptr(),
                                    page_table.data_ptr(), page_table.shape[1], mask.data_ptr(), scale,
                                    out.data_ptr(), out_ld, lse.data_ptr() if with_lse else None,
                                    ws.data_ptr(), wsb, _current(dev))
        if st:
            _check(st)
        return (out, lse) if with_lse else out

    def compact(self, ctx_len, page_table, path, accepted, stream=None):
        """Moves each lane's accepted drafts (path int32 [lanes][n], accepted int32 [lanes]) to the
        front of its drafted tokens, in every layer."""
        import torch
        i32, lanes, L, gpu = torch.int32, ctx_len.numel(), _lib or lib(), self._gpu
        if not (ctx_len.dtype is i32 and ctx_len.is_contiguous() and page_table.dtype is i32
                and page_table.is_contiguous() and page_table.dim() == 2 and page_table.shape[0] == lanes
                and gpu >= 0 and ctx_len.get_device() == gpu and page_table.get_device() == gpu):
            self._bad_lanes(None, ctx_len, page_table, lanes)
        if not (path.dtype is i32 and path.is_contiguous() and path.dim() == 2 and path.shape[0] == lanes
                and path.get_device() == gpu):
            _refuse("path: not a contiguous int32 matrix of %d rows on the cache's GPU" % lanes)
        if not (accepted.dtype is i32 and accepted.is_contiguous() and accepted.numel() == lanes
                and accepted.get_device() == gpu):
            _refuse("accepted: not %d contiguous int32 values on the cache's GPU" % lanes)
        st = L.nvfp4_cache_compact(self._ref, lanes, ctx_len.data_ptr(), page_table.data_ptr(),
                                   page_table.shape[1], path.data_ptr(), path.shape[1], accepted.data_ptr(),
                                   _current(self.device) if stream is None else _stream(stream))
        if st:
            _check(st)

    def update(self, page_table, length, refs, parent, keep=None, reserve=None, stream=None):
        """New tables from old ones (reorder, fork, truncate, free, make room): returns
        (page_table, length, refs, short), all int32; shared partly filled pages are copied."""
        import torch
        if stream is not None and self._gpu >= 0:
            with _on(stream, self.device):
                return self.update(page_table, length, refs, parent, keep, reserve)
        i32, lanes, L, dev, gpu = torch.int32, length.numel(), _lib or lib(), self.device, self._gpu
        if not (length.dtype is i32 and length.is_contiguous() and page_table.dtype is i32
                and page_table.is_contiguous() and page_table.dim() == 2 and page_table.shape[0] == lanes
                and gpu >= 0 and length.get_device() == gpu and page_table.get_device() == gpu):
            self._bad_lanes(None, length, page_table, lanes, "length")
        if not (refs.dtype is i32 and refs.is_contiguous() and refs.numel() == self.pages
                and refs.get_device() == gpu):
            _refuse("refs: not %d contiguous int32 values on the cache's GPU" % self.pages)
        n, width = parent.numel(), page_table.shape[1]
        for x, name in ((parent, "parent"), (keep, "keep"), (reserve, "reserve")):
            if x is not None and not (x.dtype is i32 and x.is_contiguous() and x.numel() == n
                                      and x.get_device() == gpu):
                _refuse("%s: not %d contiguous int32 values on the cache's GPU" % (name, n))
        table = page_table.new_empty((n, width))
        new_len = torch.empty_like(parent)
        new_refs = torch.empty_like(refs)
        short = refs.new_empty(1)
        wsb = self._update_ws.get((n, width))
        if wsb is None:
            wsb = L.nvfp4_cache_update_workspace_bytes(self.pages, n, width)
            self._update_ws[n, width] = wsb
        ws = refs.new_empty(wsb // 4 + 4)
        st = L.nvfp4_cache_update(self._ref, lanes, page_table.data_ptr(), length.data_ptr(), refs.data_ptr(),
                                  width, n, parent.data_ptr(), None if keep is None else keep.data_ptr(),
                                  None if reserve is None else reserve.data_ptr(), table.data_ptr(),
                                  new_len.data_ptr(), new_refs.data_ptr(), short.data_ptr(), ws.data_ptr(), wsb,
                                  _current(dev))
        if st:
            _check(st)
        return table, new_len, new_refs, short


class Gemm:
    """A plan plus its workspace: ``Gemm(max_M, K, N, out_dtype)(w, act, out)``."""

    def __init__(self, max_M, K, N, out_dtype=OUT_BF16, split_k=0, waves=0, chunks=0,
                 windows=0, device="cuda", verify_waves=0, verify_windows=0, tile_max_m=0,
                 tile_superblocks=0, verify_ranges=0, prefill_schedule=0):
        import torch
        self.plan, self.ws_bytes = nvfp4_gemm_create(max_M, K, N, out_dtype, split_k, waves,
                                                     chunks, windows, verify_waves,
                                                     verify_windows, tile_max_m,
                                                     tile_superblocks, verify_ranges,
                                                     prefill_schedule)
        self.K, self.N, self.max_M, self.out_dtype = K, N, max_M, out_dtype
        self.workspace = None
        if self.ws_bytes:
            self.workspace = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=device)

    def __call__(self, w: PackedWeight, act, out, M=None, stream=None):
        M = act.shape[0] if M is None else M
        nvfp4_gemm_run(self.plan, M, self.K, self.N, w.codes, w.scales, w.tensor_scale, act, out,
                       self.workspace, stream)
        return out

    def __del__(self):
        try:
            if self.plan:
                nvfp4_gemm_destroy(self.plan)
                self.plan = None
        except Exception:
            pass
