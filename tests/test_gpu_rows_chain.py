"""The norm, 8-bit rows and products and log probabilities together, as a decode step and a prefill chunk use
them: each step against the oracle of what the step before wrote; captured and replayed; on other streams."""
import numpy as np
import pytest

from oracle import rows as oracle
from tests.gpu_util import host, require_gpu

pytestmark = pytest.mark.gpu

K, F, V = 640, 1280, 5003


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


class Model:
    """One layer's MLP and the head, in 8 bits."""

    def __init__(self, nv, seed=0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        draw = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.nv = nv
        self.norm1, self.norm2 = (1 + 0.2 * draw(K)).to(torch.bfloat16), 0.1 * draw(K)
        self.gate_up, self.down, self.head = (nv.Int8Weight.quantize(draw(n, k) / k ** 0.5) for n, k in ((2 * F, K), (K, F), (V, K)))
        self.bias = draw(2 * F)

    def step(self, x, stream, tokens, k=5):
        """x: the attention's output rows; stream: the residual stream.  All that it makes, by name."""
        import torch
        nv, o = self.nv, {}
        o["q1"], o["s1"], o["h1"] = nv.rms_norm(x, self.norm1, 1e-6, residual=stream, dtype=torch.int8)
        o["gu"] = nv.int8_gemm(o["q1"], o["s1"], self.gate_up, bias=self.bias)
        o["q2"], o["s2"] = nv.int8_quantize(o["gu"], swiglu=True)
        o["mlp"] = nv.int8_gemm(o["q2"], o["s2"], self.down)
        o["y"], o["h2"] = nv.rms_norm(o["mlp"], self.norm2, 1e-6, residual=o["h1"], weight_offset=1.0)
        o["q3"], o["s3"] = nv.int8_quantize(o["y"])
        o["logits"] = nv.int8_gemm(o["q3"], o["s3"], self.head, dtype=torch.float32)
        o["lp"], o["entropy"], o["top"], o["top_lp"] = nv.logprobs(o["logits"], tokens, k=k)
        return o


def _inputs(rows, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((rows, K), generator=g, device="cuda").to(torch.bfloat16), torch.randn((rows, K), generator=g, device="cuda").to(torch.bfloat16),
            torch.randint(0, V, (rows,), generator=g, device="cuda").to(torch.int32))


def _weights(nv, w):
    import torch
    codes = torch.empty((w.N, w.K), dtype=torch.int8, device="cuda")
    nv.nvfp4_int8_unpack(w.packed, w.K, w.N, codes)
    return host(codes), host(w.scale)


def _product(nv, o, q, s, out, w, bias=None, bf16=True):
    y, mag = oracle.int8_gemm(host(o[q]), host(o[s]), *_weights(nv, w), None if bias is None else host(bias))
    tol = 3.01 * 2.0 ** -24 * mag + 1.01 * 2.0 ** -24 * np.abs(y)
    if bf16:
        tol = tol + 2.0 ** -8 * (np.abs(y) + tol)
    assert (np.abs(host(o[out]).astype(np.float64) - y) <= tol).all(), out


@pytest.mark.parametrize("rows", [1, 8, 64, 300])
def test_each_step_of_a_chain(nv, rows):
    import torch
    m = Model(nv)
    x, stream, tokens = _inputs(rows, rows)
    o = m.step(x, stream, tokens)
    torch.cuda.synchronize()

    def codes(y, q, s):
        want, scale = oracle.codes(y)
        assert np.array_equal(host(o[s]), scale) and np.array_equal(host(o[q]), want), q
    y, h = oracle.rms_norm(host(x), host(m.norm1), 1e-6, 0.0, host(stream), "bf16")
    assert np.array_equal(host(o["h1"]), h)
    codes(y, "q1", "s1")
    _product(nv, o, "q1", "s1", "gu", m.gate_up, m.bias)
    codes(oracle.swiglu(host(o["gu"])), "q2", "s2")
    _product(nv, o, "q2", "s2", "mlp", m.down)
    y, h = oracle.rms_norm(host(o["mlp"]), host(m.norm2), 1e-6, 1.0, host(o["h1"]), "bf16")
    assert np.array_equal(host(o["h2"]), h) and np.array_equal(host(o["y"]), oracle.bf16(y))
    codes(host(o["y"]), "q3", "s3")
    _product(nv, o, "q3", "s3", "logits", m.head, bf16=False)
    lp, H, top, top_lp, *_ = oracle.logprobs(host(o["logits"]), host(tokens), 5, 1.0)
    assert np.array_equal(host(o["top"]), top)
    for got, want in ((host(o["lp"]), lp[:, 0]), (host(o["entropy"]), H), (host(o["top_lp"]), top_lp)):
        assert np.allclose(got, want, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("rows", [8, 100])
def test_captured_and_replayed(nv, rows):
    """Two graphs that share one pool, replayed in turn with new inputs and eager work between: each replay equals the
    eager result."""
    import torch
    m = Model(nv, 1)
    held = [t.clone() for t in _inputs(rows, 0)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step(*held)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0][0].pool() if graphs else None):
            o = m.step(*held)
        graphs.append((g, o))
    for n in range(6):
        for a, b in zip(held, _inputs(rows, 10 + n)):
            a.copy_(b)
        g, o = graphs[n % 2]
        g.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in o.items()}
        want = m.step(*held)
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(got[k], want[k]), (n, k)


@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_a_stream_of_the_callers(nv, kind):
    """Results on a stream of the caller's equal those on the current one, while the current one allocates and
    overwrites what it is given."""
    import torch
    m = Model(nv, 2)
    x, stream, tokens = _inputs(100, 3)
    want = m.step(x, stream, tokens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = side if kind == "stream" else side.cuda_stream
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    q, sc, h = nv.rms_norm(x, m.norm1, 1e-6, residual=stream, dtype=torch.int8, stream=s)
    gu = nv.int8_gemm(q, sc, m.gate_up, bias=m.bias, stream=s)
    q2, s2 = nv.int8_quantize(gu, swiglu=True, stream=s)
    mlp = nv.int8_gemm(q2, s2, m.down, stream=s)
    got = nv.logprobs(want["logits"], tokens, k=5, stream=s)
    held = [torch.full_like(t, 1) for t in (q, sc, h, gu, q2, s2, mlp, *got) for _ in range(3)]
    side.synchronize()
    for a, b in zip((q, sc, h, gu, q2, s2, mlp, *got), ("q1", "s1", "h1", "gu", "q2", "s2", "mlp", "lp", "entropy", "top", "top_lp")):
        assert torch.equal(a, want[b]), b
    mine = {(t.data_ptr(), t.numel() * t.element_size()) for t in held}
    for t in (q, sc, h, gu, q2, s2, mlp, *got):
        assert all(p + n <= t.data_ptr() or t.data_ptr() + t.numel() * t.element_size() <= p for p, n in mine)


def test_two_streams_at_once(nv):
    """Calls of two streams at the same time share nothing."""
    import torch
    m = Model(nv, 4)
    ins = [_inputs(r, 20 + r) for r in (100, 8)]
    want = [m.step(*i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [[] for _ in ins]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[n].append(m.step(*ins[n]))
    torch.cuda.synchronize()
    for n, w in enumerate(want):
        for o in got[n]:
            for k in w:
                assert torch.equal(o[k], w[k]), (n, k)


def test_pieces_captured_and_replayed(nv):
    """A product cut along K, whose pieces' sums lie in a workspace that two graphs share, on two widths."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    w = nv.Int8Weight.quantize(torch.randn((512, 17408), generator=g, device="cuda"))
    held = {M: nv.int8_quantize(torch.randn((M, 17408), generator=g, device="cuda")) for M in (100, 40)}
    for M in held:
        assert nv.nvfp4_int8_gemm_workspace_bytes(M, 17408, 512) > 0
        nv.int8_gemm(*held[M], w)
    torch.cuda.synchronize()
    graphs = {}
    for M in held:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=next(iter(graphs.values()))[0].pool() if graphs else None):
            out = nv.int8_gemm(*held[M], w)
        graphs[M] = graph, out
    for n in range(6):
        M = (100, 40)[n % 2]
        q, s = nv.int8_quantize(torch.randn((M, 17408), generator=g, device="cuda"))
        held[M][0].copy_(q)
        held[M][1].copy_(s)
        graphs[M][0].replay()
        torch.cuda.synchronize()
        got = graphs[M][1].clone()
        assert torch.equal(got, nv.int8_gemm(q, s, w)), n
        acc = q.double() @ w_double(nv, w).t()
        y = acc * s.double()[:, None] * w.scale.double()
        assert ((got.double() - y).abs() <= 2.0 ** -8 * y.abs() * 1.001).all()


def w_double(nv, w):
    import torch
    codes = torch.empty((w.N, w.K), dtype=torch.int8, device="cuda")
    nv.nvfp4_int8_unpack(w.packed, w.K, w.N, codes)
    return codes.double()
