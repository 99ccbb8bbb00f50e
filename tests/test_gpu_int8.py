"""GPU parity of the 8-bit product against exact sums, and of its packed layout."""
import numpy as np
import pytest

from oracle import rows as oracle
from tests.gpu_util import canary_out, dev, host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


def _case(seed, M, K, N):
    rng = np.random.default_rng(seed)
    a, w = rng.integers(-128, 128, (M, K), dtype=np.int8), rng.integers(-128, 128, (N, K), dtype=np.int8)
    return a, (rng.random(M) + 0.5).astype(np.float32), w, ((rng.random(N) + 0.5) / 1000).astype(np.float32), rng.standard_normal(N).astype(np.float32) * 30


def _check(out, y, s, bf16, what):
    """The sum is exact; its conversion and two products round by 2^-24 each, the bias's addition once more,
    bf16 by half a step (2^-8 of the value, at most)."""
    o = host(out).astype(np.float64)
    tol = 3.01 * 2.0 ** -24 * s + 1.01 * 2.0 ** -24 * np.abs(y)
    if bf16:
        tol = tol + 2.0 ** -8 * (np.abs(y) + tol)
    bad = ~(np.abs(o - y) <= tol)
    assert not bad.any(), "%s: %d of %d outside the bound, first %s: %r, not %r" % (what, bad.sum(), bad.size, np.argwhere(bad)[0], o[bad][0], y[bad][0])


@pytest.mark.parametrize("K,N", [(16, 1), (48, 17), (64, 16), (80, 100), (1040, 1003), (2048, 64), (5120, 272), (17408, 33)])
def test_pack_is_a_bijection(nv, K, N):
    import torch
    _, _, w, s, _ = _case(K + N, 1, K, N)
    p = nv.Int8Weight.from_canonical(dev(w), dev(s))
    back = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    nv.nvfp4_int8_unpack(p.packed, K, N, back)
    assert np.array_equal(host(back), w)
    tiles, steps = -(-N // 16), 2 * -(-K // 128)
    whole = np.zeros((tiles * 16, steps * 64), np.int8)
    whole[:N, :K] = w
    want = whole.reshape(tiles, 16, steps, 4, 16).transpose(0, 2, 3, 1, 4)
    assert np.array_equal(host(p.packed).reshape(want.shape), want)


WIDTHS = [1, 2, 5, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300, 511, 700]


@pytest.mark.parametrize("M", WIDTHS)
def test_product(nv, M):
    import torch
    for i, (K, N) in enumerate([(16, 1), (48, 17), (64, 256), (80, 100), (528, 1003), (2048, 300)]):
        a, sa, w, sw, bias = _case(M * 100 + i, M, K, N)
        weight = nv.Int8Weight.from_canonical(dev(w), dev(sw))
        for bf16 in (False, True):
            b = bias if (i + bf16) % 2 else None
            y, s = oracle.int8_gemm(a, sa, w, sw, b)
            out, canary = canary_out(M, N, torch.bfloat16 if bf16 else torch.float32)
            nv.int8_gemm(dev(a), dev(sa), weight, dtype=out.dtype, bias=None if b is None else dev(b), out=out)
            torch.cuda.synchronize()
            canary((M, K, N))
            _check(out, y, s, bf16, (M, K, N, bf16))


@pytest.mark.parametrize("M", [20, 70, 130, 300])
def test_every_number_of_stages(nv, M):
    """K in stages of 128, from one to more than the pieces of a long sum have; the last one whole or begun."""
    import torch
    for stages in list(range(1, 27)) + [40, 47, 62, 97, 136, 203]:
        K, N = 128 * stages - 16 * (stages % 3), 300
        a, sa, w, sw, _ = _case(M * 1000 + stages, M, K, N)
        y, s = oracle.int8_gemm(a, sa, w, sw, None)
        out = nv.int8_gemm(dev(a), dev(sa), nv.Int8Weight.from_canonical(dev(w), dev(sw)), dtype=torch.float32)
        _check(out, y, s, False, (M, K, N))


@pytest.mark.parametrize("M", [17, 24, 31, 32, 33])
@pytest.mark.parametrize("K,N", [(4112, 8192), (5120, 8200), (6000, 12289), (8192, 8192), (8208, 8192)])
def test_streamed_groups_of_rows(nv, M, K, N):
    """Widths that are streamed in two groups of rows, and their neighbours that are not; wide matrices by sampled columns."""
    import torch
    a, sa, w, sw, bias = _case(M + K + N, M, K, N)
    weight = nv.Int8Weight.from_canonical(dev(w), dev(sw))
    at = np.unique(np.concatenate([np.arange(24), np.arange(N - 40, N), np.random.default_rng(M).integers(0, N, 200)]))
    y, s = oracle.int8_gemm(a, sa, w[at], sw[at], bias[at])
    for bf16 in (False, True):
        out, canary = canary_out(M, N, torch.bfloat16 if bf16 else torch.float32)
        nv.int8_gemm(dev(a), dev(sa), weight, dtype=out.dtype, bias=dev(bias), out=out)
        torch.cuda.synchronize()
        canary((M, K, N))
        _check(out[:, torch.from_numpy(at).cuda()], y, s, bf16, (M, K, N, bf16))
        if not bf16:
            part = nv.int8_gemm(dev(a[:9]), dev(sa[:9]), weight, dtype=torch.float32, bias=dev(bias))
            assert torch.equal(part, out[:9])


@pytest.mark.parametrize("M", [1, 4, 5, 9, 16])
@pytest.mark.parametrize("K,N", [(12288, 100), (12304, 100), (17408, 2048), (17408, 6400), (20480, 33), (20496, 33)])
def test_long_rows(nv, M, K, N):
    """Sums of more than 12 steps a wave, streamed or as tiles."""
    import torch
    a, sa, w, sw, bias = _case(M + K + N, M, K, N)
    out = nv.int8_gemm(dev(a), dev(sa), nv.Int8Weight.from_canonical(dev(w), dev(sw)), dtype=torch.float32, bias=dev(bias))
    at = np.unique(np.concatenate([np.arange(min(N, 24)), np.arange(max(0, N - 40), N)]))
    y, s = oracle.int8_gemm(a, sa, w[at], sw[at], bias[at])
    _check(out[:, torch.from_numpy(at).cuda()], y, s, False, (M, K, N))


# The round's matrices and the head's width, by sampled columns; prefill chunks with ragged ends.
@pytest.mark.parametrize("M,K,N", [(8, 5120, 7168), (3, 6144, 5120), (64, 17408, 5120), (8, 5120, 152064), (24, 5120, 34816),
                                   (2048, 5120, 7168), (2048, 6144, 5120), (1000, 17408, 5120), (333, 5136, 6001), (2048, 5120, 17408)])
def test_full_size(nv, M, K, N):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    a = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sw = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    out = nv.int8_gemm(a, sa, nv.Int8Weight.from_canonical(w, sw), dtype=torch.float32)
    again = nv.int8_gemm(a, sa, nv.Int8Weight.from_canonical(w, sw), dtype=torch.float32)
    assert torch.equal(out, again)
    rng = np.random.default_rng(1)
    cols = np.unique(np.concatenate([[0, N - 1], rng.integers(0, N, 300), np.arange(max(0, N - 40), N)]))
    rows = np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, 300)]))
    at = torch.from_numpy(cols).cuda()
    y, s = oracle.int8_gemm(host(a), host(sa), host(w[at]), host(sw[at]))
    _check(out[:, at], y, s, False, (M, K, N, "columns"))
    at = torch.from_numpy(rows).cuda()
    a64 = a[at].cpu().numpy()
    acc = a64.astype(np.float32).astype(np.float64)[:40] @ host(w).astype(np.float64).T if N < 40000 else None
    if acc is not None:
        y = acc * host(sa[at]).astype(np.float64)[:40, None] * host(sw).astype(np.float64)
        _check(out[at[:40]], y, np.abs(y), False, (M, K, N, "rows"))


def test_results_do_not_depend_on_the_width(nv):
    import torch
    a, sa, w, sw, bias = _case(3, 300, 1552, 530)
    weight = nv.Int8Weight.from_canonical(dev(w), dev(sw))
    whole = nv.int8_gemm(dev(a), dev(sa), weight, dtype=torch.float32, bias=dev(bias))
    for M in (1, 7, 16, 30, 64, 65, 130, 257):
        part = nv.int8_gemm(dev(a[:M]), dev(sa[:M]), weight, dtype=torch.float32, bias=dev(bias))
        assert torch.equal(part, whole[:M]), M


@pytest.mark.parametrize("M", [1, 8, 40, 64, 70, 300])
def test_strided_rows(nv, M):
    """Rows apart, outputs apart and off 16 bytes; what lies between them stays."""
    import torch
    K, N = 208, 77
    a, sa, w, sw, bias = _case(M, M, K, N)
    weight = nv.Int8Weight.from_canonical(dev(w), dev(sw))
    wide = torch.full((M, K + 48), 127, dtype=torch.int8, device="cuda")
    wide[:, :K] = dev(a)
    y, s = oracle.int8_gemm(a, sa, w, sw, bias)
    for ld, skip in ((N, 1), (N + 3, 0), (80, 0), (96, 5)):
        for t in (torch.float32, torch.bfloat16):
            buf = torch.full((M * ld + skip,), 5.0, dtype=t, device="cuda")
            out = buf[skip:].view(M, ld)[:, :N]
            nv.int8_gemm(wide[:, :K], dev(sa), weight, dtype=t, bias=dev(bias), out=out)
            _check(out, y, s, t is torch.bfloat16, (M, ld, skip))
            assert (buf[skip:].view(M, ld)[:, N:] == 5.0).all() and (buf[:skip] == 5.0).all()


def test_the_longest_sum(nv):
    """-128 times -128 over the largest K: 2^31 less 262144."""
    import torch
    K = nv.INT8_MAX_K
    for M in (1, 20, 70):
        a, w = np.full((M, K), -128, np.int8), np.full((5, K), -128, np.int8)
        w[1] = 127
        out = nv.int8_gemm(dev(a), torch.ones(M, device="cuda"), nv.Int8Weight.from_canonical(dev(w), torch.ones(5, device="cuda")), dtype=torch.float32)
        want = np.float32(np.array([16384, -16256, 16384, 16384, 16384], np.float64) * K)
        assert np.array_equal(host(out), np.broadcast_to(want, (M, 5)))


def test_scales_that_are_no_numbers(nv):
    """A row of a NaN or an infinity gives NaN in its row alone."""
    import torch
    x = torch.randn((4, 64), device="cuda")
    x[1, 3], x[2, 9] = float("nan"), float("inf")
    q, s = nv.int8_quantize(x)
    w = torch.randn((40, 64), device="cuda")
    out = nv.int8_gemm(q, s, nv.Int8Weight.quantize(w), dtype=torch.float32)
    bad = torch.isnan(out).all(1).tolist()
    assert bad == [False, True, True, False] and torch.isfinite(out[::3]).all()
