"""GPU parity of the 8-bit product in each of its tiles, in one piece and in several along K, whole and ragged, to both
types, with and without a bias: every output against exact sums."""
import pytest

from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


def _case(M, K, N):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    a = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sw = torch.rand(M, generator=g, device="cuda") + 0.5, (torch.rand(N, generator=g, device="cuda") + 0.5) / 1000
    return a, sa, w, sw, torch.randn(N, generator=g, device="cuda") * 30


def _products(nv, M, K, N, layouts):
    import torch
    a, sa, w, sw, bias = _case(M, K, N)
    weight = nv.Int8Weight.from_canonical(w, sw)
    plain = torch.matmul(a.double(), w.double().t().contiguous()) * sa.double()[:, None] * sw.double()  # (sums are whole numbers below 2^53)
    for b in (None, bias):
        y = plain if b is None else plain + b.double()
        for t in (torch.float32, torch.bfloat16):
            # The sum's conversion and two products round by 2^-24 each, the bias's addition once more, bf16 by half a step.
            tol = 3.01 * 2.0 ** -24 * plain.abs() + 1.01 * 2.0 ** -24 * y.abs()
            if t is torch.bfloat16:
                tol += 2.0 ** -8 * (y.abs() + tol)
            for ld, skip in layouts:
                buf = torch.full((skip + M * ld + 4096,), 5.0, dtype=t, device="cuda")
                out = buf[skip:skip + M * ld].view(M, ld)[:, :N]
                out.fill_(float("nan"))
                nv.int8_gemm(a, sa, weight, dtype=t, bias=b, out=out)
                bad = ~((out.double() - y).abs() <= tol)
                what = (M, K, N, b is not None, t, ld, skip)
                assert not bad.any(), "%s: %d of %d outside the bound, first %s: %r, not %r" % (
                    what, bad.sum(), bad.numel(), bad.nonzero()[0].tolist(), out[bad][0].item(), y[bad][0].item())
                rest = buf[skip:skip + M * ld].view(M, ld)[:, N:]
                assert (rest == 5.0).all() and (buf[:skip] == 5.0).all() and (buf[skip + M * ld:] == 5.0).all(), what


# (as 256 compute units choose)
TILES = [
    (256, 1024, 35072), (2001, 1040, 17403), (245, 224, 92112), (600, 336, 9001), (70, 96, 33440),  # 128 x 256, one piece
    (842, 12512, 2449), (65, 15584, 16821), (279, 14672, 3759),                                     # and several
    (512, 1024, 4992), (333, 5136, 6001), (515, 992, 4957), (2048, 1024, 5120),                     # 128 x 128
    (128, 17408, 5120), (1149, 14800, 530), (356, 12944, 2201), (199, 16176, 1588),
    (477, 1168, 2736), (513, 4096, 2050), (48, 1040, 20003), (64, 512, 17408),                      # 64 x 128
    (64, 17408, 5120), (153, 13360, 5014), (1390, 12272, 121), (520, 8208, 1003),
    (300, 1040, 3001), (668, 64, 1441), (32, 2048, 4096), (100, 5120, 7168),                        # 32 x 128
    (17, 3184, 124), (258, 6416, 245), (73, 12864, 245),
]


@pytest.mark.parametrize("M,K,N", TILES)
def test_tiles(nv, M, K, N):
    """Outputs side by side; off 16 bytes with a stride off them too; and 16-byte rows of a wider buffer."""
    _products(nv, M, K, N, [(N, 0), (N + 3, 1), (-(-N // 16) * 16 + 16, 0)])


@pytest.mark.parametrize("stages", list(range(1, 12)))
@pytest.mark.parametrize("M,N", [(600, 9001), (300, 7001), (48, 20003)])
def test_wide_tiles_by_their_stages(nv, M, N, stages):
    """K of one stage of 128 up, the last one whole or begun."""
    _products(nv, M, 128 * stages - 16 * (stages % 4), N, [(N, 0)])


@pytest.mark.parametrize("M", [1, 7, 16])
@pytest.mark.parametrize("K,N", [(512, 300), (1008, 40003), (2048, 7001), (4096, 70001), (8192, 7001), (8208, 7001), (12288, 7168), (12304, 7001),
                                 (16384, 7001), (17408, 5120), (20480, 7001)])
def test_streamed_by_their_steps(nv, M, K, N):
    """4, 8, 12 and 20 steps a wave, one tile a workgroup and more."""
    _products(nv, M, K, N, [(N, 0), (N + 3, 1)])
