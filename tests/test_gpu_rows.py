"""GPU parity of the norm and the 8-bit rows: bit for bit against the fp64 oracle."""
import numpy as np
import pytest

from oracle import rows as oracle
from tests.gpu_util import canary_out, host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


def _types():
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8}


def _dev(x, name, pad=0, skip=0):
    """A device matrix of a type, its rows `pad` values apart beyond their width and `skip` from the start of memory."""
    import torch
    t = torch.zeros(skip + x.shape[0] * (x.shape[1] + pad), dtype=_types()[name], device="cuda")
    v = t[skip:].view(x.shape[0], x.shape[1] + pad)[:, :x.shape[1]]
    v.copy_(torch.from_numpy(np.asarray(x, np.float32)))
    return v


def _values(rng, rows, K, name, wide=False):
    x = rng.standard_normal((rows, K))
    if wide:
        x *= np.exp2(rng.integers(-20, 20, (rows, 1)))
    x.flat[rng.choice(x.size, min(3, x.size), replace=False)] = [0.0, -0.0, 12.5][:min(3, x.size)]
    return oracle.to_type(x, name)


def _same(got, want, what):
    got, want = host(got).astype(np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    bad = ~((got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), "%s: %d of %d differ, first %s: %r, not %r" % (what, bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], want[bad][0])


# Row lengths around what 64, 256 and 1024 threads hold (1536, 6144, 24576), aligned or not; rows next to
# each other or apart; every type.
LENGTHS = [1, 7, 8, 16, 100, 1000, 1001, 1536, 1544, 5120, 5121, 6144, 6152, 17408, 24576, 24584, 30001, 49152]


@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("out", ["bf16", "f32", "int8"])
def test_norm(nv, K, out):
    import torch
    rng = np.random.default_rng(K)
    for rows, x_type, r_type, w_type, pad, offset in ((5, "bf16", "bf16", "bf16", 0, 0.0), (3, "bf16", "f32", "f32", 8, 1.0),
                                                      (2, "f32", "bf16", "bf16", 3, 0.0), (1, "f32", "f32", "f32", 0, 0.5),
                                                      (9, "bf16", None, "bf16", 0, 0.0), (2, "f32", None, "bf16", 8, 1.0)):
        what = (K, out, rows, x_type, r_type)
        x, w = _values(rng, rows, K, x_type, True), _values(rng, 1, K, w_type)[0]
        r = None if r_type is None else _values(rng, rows, K, r_type, True)
        y, h = oracle.rms_norm(x, w, 1e-5, offset, r, r_type)
        res = None if r is None else _dev(r, r_type, pad)
        got = nv.rms_norm(_dev(x, x_type, pad), _dev(w[None], w_type)[0], 1e-5, residual=res, dtype=_types()[out], weight_offset=offset)
        got = list(got) if isinstance(got, tuple) else [got]
        torch.cuda.synchronize()
        if r is not None:
            _same(got.pop(), h, what + ("residual",))
            _same(res, r, what + ("untouched",))
        if out == "int8":
            q, s = oracle.codes(y)
            _same(got[1], s, what + ("scale",))
            _same(got[0], q, what + ("codes",))
        else:
            _same(got[0], oracle.to_type(y, out), what)


@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("swiglu", [False, True])
def test_quantize(nv, K, swiglu):
    import torch
    rng = np.random.default_rng(K + swiglu)
    for rows, name, pad, skip in ((5, "bf16", 0, 0), (2, "f32", 8, 0), (3, "bf16", 3, 1), (1, "f32", 0, 1)):
        x = _values(rng, rows, K * (1 + swiglu), name, not swiglu)
        q, s = oracle.codes(oracle.swiglu(x) if swiglu else x)
        got, scale = nv.int8_quantize(_dev(x, name, pad, skip), swiglu=swiglu)
        torch.cuda.synchronize()
        _same(scale, s, (K, name, "scale"))
        _same(got, q, (K, name, "codes"))


def test_outputs_in_place_and_apart(nv):
    """residual_out is the residual, out is x; and rows apart leave what lies between them alone."""
    import torch
    rng = np.random.default_rng(5)
    for K in (40, 1001, 5120, 30000):
        x, r, w = _values(rng, 4, K, "bf16"), _values(rng, 4, K, "bf16"), _values(rng, 1, K, "bf16")[0]
        y, h = oracle.rms_norm(x, w, 0.0, 0.0, r, "bf16")
        xd, rd = _dev(x, "bf16", 24), _dev(r, "bf16", 8)
        whole = rd.as_strided((4, K + 8), (K + 8, 1))
        whole[:, K:] = 7.0
        got, stream = nv.rms_norm(xd, _dev(w[None], "bf16")[0], 0.0, residual=rd, residual_out=rd, out=xd)
        assert got.data_ptr() == xd.data_ptr() and stream.data_ptr() == rd.data_ptr()
        _same(xd, oracle.bf16(y), K)
        _same(rd, h, K)
        assert (whole[:, K:] == 7.0).all() and (xd.as_strided((3, 24), (K + 24, 1), K) == 0).all()
    for K in (33, 48, 5120):
        buf = torch.full((6, K + 16), 99, dtype=torch.int8, device="cuda")
        x = _values(rng, 6, K, "f32")
        q, s = oracle.codes(x)
        codes, scale = nv.int8_quantize(_dev(x, "f32"), codes=buf[:, :K])
        _same(codes, q, K)
        assert (buf[:, K:] == 99).all()


def test_the_end_of_the_output(nv):
    import torch
    rng = np.random.default_rng(6)
    for K in (5, 1001, 5120, 24584):
        for t in (torch.bfloat16, torch.float32):
            out, canary = canary_out(3, K, t)
            nv.rms_norm(_dev(_values(rng, 3, K, "f32"), "f32"), torch.ones(K, device="cuda"), 1e-6, dtype=t, out=out)
            torch.cuda.synchronize()
            canary(K)
            assert torch.isfinite(out).all()


def test_special_rows(nv):
    """Zeros, infinities and NaN stay in their row; the smallest and largest values."""
    import torch
    K = 96
    x = np.ones((8, K))
    x[0] = 0.0
    x[1, 5] = np.inf
    x[2, 7] = np.nan
    x[3] = 2.0 ** -149
    x[4] = np.linspace(-1, 1, K) * 3.3e38
    x[5] = np.arange(K) * 2.0 ** -149
    x[6] = -0.0
    x = x.astype(np.float32).astype(np.float64)
    q, s = oracle.codes(x)
    codes, scale = nv.int8_quantize(_dev(x, "f32"))
    _same(scale, s, "scale")
    _same(codes, q, "codes")
    w = np.linspace(0.5, 2, K).astype(np.float32)
    for eps in (0.0, 1e-6):
        y, _ = oracle.rms_norm(x, w, eps)
        got = nv.rms_norm(_dev(x, "f32"), torch.from_numpy(w).cuda(), eps, dtype=torch.float32)
        _same(got, oracle.to_type(y, "f32"), "norm")
        q, s = oracle.codes(y)
        codes, scale = nv.rms_norm(_dev(x, "f32"), torch.from_numpy(w).cuda(), eps, dtype=torch.int8)
        _same(scale, s, "scale")
        _same(codes, q, "codes")


def test_ties_go_to_the_even_code(nv):
    """Scales whose inverse is not exact, and values half way between two codes."""
    for m in (1.0, 3.0, 5.0, 7.0, 49.0, 0.1875, 65521.0):
        x = np.concatenate([[127.0], np.arange(-126, 127) + 0.5]) * m
        assert (x.astype(np.float32) == x).all()
        q, s = oracle.codes(x[None])
        assert s[0] == np.float32(m)
        codes, scale = nv.int8_quantize(_dev(x[None], "f32"))
        _same(scale, s, m)
        _same(codes, q, m)


def test_many_rows(nv):
    import torch
    rng = np.random.default_rng(8)
    x = _values(rng, 70001, 24, "bf16")
    q, s = oracle.codes(x)
    codes, scale = nv.int8_quantize(_dev(x, "bf16"))
    _same(scale, s, "scale")
    _same(codes, q, "codes")
    y, _ = oracle.rms_norm(x, np.ones(24), 1e-6)
    _same(nv.rms_norm(_dev(x, "bf16"), torch.ones(24, device="cuda"), 1e-6), oracle.bf16(y), "norm")


def test_swiglu_of_extreme_gates(nv):
    """Exponentials past fp32 either way, rows of nothing but such values, tiny and huge rows."""
    rng = np.random.default_rng(11)
    K = 1032
    rows = []
    for scale, up in ((30, 1), (100, 1), (300, 1), (1e4, 1e3), (1, 1e-25), (1e-25, 1), (1, 1e25), (60, 1e18), (120, 1e30), (3e37, 1), (1e-38, 1e-3)):
        rows.append(np.concatenate([rng.standard_normal(K) * scale, rng.standard_normal(K) * up]))
    rows.append(np.concatenate([np.full(K, -90.0), rng.standard_normal(K)]))      # every value below fp32's least
    rows.append(np.concatenate([np.full(K, -88.0), rng.standard_normal(K) * 1e30]))
    rows.append(np.concatenate([np.full(K, -300.0), rng.standard_normal(K) * 1e38]))
    rows.append(np.concatenate([-np.abs(rng.standard_normal(K)) * 40, rng.standard_normal(K)]))
    for name in ("f32", "bf16"):
        with np.errstate(over="ignore"):
            x = oracle.to_type(np.stack(rows), name)
        q, s = oracle.codes(oracle.swiglu(x))
        codes, scale = nv.int8_quantize(_dev(x, name), swiglu=True)
        _same(scale, s, name)
        _same(codes, q, name)


def test_norm_of_extreme_rows(nv):
    """Tiny and huge values and weights beside ordinary ones, to every type."""
    import torch
    rng = np.random.default_rng(12)
    K = 520
    x = rng.standard_normal((7, K))
    x[0] *= 1e-38
    x[1] *= 1e37
    x[2, ::3] *= 1e-36
    x[3, ::5] *= 1e-30
    x[4] = 0
    x[4, 7] = 1e-40
    x[5, ::2] = 0
    x[6, 1:] *= 1e-12
    for w in (rng.standard_normal(K), np.zeros(K), rng.standard_normal(K) * 1e30, np.where(rng.random(K) < 0.5, 0, 1e-20), rng.standard_normal(K) * 2.0 ** 45):
        for name in ("f32", "bf16"):
            v, wv = oracle.to_type(x, name), oracle.to_type(w, "f32")
            for eps in (0.0, 1e-6, 1e36):
                y, _ = oracle.rms_norm(v, wv, eps)
                wd = torch.from_numpy(wv.astype(np.float32)).cuda()
                for t in ("bf16", "f32"):
                    _same(nv.rms_norm(_dev(v, name), wd, eps, dtype=_types()[t]), oracle.to_type(y, t), (name, eps, t))
                q, s = oracle.codes(y)
                codes, scale = nv.rms_norm(_dev(v, name), wd, eps, dtype=torch.int8)
                _same(scale, s, (name, eps))
                _same(codes, q, (name, eps))


def test_codes_of_many_draws(nv):
    """Millions of values, tens of thousands of them next to a border of fp32's error."""
    import torch
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn((256, 8192), generator=g, device="cuda").to(torch.bfloat16)
        for swiglu in (False, True):
            y = x.double()
            if swiglu:
                y = y[:, :4096] * y[:, 4096:] / (1 + torch.exp(-y[:, :4096]))
            s = (y.abs().amax(1) / 127).float()
            codes, scale = nv.int8_quantize(x, swiglu=swiglu)
            assert torch.equal(scale, s) and torch.equal(codes, torch.round(y / s.double()[:, None]).to(torch.int8))
        h = x.double()
        w = torch.randn(8192, generator=g, device="cuda").to(torch.bfloat16)
        y = h * (h.square().mean(1, keepdim=True) + float(np.float32(1e-6))).rsqrt() * w.double()
        s = (y.abs().amax(1) / 127).float()
        codes, scale = nv.rms_norm(x, w, 1e-6, dtype=torch.int8)
        assert torch.equal(scale, s) and torch.equal(codes, torch.round(y / s.double()[:, None]).to(torch.int8))
        out = nv.rms_norm(x, w, 1e-6).double()
        low = torch.nextafter(out.to(torch.bfloat16), torch.full_like(x, -float("inf"))).double()
        high = torch.nextafter(out.to(torch.bfloat16), torch.full_like(x, float("inf"))).double()
        assert ((y - out).abs() <= torch.minimum((y - low).abs(), (y - high).abs())).all()
