"""GPU parity of every vector that a thread of the row kernels holds: lengths up to each kernel's last value, on both sides of
the number of rows that chooses between them, for every kind of row and type."""
import numpy as np
import pytest

from oracle import rows as oracle
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

KINDS = 23  # distinct rows, repeated


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


def _types():
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8}


def _rows(rng, K, name):
    x = rng.standard_normal((KINDS, K)) * np.exp2(rng.integers(-8, 8, (KINDS, 1)))
    x[0] = 0.0
    for i in range(1, KINDS):  # the largest value of a row in each part of it
        x[i, i * (K - 1) // (KINDS - 1)] = (-1) ** i * 9.0 * np.abs(x[i]).max()
    return oracle.to_type(x, name)


def _dev(x, rows, name, pad=0):
    import torch
    t = torch.from_numpy(np.asarray(x, np.float32)).cuda().to(_types()[name])
    out = torch.zeros((rows, x.shape[1] + pad), dtype=t.dtype, device="cuda")[:, :x.shape[1]]
    return out.copy_(t[torch.arange(rows, device="cuda") % KINDS])


def _same(got, want, what):
    import torch
    want = torch.from_numpy(np.asarray(want, np.float64)).cuda()[torch.arange(got.shape[0], device="cuda") % KINDS]
    bad = ~((got.double() == want) | (got.double().isnan() & want.isnan()))
    assert not bad.any(), "%s: %d of %d differ, first %s: %r, not %r" % (
        what, bad.sum(), bad.numel(), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item())


# 64 threads hold up to 512, 1024 and 1536 values in one, two and three vectors; 256 threads 2048, 4096 and 6144; 1024 threads 8192,
# 16384 and 24576.  Of 4097 to 8192 values 1024 threads take rows up to 512, and above 6144 all of them, in one vector each.
SIZES = ([(9, K) for K in (512, 520, 1024, 1032, 1528, 1536, 2048, 2056, 4088, 4096, 4104, 6144, 8184, 8192, 8200, 16384, 16392, 24576)]
         + [(512, 4104), (512, 5120), (512, 6144)] + [(513, K) for K in (4096, 4104, 5120, 6136, 6144, 6152, 8192)] + [(9, K) for K in (1025, 1535, 2049, 4097, 6143)])


@pytest.mark.parametrize("rows,K", SIZES)
def test_norm(nv, rows, K):
    rng = np.random.default_rng(rows + K)
    for x_type, r_type, w_type, pad, offset in (("bf16", "bf16", "bf16", 0, 0.0), ("bf16", "f32", "bf16", 8, 1.0), ("f32", "bf16", "f32", 0, 0.0),
                                                ("bf16", None, "bf16", 8, 0.0), ("f32", None, "bf16", 0, 0.5)):
        x, w = _rows(rng, K, x_type), oracle.to_type(rng.standard_normal(K), w_type)
        r = None if r_type is None else _rows(rng, K, r_type)
        y, h = oracle.rms_norm(x, w, 1e-5, offset, r, r_type)
        xd, res = _dev(x, rows, x_type, pad), None if r is None else _dev(r, rows, r_type, pad)
        wd = _dev(np.broadcast_to(w, (KINDS, K)), 1, w_type)[0]
        for out in ("bf16", "f32", "int8"):
            what = (rows, K, x_type, r_type, out)
            got = nv.rms_norm(xd, wd, 1e-5, residual=res, dtype=_types()[out], weight_offset=offset)
            got = list(got) if isinstance(got, tuple) else [got]
            if r is not None:
                _same(got.pop(), h, what + ("residual",))
            if out == "int8":
                q, s = oracle.codes(y)
                _same(got[1], s, what + ("scale",))
                _same(got[0], q, what + ("codes",))
            else:
                _same(got[0], oracle.to_type(y, out), what)


@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("swiglu", [False, True])
def test_quantize(nv, rows, K, swiglu):
    rng = np.random.default_rng(rows + K + swiglu)
    for name, pad in (("bf16", 0), ("f32", 8)):
        x = _rows(rng, K, name)
        if swiglu:
            with np.errstate(over="ignore"):
                x = np.concatenate([np.clip(x, -40, 40) if name == "f32" else oracle.bf16(np.clip(x, -40, 40)), _rows(rng, K, name)], axis=1)
        q, s = oracle.codes(oracle.swiglu(x) if swiglu else x)
        got, scale = nv.int8_quantize(_dev(x, rows, name, pad), swiglu=swiglu)
        _same(scale, s, (rows, K, name, "scale"))
        _same(got, q, (rows, K, name, "codes"))


@pytest.mark.parametrize("K", [1536, 4096, 5121])
def test_rows_at_the_top_of_the_range(nv, K):
    """Rows whose root mean square's inverse is below fp32's normal numbers, and keeps fewer bits there."""
    import torch
    rng = np.random.default_rng(K)
    for name in ("bf16", "f32"):
        x = (1 + 0.98 * rng.random((64, K))) * 2.0 ** 127 * rng.choice([-1, 1], (64, K))
        x[1::2, ::3] *= 2.0 ** -rng.integers(0, 40, x[1::2, ::3].shape)
        x, w = oracle.to_type(x, name), oracle.to_type(rng.standard_normal(K), "bf16")
        assert np.isfinite(x).all() and (1 / np.sqrt((x * x).mean(axis=1)) < 2.0 ** -126).all()
        y, _ = oracle.rms_norm(x, w, 0.0)
        xd, wd = (torch.from_numpy(v.astype(np.float32)).cuda().to(_types()[t]) for v, t in ((x, name), (w, "bf16")))
        for out in ("bf16", "f32"):
            got = nv.rms_norm(xd, wd, 0.0, dtype=_types()[out])
            assert np.array_equal(got.double().cpu().numpy(), oracle.to_type(y, out)), (K, name, out)
        q, s = oracle.codes(y)
        codes, scale = nv.rms_norm(xd, wd, 0.0, dtype=torch.int8)
        assert np.array_equal(scale.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy(), q), (K, name)
