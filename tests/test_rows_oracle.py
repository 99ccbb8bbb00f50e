"""Pins of the row oracle against torch, exact fractions and closed forms."""
from fractions import Fraction

import numpy as np

from oracle import rows


def test_bf16_rounding():
    import torch
    rng = np.random.default_rng(1)
    x = rng.standard_normal(20000) * np.exp2(rng.integers(-140, 128, 20000))
    x = np.concatenate([x, [0.0, -0.0, np.inf, -np.inf, 2.0 ** -133, 2.0 ** -134, 1.5 * 2.0 ** -134, 3.39e38, 3.4028e38]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    assert np.array_equal(rows.bf16(x.astype(np.float64)), want)
    # what fp32 would turn into a tie
    assert rows.bf16(1 + 2.0 ** -8) == 1.0 and rows.bf16(1 + 2.0 ** -8 + 2.0 ** -40) == 1 + 2.0 ** -7
    assert np.isnan(rows.bf16(np.nan))


def test_norm_by_fractions():
    x, w = [3.0, -4.0, 0.5], [1.0, 0.5, -2.0]
    y, h = rows.rms_norm([x], w, 0.25, 1.0)
    mean = sum(Fraction(v) ** 2 for v in x) / 3 + Fraction(1, 4)
    want = [float(Fraction(v) * (Fraction(u) + 1)) / float(mean) ** 0.5 for v, u in zip(x, w)]
    assert np.allclose(y[0], want, rtol=1e-15) and np.array_equal(h[0], x)
    y, h = rows.rms_norm([[1.0]], [1.0], 0.0, 0.0, [[2.0 ** -9]], "bf16")
    assert h[0, 0] == 1.0 and y[0, 0] == 1.0  # the norm is of the stream as it is stored
    y, h = rows.rms_norm([[1.0]], [1.0], 0.0, 0.0, [[2.0 ** -9]], "f32")
    assert h[0, 0] == 1 + 2.0 ** -9


def test_norm_against_torch():
    import torch
    x = np.random.default_rng(2).standard_normal((5, 77))
    w = np.linspace(-1, 2, 77)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (77,), torch.from_numpy(w), float(np.float32(1e-5))).numpy()
    assert np.allclose(rows.rms_norm(x, w, 1e-5)[0], want, rtol=1e-14, atol=0)


def test_swiglu_against_torch():
    import torch
    x = np.random.default_rng(3).standard_normal((4, 20)) * 10
    t = torch.from_numpy(x)
    want = (torch.nn.functional.silu(t[:, :10]) * t[:, 10:]).numpy()
    assert np.allclose(rows.swiglu(x), want, rtol=1e-14, atol=1e-300)


def test_codes_by_fractions():
    x = np.random.default_rng(4).standard_normal((3, 50)).astype(np.float32).astype(np.float64)
    x[2] = np.round(x[2] * 8) * 1.5
    x[2, 0] = 127 * 3.0  # scale 3: multiples of 1.5 are ties
    q, s = rows.codes(x)
    for r in range(3):
        most = max(abs(Fraction(float(v))) for v in x[r])
        near = Fraction(float(s[r]))
        step = Fraction(float(np.spacing(s[r])))
        assert abs(most / 127 - near) <= step / 2
        for v, c in zip(x[r], q[r]):
            exact = Fraction(float(v)) / near
            assert abs(exact - int(c)) < Fraction(1, 2) or (abs(exact - int(c)) == Fraction(1, 2) and int(c) % 2 == 0)
    q, s = rows.codes([[0.0, -0.0], [1.0, np.nan], [np.inf, 1.0]])
    assert not q.any() and s[0] == 0 and np.isnan(s[1]) and np.isinf(s[2])


def test_product_by_integers():
    rng = np.random.default_rng(5)
    a, w = rng.integers(-128, 128, (3, 40), dtype=np.int8), rng.integers(-128, 128, (4, 40), dtype=np.int8)
    y, s = rows.int8_gemm(a, np.float32([1, 2, 0.5]), w, np.float32([1, 1, 4, 1]), np.float32([0, 8, 0, 0]))
    for m in range(3):
        for n in range(4):
            v = sum(int(p) * int(q) for p, q in zip(a[m], w[n])) * [1, 2, 0.5][m] * [1, 1, 4, 1][n]
            assert y[m, n] == v + [0, 8, 0, 0][n] and s[m, n] == abs(v)


def test_logprobs_against_torch():
    import torch
    x = np.random.default_rng(6).standard_normal((4, 300)) * 3
    x[1, :100] = -np.inf
    x[2, 5:20] = x[2, 4]
    tokens = [[0, 299], [50, 150], [4, 19], [-1, 300]]
    lp, H, top, top_lp, every, E, E2 = rows.logprobs(x, tokens, 7, 0.5)
    want = torch.log_softmax(torch.from_numpy(x) * 0.5, 1).numpy()
    assert np.allclose(every, want, rtol=1e-12)
    assert np.allclose(lp[:3], np.take_along_axis(want[:3], np.array(tokens[:3]), 1), rtol=1e-12) and np.isneginf(lp[3]).all()
    assert np.allclose(H, torch.distributions.Categorical(logits=torch.from_numpy(x) * 0.5).entropy().numpy()[[0, 1, 2, 3]], rtol=1e-9)
    for r in range(4):
        by = sorted(range(300), key=lambda i: (-x[r, i], i))[:7]
        assert top[r].tolist() == by and np.array_equal(top_lp[r], every[r, by])
    lp, H, top, top_lp, *_ = rows.logprobs(np.full((1, 3), -np.inf), [[1]], 2, 1.0)
    assert np.isneginf(lp).all() and H[0] == 0 and top.tolist() == [[0, 1]] and np.isneginf(top_lp).all()
    lp, H, *_ = rows.logprobs(np.zeros((1, 8)), [[3]], 0, 1.0)
    assert np.allclose(lp, -np.log(8)) and np.allclose(H, np.log(8))
