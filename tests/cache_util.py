"""Inputs and bounds shared by the paged-cache tests (not a test module)."""
from __future__ import annotations

import numpy as np

from tests.gpu_util import host


def bf16(x):
    """Nearest bf16 of float64 values, as float64 (ties to even)."""
    import torch
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


class Lanes:
    """Lanes of a cache: contexts, rows, and a table over pages in random order."""

    def __init__(self, seed, ctx, rows, page, spare=3):
        rng = np.random.default_rng(seed)
        need = [-(-(c + r) // page) for c, r in zip(ctx, rows)]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(ctx), max(max(need), 1) + 1), -1, np.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.ctx = np.array(ctx, np.int32)
        self.start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.rows = rows

    def dev(self):
        import torch
        return [torch.from_numpy(x).cuda() for x in (self.start, self.ctx, self.table)]


def cache_tensors(seed, layers, pages, heads, page, dim, dtype, fill=None):
    """(k, v) device tensors of N(0, 1) draws, or of one byte value everywhere."""
    import torch
    shapes = (layers, pages, heads, page, dim), (layers, pages, heads, page // 16, dim, 16)
    t = torch.float8_e4m3fn if dtype == "e4m3" else torch.bfloat16
    if fill is not None:
        return [torch.full((int(np.prod(s)) * (1 if dtype == "e4m3" else 2),), fill, dtype=torch.uint8, device="cuda").view(t).view(s) for s in shapes]
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").to(t) for s in shapes]


def values(t, scale=1.0):
    """float64 values of a cache tensor."""
    return t.float().cpu().numpy().astype(np.float64) * scale


def chain(n):
    """Mask words of a chain of n drafts, as signed 64-bit integers."""
    return np.array([(2 << t) - 1 if t < 63 else -1 for t in range(n)], np.int64)


def check_attention(out, lse, want, tokens, dim, what):
    """The kernel's results against the oracle's.

    A score is a sum of dim exact products in fp32: off by at most (dim + 8) 2^-24 S, S the sum of
    their magnitudes, the scaling included; exp turns an error d into a relative one of the weight.
    A weight enters the second product with 16 significant bits (2^-17), and the fp32 sums over
    n tokens, split over waves and workers, are off by at most (n + 64) 2^-24 of the sum of
    magnitudes.  Errors of weights come in twice (numerator and denominator).  The bf16 store adds
    half a unit of the last place, at most 2^-8 of the value."""
    y, ylse, absum, smax = want
    o, z = host(out).reshape(y.shape), host(lse).astype(np.float64)
    d = (dim + 8) * 2.0 ** -24 * smax + 2.0 ** -21
    eps = 2 * (d + 2.0 ** -17) + 2 * (tokens + 64) * 2.0 ** -24
    tol = eps[..., None] * absum
    bad = np.abs(o - y) > tol + 2.0 ** -8 * (np.abs(y) + tol)
    assert np.isfinite(o).all(), what
    assert not bad.any(), "%s: %d of %d outputs outside the bound, first %s: %r, not %r" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], o[bad][0], y[bad][0])
    empty = np.isneginf(ylse)
    assert np.array_equal(np.isneginf(z), empty), what
    zt = d + (tokens + 64) * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(empty, 0, ylse))
    badz = np.abs(np.where(empty, 0, z) - np.where(empty, 0, ylse)) > zt
    assert not badz.any(), "%s: lse" % what
