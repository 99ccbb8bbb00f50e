"""fp64 oracle of the paged-cache operators and of beam selection (plain numpy).

Test infrastructure only, like the rest of this package: written from the definitions
in ``include/nvfp4.h`` with loops over lanes and tokens, sharing no code with the HIP
path.  Caches are numpy arrays in the library's layout, K [layers][pages][kv_heads]
[page_tokens][dim] and V [layers][pages][kv_heads][page_tokens / 16][dim][16], holding
the values the cache stands for (scales applied) as float64.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def k_token(k, layer, table, t):
    """K of a lane's token t, [kv_heads][dim] (a view)."""
    tokens = k.shape[3]
    return k[layer, table[t // tokens], :, t % tokens]


def v_token(v, layer, table, t):
    """V of a lane's token t, [kv_heads][dim] (a view)."""
    tokens = 16 * v.shape[3]
    o = t % tokens
    return v[layer, table[t // tokens], :, o // 16, :, o % 16]


def rotate(x, pos, inv_freq, axis=None, interleaved=False, factor=1.0):
    """x [rows][heads][dim] turned by the rows' positions [rows][axes]."""
    pairs = len(inv_freq)
    axis = np.zeros(pairs, int) if axis is None else np.asarray(axis, int)
    a = pos.astype(np.float64)[:, axis] * np.asarray(inv_freq, np.float64)
    c, s = factor * np.cos(a)[:, None], factor * np.sin(a)[:, None]
    i = np.arange(pairs)
    u, w = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    y = x.astype(np.float64).copy()
    y[..., u] = x[..., u] * c - x[..., w] * s
    y[..., w] = x[..., u] * s + x[..., w] * c
    return y


def tree_attention(q, k, v, layer, row_start, ctx, table, mask, scale, q_heads):
    """(out [rows][q_heads][dim], lse [rows][q_heads], A, S): A = sum w |v| / sum w and S, per row
    and head, the largest sum |q k| * scale over the tokens seen, for error bounds."""
    rows, dim = int(row_start[-1]), k.shape[4]
    kv_heads, tokens, pages = k.shape[2], k.shape[3], k.shape[1]
    group = q_heads // kv_heads
    q = np.asarray(q, np.float64).reshape(rows, q_heads, dim)
    out = np.zeros((rows, q_heads, dim))
    absum = np.zeros((rows, q_heads, dim))
    lse = np.full((rows, q_heads), -np.inf)
    smax = np.zeros((rows, q_heads))
    for b in range(len(ctx)):
        r0, r1 = int(row_start[b]), int(row_start[b + 1])
        n = min(int(ctx[b]) + r1 - r0, tokens * table.shape[1])
        here = [t for t in range(n) if 0 <= table[b, t // tokens] < pages]
        if not here or r0 == r1:
            continue
        kk = np.stack([k_token(k, layer, table[b], t) for t in here])
        vv = np.stack([v_token(v, layer, table[b], t) for t in here])
        at = [t - int(ctx[b]) for t in here]
        for r in range(r0, r1):
            word = int(mask[r]) & 0xFFFFFFFFFFFFFFFF
            seen = np.array([j < 0 or (word >> j) & 1 == 1 for j in at])
            if not seen.any():
                continue
            for h in range(q_heads):
                kh, vh = kk[seen, h // group], vv[seen, h // group]
                s = kh @ q[r, h] * scale
                m = s.max()
                w = np.exp(s - m)
                out[r, h] = w @ vh / w.sum()
                absum[r, h] = w @ np.abs(vh) / w.sum()
                lse[r, h] = m + np.log(w.sum())
                smax[r, h] = (np.abs(kh) @ np.abs(q[r, h])).max() * scale
    return out, lse, absum, smax


def append(k, v, layer, qkv, q_heads, row_start, ctx, table, pos, inv_freq, axis=None, interleaved=False, factor=1.0):
    """Writes k and v of the rows into the cache (in place); returns the rotated q [rows][heads][dim]."""
    kv_heads, dim, tokens, pages = k.shape[2], k.shape[4], k.shape[3], k.shape[1]
    x = np.asarray(qkv, np.float64).reshape(-1, q_heads + 2 * kv_heads, dim)
    h = rotate(x[:, :q_heads + kv_heads], pos, inv_freq, axis, interleaved, factor)
    for b in range(len(ctx)):
        for t in range(int(row_start[b + 1]) - int(row_start[b])):
            r, p = int(row_start[b]) + t, int(ctx[b]) + t
            if p // tokens >= table.shape[1] or not 0 <= table[b, p // tokens] < pages:
                continue
            k_token(k, layer, table[b], p)[:] = h[r, q_heads:]
            v_token(v, layer, table[b], p)[:] = x[r, q_heads + kv_heads:]
    return h[:, :q_heads]


def compact(k, v, ctx, table, path, accepted):
    """Moves the accepted drafts (in place, every layer)."""
    tokens, pages, width = k.shape[3], k.shape[1], 16 * v.shape[3] * table.shape[1]
    for layer in range(k.shape[0]):
        for b in range(len(ctx)):
            moves = []
            for j in range(min(max(int(accepted[b]), 0), path.shape[1], 64)):
                s, d, p = int(ctx[b]) + int(path[b, j]), int(ctx[b]) + j, int(path[b, j])
                if not 0 <= p < 64 or s >= width or d >= width:
                    continue
                if all(0 <= table[b, t // tokens] < pages for t in (s, d)):
                    moves.append((d, k_token(k, layer, table[b], s).copy(), v_token(v, layer, table[b], s).copy()))
            for d, kk, vv in moves:
                k_token(k, layer, table[b], d)[:] = kk
                v_token(v, layer, table[b], d)[:] = vv


def update(table, length, refs, parent, keep, reserve, tokens):
    """(table, length, refs, short, copies): the new page tables and the (source, destination) pages."""
    pages, width = len(refs), table.shape[1]
    refs = [int(x) for x in refs]
    valid = lambda p: 0 <= p < pages  # noqa: E731
    for p in table.ravel():
        if valid(p):
            refs[p] -= 1
    new = np.full((len(parent), width), -1, np.int64)
    lens = np.zeros(len(parent), np.int64)
    for i, p in enumerate(parent):
        if 0 <= p < len(table):
            n = min(max(int(length[p]), 0), width * tokens)
            if keep is not None:
                n = min(n, max(int(keep[i]), 0))
            lens[i] = n
            for j in range(-(-n // tokens)):
                if valid(table[p, j]):
                    new[i, j] = table[p, j]
                    refs[table[p, j]] += 1
    last = [int(new[i, (n - 1) // tokens]) if n % tokens else -1 for i, n in enumerate(lens)]
    wants = []  # (lane, entry, source page or None)
    for i, n in enumerate(lens):
        q, held = last[i], -(-int(n) // tokens)
        if q >= 0 and not (last.count(q) == refs[q] and last.index(q) == i):
            wants.append((i, held - 1, q))
        room = 0 if reserve is None else max(int(reserve[i]), 0)
        for j in range(held, min(-(-(int(n) + room) // tokens), width)):
            wants.append((i, j, None))
    free = [p for p in range(pages) if refs[p] == 0]
    copies = []
    for (i, j, q) in wants:
        p = free.pop(0) if free else -1
        new[i, j] = p
        if p >= 0:
            refs[p] = 1
        if q is not None:
            refs[q] -= 1
            if p >= 0:
                copies.append((q, p))
    return new, lens, np.array(refs), sum(1 for i, j, _ in wants if new[i, j] < 0), copies


def beam_scores(logits, score, done, eos):
    """fp64 scores [rows][V] of every candidate."""
    x = np.asarray(logits, np.float64)
    out = np.full(x.shape, -np.inf)
    for r in range(len(x)):
        if score[r] == -np.inf:
            continue
        if done is not None and done[r]:
            out[r, eos] = score[r]
            continue
        m = x[r].max()
        if m == -np.inf:
            continue
        out[r] = float(score[r]) + (x[r] - m) - np.log(np.exp(x[r] - m).sum())
    return out


def beam_select(scores, batch, beams, k):
    """(score, parent, token) of the k best of each request's [beams][V] scores; equal ones by row, then token."""
    V = scores.shape[1]
    flat = scores.reshape(batch, beams * V)
    order = np.argsort(-flat, axis=1, kind="stable")[:, :k]
    return np.take_along_axis(flat, order, 1), order // V + beams * np.arange(batch)[:, None], order % V
