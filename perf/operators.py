"""Cases of the operators around a paged key/value cache: what serves a decode round beside its matrix products.

Five operators over one cache (K pages [kv head][token][dim], V pages
[kv head][token / 16][dim][token % 16]):

* ``append``: the rows of a qkv product get rotary positions (one to three axes); q comes back, k and v go into the cache;
* ``attention``: each row attends to its lane's context and to the drafted tokens its mask word names;
* ``update``: page tables are reordered, forked, freed and extended; partly filled pages that get shared are copied;
* ``compact``: the accepted drafts of each lane move to the front of its drafted tokens, in every layer;
* ``beam``: the best continuations over beams and vocabulary.

``run`` with ``own`` false computes them with elementary torch operations in 32 bits, rounded once; with ``own`` true it
makes the calls of ``nvfp4_weight_streaming_amd``.  ``exact`` computes them from their definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

NEG = float("-inf")
DEV = "cuda"


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # The smallest call: one lane, one token, a short chat turn. Latency counts.
        dict(name="decode 1 lane, 300", kind="attention", lanes=1, rows=1, ctx=300, q_heads=24, kv_heads=2, dim=256, page=64,
             cache="bf16"),
        # The decode round's usual width: 8 lanes of one token, mixed context lengths.
        dict(name="decode 8 lanes, 4096", kind="attention", lanes=8, rows=1, ctx=4096, q_heads=48, kv_heads=4, dim=128, page=64,
             cache="bf16"),
        # The widest speculative round (8 lanes x (1 + 7) rows) at full context, over an 8-bit cache.
        dict(name="verify 8 x 8, 40960, 8-bit", kind="attention", lanes=8, rows=8, ctx=40960, q_heads=48, kv_heads=4, dim=128,
             page=64, cache="e4m3"),
        # Large trees: few lanes, 64 drafted tokens each, ragged, long context; the most arithmetic per byte.
        dict(name="trees 4 x 64, 16384", kind="attention", lanes=4, rows=64, ctx=16384, q_heads=48, kv_heads=4, dim=128, page=128,
             cache="bf16"),
        # A verify round's new rows: small and latency bound.
        dict(name="append 8 x 8", kind="append", lanes=8, rows=8, ctx=4100, q_heads=48, kv_heads=4, dim=128, page=64, cache="bf16",
             axes=1, pairs=64, interleaved=False),
        # A prefill chunk with image positions (time, height, width) into an 8-bit cache.
        dict(name="append chunk 2048, 3 axes", kind="append", lanes=1, rows=2048, ctx=8197, q_heads=48, kv_heads=4, dim=128,
             page=64, cache="e4m3", axes=3, pairs=64, interleaved=True),
        # Beam search's reordering after each token: one request, 8 beams, 16 attention layers.
        dict(name="update 8 beams, 4107", kind="update", batch=1, beams=8, ctx=4107, layers=16, kv_heads=4, dim=128, page=64,
             reserve=1),
        # The same for a full batch with long tables.
        dict(name="update 8 x 8 beams, 16391", kind="update", batch=8, beams=8, ctx=16391, layers=2, kv_heads=4, dim=128, page=64,
             reserve=8),
        # After each speculative round: 8 lanes of 8 drafts, 16 attention layers.
        dict(name="compact 8 x 8", kind="compact", lanes=8, rows=8, ctx=4101, layers=16, kv_heads=4, dim=128, page=64,
             cache="bf16"),
        # Large trees of a full batch, small pages, 8-bit cache, every layer.
        dict(name="compact 64 x 64, 8-bit", kind="compact", lanes=64, rows=64, ctx=517, layers=16, kv_heads=4, dim=128, page=16,
             cache="e4m3"),
        # Beam search of one request over the head's logits.
        dict(name="beam 1 x 4", kind="beam", batch=1, beams=4, V=152064, k=8, logits="f32"),
        # A batch of wide beams, 16-bit logits.
        dict(name="beam 16 x 8, bf16", kind="beam", batch=16, beams=8, V=152064, k=16, logits="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "append", "update", "compact", "beam"])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    kv = rng.choice([1, 2, 4, 8])
    if kind == "attention":
        group = rng.choice([1, 3, 4, 6, 8, 12, 16])
        while True:
            lanes, rows, ctx = _log(rng, 1, 16), rng.choice([1, _log(rng, 1, 64), 8]), _log(rng, 1, 40960)
            if lanes * rows * group * kv * ctx * dim <= 4 * 64 * 12 * 4 * 16384 * 128 // 2 and lanes * ctx * kv * dim <= 8 * 40960 * 4 * 128:
                break
        return dict(kind=kind, lanes=lanes, rows=rows, ctx=ctx, q_heads=group * kv, kv_heads=kv, dim=dim, page=page,
                    cache=rng.choice(["bf16", "e4m3"]))
    if kind == "append":
        lanes = _log(rng, 1, 16)
        rows = _log(rng, 1, max(1, 2048 // lanes))
        return dict(kind=kind, lanes=lanes, rows=rows, ctx=_log(rng, 1, 16384), q_heads=kv * rng.choice([1, 4, 6]), kv_heads=kv, dim=dim,
                    page=page, cache=rng.choice(["bf16", "e4m3"]), axes=rng.choice([1, 2, 3]), pairs=rng.choice([dim // 8, dim // 2]),
                    interleaved=rng.random() < 0.5)
    if kind == "update":
        batch, beams = _log(rng, 1, 8), _log(rng, 1, 8)
        return dict(kind=kind, batch=batch, beams=beams, ctx=_log(rng, 16, 8192), layers=rng.choice([1, 2]), kv_heads=min(kv, 4), dim=min(dim, 128),
                    page=page, reserve=_log(rng, 1, 200))
    if kind == "compact":
        return dict(kind=kind, lanes=_log(rng, 1, 64), rows=_log(rng, 2, 64), ctx=_log(rng, 1, 600), layers=_log(rng, 1, 16),
                    kv_heads=min(kv, 4), dim=dim if dim < 256 else 128, page=page, cache=rng.choice(["bf16", "e4m3"]))
    V = _log(rng, 500, 152064)
    beams = _log(rng, 1, 16)
    return dict(kind=kind, batch=_log(rng, 1, max(1, 128 // beams)), beams=beams, V=V, k=min(2 * beams, 32),
                logits=rng.choice(["f32", "bf16"]))


# ---- what a case's sizes are ---------------------------------------------------

def _rows(c):
    """Rows of each lane: full trees, and shorter ones at the odd lanes."""
    return [c["rows"] - (i * 5) % c["rows"] // 2 if i % 2 else c["rows"] for i in range(c["lanes"])]


def _ctx(c):
    """Context lengths of the lanes: from the longest down to about a quarter of it, odd ones among them."""
    n = c["lanes"]
    return [max(1, c["ctx"] - (3 * c["ctx"] * i) // (4 * n) - i) for i in range(n)]


def _esize(c):
    return 1 if c.get("cache") == "e4m3" else 2


def work(case):
    c = case
    if c["kind"] == "beam":
        rows = c["batch"] * c["beams"]
        n = rows * c["V"]
        return {"bytes": n * (4 if c["logits"] == "f32" else 2) + rows * 5 + c["batch"] * c["k"] * 13, "flops": 4.0 * n}
    kv = c["kv_heads"] * c["dim"]
    if c["kind"] == "attention":
        q = c["q_heads"] * c["dim"]
        rows, ctx = _rows(c), _ctx(c)
        tokens = sum(r + n for r, n in zip(rows, ctx))
        return {"bytes": tokens * 2 * kv * _esize(c) + sum(rows) * (2 * 2 * q + 4 * c["q_heads"] + 8) + 4 * tokens // c["page"],
                "flops": sum(4.0 * r * q * (n + r) for r, n in zip(rows, ctx))}
    if c["kind"] == "append":
        r, q = sum(_rows(c)), c["q_heads"] * c["dim"]
        return {"bytes": r * (2 * (q + 2 * kv) + 2 * q + 2 * kv * _esize(c) + 4 * c["axes"]), "flops": 6.0 * r * 2 * c["pairs"] * (c["q_heads"] + c["kv_heads"])}
    if c["kind"] == "compact":
        moved = sum(_accepted(r, i) for i, r in enumerate(_rows(c)))
        return {"bytes": moved * c["layers"] * 2 * kv * _esize(c) * 2 + 8 * moved, "flops": 0.0}
    lanes, P = c["batch"] * c["beams"], c["page"]
    wide = -(-(c["ctx"] + c["reserve"]) // P) + 1
    copies = sum(1 for i, (p, n) in enumerate(zip(_parents(c), _lens(c))) if p >= 0 and n % P and _parents(c).index(p) != i)
    return {"bytes": copies * c["layers"] * 2 * kv * 2 * P * 2 + 2 * 4 * lanes * wide + 8 * _pool(c), "flops": 0.0}


# ---- inputs --------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g, np.random.default_rng(int(seed) & 0x7FFFFFFF)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _int(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


K_SCALE, V_SCALE = 0.07, 0.055


def _cache(g, c, layers, pages):
    """K and V pages and their scales; an 8-bit cache stands for E4M3 values times its scale."""
    k = _randn(g, layers, pages, c["kv_heads"], c["page"], c["dim"])
    v = _randn(g, layers, pages, c["kv_heads"], c["page"] // 16, c["dim"], 16)
    if c.get("cache") == "e4m3":
        return (k.float() / K_SCALE).to(torch.float8_e4m3fn), (v.float() / V_SCALE).to(torch.float8_e4m3fn), K_SCALE, V_SCALE
    return k, v, 1.0, 1.0


def _tables(r, need):
    """Tables of lanes that need so many pages each, over a pool in random order with a few pages to spare."""
    pages = sum(need) + 3
    order = r.permutation(pages).astype(np.int32)
    table = np.full((len(need), max(need) + 1), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, pages


def _tree(r, n):
    """Mask words of a random tree of n drafted tokens: each sees itself and its ancestors."""
    words, depth = [], []
    for i in range(n):
        p = -1 if i == 0 else int(r.integers(max(0, i - 4), i))
        words.append((words[p] if p >= 0 else 0) | (1 << i))
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return words, depth


def _signed(w):
    return w - (1 << 64) if w >> 63 else w


def _accepted(rows, lane):
    """How many drafts a lane accepts: from one to all, about half."""
    return max(1, rows * (1 + lane % 3) // 3) if rows > 1 else 1


def _parents(c):
    """The parent lane of each beam: within its request, with some chosen twice; every eighth request's last beam ends."""
    n = c["beams"]
    return [-1 if n > 2 and b % 8 == 7 and i == n - 1 else b * n + (i * i + b) % n for b in range(c["batch"]) for i in range(n)]


def _lens(c):
    """What each new lane keeps: its request's length."""
    return [max(1, c["ctx"] - (b * c["ctx"]) // (2 * c["batch"]) - 3 * b) for b in range(c["batch"]) for _ in range(c["beams"])]


def _pool(c):
    lanes, P = c["batch"] * c["beams"], c["page"]
    return lanes * (-(-c["ctx"] // P) + 2 * (-(-c["reserve"] // P)) + 4)


def prepare(case, seed):
    c = dict(case)
    g, r = _gen(seed)
    s = {"c": c}
    kind = c["kind"]
    if kind == "beam":
        rows = c["batch"] * c["beams"]
        x = torch.randn(rows, c["V"], generator=g, device=DEV) * 4.0
        s["logits"] = x if c["logits"] == "f32" else x.to(torch.bfloat16)
        s["score"] = -10.0 * torch.rand(rows, generator=g, device=DEV)
        done = (r.random(rows) < 0.1) & (np.arange(rows) % c["beams"] != 0)
        s["done"] = torch.tensor(done.astype(np.uint8), device=DEV)
        return s
    if kind == "update":
        P, n, lens = c["page"], c["beams"], _lens(c)
        lanes, pages = len(lens), _pool(c)
        order = r.permutation(pages).astype(np.int32)
        table = np.full((lanes, -(-(c["ctx"] + c["reserve"]) // P) + 1), -1, np.int32)
        at = 0
        for i, m in enumerate(lens):  # beams of a request share the first half of their pages
            have, shared = -(-m // P), (m // P) // 2
            if i % n:
                table[i, :shared] = table[i - i % n, :shared]
            else:
                shared = 0
            table[i, shared:have] = order[at:at + have - shared]
            at += have - shared
        refs = np.bincount(table[table >= 0].ravel(), minlength=pages)
        s |= dict(table=_int(table), length=_int(lens), refs=_int(refs), parent=_int(_parents(c)), keep=_int(lens),
                  reserve=_int([c["reserve"]] * lanes))
        s["k"], s["v"], s["ks"], s["vs"] = _cache(g, c, c["layers"], pages)
    else:
        rows, ctx = _rows(c), _ctx(c)
        table, pages = _tables(r, [-(-(m + t) // c["page"]) for m, t in zip(ctx, rows)])
        s["k"], s["v"], s["ks"], s["vs"] = _cache(g, c, c.get("layers", 1), pages)
        s |= dict(table=_int(table), ctx=_int(ctx), most=max(rows))
        starts = np.concatenate([[0], np.cumsum(rows)])
        s["start"] = _int(starts)
        if kind == "compact":
            path = np.zeros((len(rows), max(rows)), np.int32)
            for i, t in enumerate(rows):
                m = _accepted(t, i)
                path[i, :m] = np.sort(r.permutation(t)[:m])
            s |= dict(path=_int(path), accepted=_int([_accepted(t, i) for i, t in enumerate(rows)]))
        else:
            total = int(starts[-1])
            trees = [_tree(r, t) if kind == "attention" else ([], range(t)) for t in rows]
            if kind == "attention":
                s["q"] = 2.0 * _randn(g, total, c["q_heads"] * c["dim"])
                s["mask"] = torch.tensor([_signed(w) for t in trees for w in t[0]], dtype=torch.int64, device=DEV)
            else:
                s["qkv"] = _randn(g, total, (c["q_heads"] + 2 * c["kv_heads"]) * c["dim"])
                at = np.concatenate([m + np.arange(t) for m, t in zip(ctx, rows)])
                pos = np.stack([at] + [r.integers(0, 64, total) for _ in range(c["axes"] - 1)], 1)
                s["pos"] = _int(pos)
                s["inv_freq"] = (1e6 ** (-torch.arange(c["pairs"], device=DEV, dtype=torch.float64) / c["pairs"])).float()
                s["axis"] = torch.tensor(np.arange(c["pairs"]) % c["axes"], dtype=torch.uint8, device=DEV)
                s["factor"] = 1.05
    if own:
        import nvfp4_weight_streaming_amd as nv
        s["cache"] = nv.PagedCache(s["k"], s["v"], s["ks"], s["vs"])
    return s


# ---- one pass --------------------------------------------------------------------

def run(state):
    s, c = state, state["c"]
    kind = c["kind"]
    if not own:
        return _PLAIN[kind](s, c)
    import nvfp4_weight_streaming_amd as nv
    if kind == "attention":
        out, lse = s["cache"].attend(0, s["q"], s["start"], s["ctx"], s["table"], s["mask"], s["most"], c["dim"] ** -0.5, with_lse=True)
        return {"out": out, "lse": lse}
    if kind == "append":
        q = s["cache"].append(0, s["qkv"], c["q_heads"], s["start"], s["ctx"], s["table"], s["pos"], s["inv_freq"],
                              pair_axis=s["axis"], interleaved=c["interleaved"], factor=s["factor"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    if kind == "update":
        table, length, refs, short = s["cache"].update(s["table"], s["length"], s["refs"], s["parent"], s["keep"], s["reserve"])
        return {"table": table, "length": length, "refs": refs, "short": short, "k": s["k"], "v": s["v"]}
    if kind == "compact":
        s["cache"].compact(s["ctx"], s["table"], s["path"], s["accepted"])
        return {"k": s["k"], "v": s["v"]}
    score, parent, token, done = nv.beam_select(s["logits"], c["beams"], s["score"], c["k"], done=s["done"], eos=2)
    return {"score": score, "parent": parent, "token": token, "done": done}


# ---- plain forms -------------------------------------------------------------------

def _lane_of_rows(s, total):
    return torch.searchsorted(s["start"][1:].contiguous(), torch.arange(total, device=DEV, dtype=torch.int32), right=True)


def _plain_attention(s, c):
    lanes, G, Hk, D, P = c["lanes"], c["q_heads"] // c["kv_heads"], c["kv_heads"], c["dim"], c["page"]
    total, T = s["q"].shape[0], s["most"]
    table = s["table"].clamp(min=0).long()
    n = table.shape[1] * P
    k = s["k"][0].view(torch.uint8)[table].view(s["k"].dtype).float() * s["ks"]  # [lanes, pages, heads, P, D]
    v = s["v"][0].view(torch.uint8)[table].view(s["v"].dtype).float() * s["vs"]  # [lanes, pages, heads, P / 16, D, 16]
    k = k.permute(0, 2, 1, 3, 4).reshape(lanes, Hk, n, D)
    v = v.permute(0, 2, 1, 3, 5, 4).reshape(lanes, Hk, n, D)
    t = torch.arange(T, device=DEV)
    row = s["start"][:-1, None].long() + t  # [lanes, T]
    real = row < s["start"][1:, None]
    row = row.clamp(max=total - 1)
    q = s["q"][row].float().view(lanes, T, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(lanes, Hk, T * G, D)
    at = torch.arange(n, device=DEV) - s["ctx"][:, None]  # place among the drafted tokens
    bits = (s["mask"][row][:, :, None] >> at.clamp(0, 63)[:, None, :]) & 1
    seen = (at < 0)[:, None, :] | ((bits == 1) & (at < 64)[:, None, :] & (at < (s["start"][1:] - s["start"][:-1])[:, None])[:, None, :])
    seen = seen[:, None, :, None, :].expand(lanes, 1, T, G, n).reshape(lanes, 1, T * G, n)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).masked_fill_(~seen, NEG)
    m = x.amax(3, keepdim=True)
    x = x.sub_(torch.where(m == NEG, 0.0, m)).exp_()
    z = x.sum(3, keepdim=True)
    v = v.masked_fill((at >= (s["start"][1:] - s["start"][:-1])[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(x, v) / torch.where(z == 0, 1.0, z)
    lse = (m + z.log()).view(lanes, Hk, T, G).permute(0, 2, 1, 3).reshape(lanes * T, Hk * G)
    o = o.view(lanes, Hk, T, G, D).permute(0, 2, 1, 3, 4).reshape(lanes * T, Hk * G * D)
    keep = _rows_at(s, real, total)
    return {"out": o[keep].to(torch.bfloat16), "lse": lse[keep]}


def _rows_at(s, real, total):
    """Where each row stands in a [lanes, T] layout."""
    lane = _lane_of_rows(s, total)
    return lane * real.shape[1] + torch.arange(total, device=DEV) - s["start"][lane]


def _store(cache, at, value):
    """cache[at] = value by the cache's bytes (8-bit types have no indexed store)."""
    b = cache.view(torch.uint8) if cache.element_size() == 1 else cache
    v = value.clamp(-448, 448).to(cache.dtype).view(torch.uint8) if cache.element_size() == 1 else value.to(cache.dtype)
    b[at] = v


def _plain_append(s, c):
    Hq, Hk, D, P, n = c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["pairs"]
    total = s["qkv"].shape[0]
    x = s["qkv"].float().view(total, Hq + 2 * Hk, D)
    a = s["pos"].float()[:, s["axis"].long()] * s["inv_freq"]
    cos, sin = (a.cos() * s["factor"])[:, None], (a.sin() * s["factor"])[:, None]
    h = x[:, :Hq + Hk]
    if c["interleaved"]:
        u, w = h[..., 0:2 * n:2], h[..., 1:2 * n:2]
        turned = torch.stack([u * cos - w * sin, u * sin + w * cos], -1).flatten(-2)
    else:
        u, w = h[..., :n], h[..., n:2 * n]
        turned = torch.cat([u * cos - w * sin, u * sin + w * cos], -1)
    h = torch.cat([turned, h[..., 2 * n:]], -1)
    lane = _lane_of_rows(s, total)
    at = s["ctx"][lane] + torch.arange(total, device=DEV) - s["start"][lane]
    page, off = s["table"][lane, at // P].long()[:, None], (at % P)[:, None].long()
    head = torch.arange(Hk, device=DEV)[None]
    _store(s["k"][0], (page, head, off), h[:, Hq:] / s["ks"])
    _store(s["v"][0], (page, head, off // 16, slice(None), off % 16), x[:, Hq + Hk:] / s["vs"])
    return {"q": h[:, :Hq].to(torch.bfloat16).reshape(total, Hq * D), "k": s["k"], "v": s["v"]}


def _count(t, pages):
    """How often each page is named."""
    t = torch.where((t < 0) | (t >= pages), pages, t).flatten().long()
    return torch.zeros(pages + 1, dtype=torch.int32, device=DEV).scatter_add_(0, t, torch.ones_like(t, dtype=torch.int32))


def _plain_update(s, c):
    P, pages = c["page"], s["refs"].numel()
    old, wide = s["table"], s["table"].shape[1]
    has = (s["parent"] >= 0) & (s["parent"] < old.shape[0])
    par = torch.where(has, s["parent"], 0).long()
    length = torch.where(has, torch.minimum(s["keep"].clamp(min=0), s["length"][par]), 0)
    held = (length + P - 1) // P
    upto = ((length + s["reserve"].clamp(min=0) + P - 1) // P).clamp(max=wide)
    col = torch.arange(wide, device=DEV)
    table = torch.where(col < held[:, None], old[par], -1)
    refs = torch.cat([s["refs"], s["refs"].new_zeros(1)]) - _count(old, pages) + _count(table, pages)
    last = table.gather(1, (held - 1).clamp(min=0).long()[:, None])[:, 0]
    part = (length % P != 0) & (last >= 0)
    q = torch.where(part, last, pages).long()
    lane = torch.arange(len(par), device=DEV)
    alone = _count(torch.where(part, last, -1), pages)
    first = torch.full((pages + 1,), len(par), device=DEV).scatter_reduce_(0, q, lane, "amin")
    copy = part & ~((alone[q] == refs[q]) & (first[q] == lane))
    need = ((col >= held[:, None]) & (col < upto[:, None])) | (copy[:, None] & (col == held[:, None] - 1))
    rank = (need.flatten().cumsum(0) - 1).view_as(need)
    free = refs[:pages] == 0
    order = torch.sort((~free).to(torch.int32), stable=True).indices
    fresh = torch.where(rank < free.sum(), order[rank.clamp(0, pages - 1)], -1)
    table = torch.where(need, fresh, table).to(torch.int32)
    refs = refs - _count(torch.where(copy, last, -1), pages) + _count(torch.where(need, table, -1), pages)
    short = (need.sum() - free.sum()).clamp(min=0).to(torch.int32).view(1)
    to = table.gather(1, (held - 1).clamp(min=0).long()[:, None])[:, 0].long()
    does = copy & (to >= 0)
    pick = torch.where(does, lane, 0).cummax(0).values  # lanes with no copy repeat one that has
    any_ = does.any()
    pick = torch.where(does[pick], pick, does.to(torch.int32).argmax())
    src, dst = torch.where(any_, q[pick], 0).clamp(max=pages - 1), torch.where(any_, to[pick], 0)
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    return {"table": table, "length": length.to(torch.int32), "refs": refs[:pages], "short": short, "k": s["k"], "v": s["v"]}


def _plain_compact(s, c):
    P, width = c["page"], s["path"].shape[1]
    j = torch.arange(width, device=DEV)
    real = j < s["accepted"][:, None]
    src = s["ctx"][:, None] + torch.where(real, s["path"], 0)
    dst = torch.where(real, s["ctx"][:, None] + j, src)
    # entries past the accepted ones repeat the lane's first move
    dst = torch.where(real, dst, s["ctx"][:, None])
    src = torch.where(real, src, src[:, :1])
    a, b = s["table"].gather(1, (src // P).long()).long(), s["table"].gather(1, (dst // P).long()).long()
    k, v = (t.view(torch.uint8) if t.element_size() == 1 else t for t in (s["k"], s["v"]))
    so, do = (src % P).long(), (dst % P).long()
    kk, vv = k[:, a, :, so], v[:, a, :, so // 16, :, so % 16]
    k[:, b, :, do] = kk
    v[:, b, :, do // 16, :, do % 16] = vv
    return {"k": s["k"], "v": s["v"]}


def _order(x):
    """Whole numbers in the order of the values of x, which are not NaN; both zeros are equal."""
    b = (x + 0.0).view(torch.int32).long()
    return torch.where(b < 0, -(b & 0x7FFFFFFF), b)


def _plain_beam(s, c):
    rows, V, k, n = s["score"].numel(), c["V"], c["k"], c["beams"]
    token = torch.arange(V, device=DEV)
    x = s["logits"].float()
    end = s["done"].bool()[:, None]
    x = torch.where(end, torch.where(token == 2, 0.0, NEG), x)
    x = torch.where((s["score"] == NEG)[:, None], NEG, x)
    m = x.amax(1, keepdim=True)
    m = torch.where(m == NEG, 0.0, m)
    z = (x - m).exp().sum(1, keepdim=True).log()
    score = torch.where(x == NEG, NEG, s["score"][:, None] + ((x - m) - z)).view(c["batch"], n * V)
    at = torch.arange(n * V, device=DEV)
    pick = torch.topk((_order(score) << 32) + (n * V - 1 - at), k, 1).indices  # equal scores: by row, then token
    parent = (pick // V + torch.arange(c["batch"], device=DEV)[:, None] * n).to(torch.int32)
    token = (pick % V).to(torch.int32)
    done = (s["done"][parent.long()].bool() | (token == 2)).to(torch.uint8)
    return {"score": score.gather(1, pick), "parent": parent, "token": token, "done": done}


_PLAIN = {"attention": _plain_attention, "append": _plain_append, "update": _plain_update, "compact": _plain_compact,
          "beam": _plain_beam}


# ---- from the definitions, in 64 bits ------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c, kind = s["c"], case["kind"]
    f64 = torch.float64
    if kind == "beam":
        out = []
        score, x, done = s["score"].to(f64), s["logits"].to(f64), s["done"].cpu().tolist()
        x = torch.log_softmax(x, 1) + score[:, None]
        for r, d in enumerate(done):
            if d:
                x[r] = NEG
                x[r, 2] = score[r]
        for b in range(c["batch"]):
            out.append(torch.sort(x[b * c["beams"]:(b + 1) * c["beams"]].flatten(), descending=True).values[:c["k"]])
        return {"score": torch.stack(out), "parent": None, "token": None, "done": None}
    table = s["table"].cpu().tolist()
    P = c["page"]
    if kind == "update":
        refs, lens = s["refs"].cpu().tolist(), s["length"].cpu().tolist()
        parents, keep, reserve = (s[n].cpu().tolist() for n in ("parent", "keep", "reserve"))
        for row in table:
            for p in row:
                if p >= 0:
                    refs[p] -= 1
        new, length = [], []
        for p, n in zip(parents, keep):
            n = min(n, lens[p]) if p >= 0 else 0
            new.append(table[p][:-(-n // P)] if n else [])
            length.append(n)
            for e in new[-1]:
                refs[e] += 1
        part = [row[-1] if n % P else None for row, n in zip(new, length)]
        free = [i for i, n in enumerate(refs) if n == 0]
        for i, (row, n) in enumerate(zip(new, length)):
            q = part[i]
            if q is not None and not (part.count(q) == refs[q] and part.index(q) == i):
                row[-1] = free.pop(0)
                for t in (s["k"], s["v"]):
                    t[:, row[-1]] = t[:, q]
            for _ in range(-(-(n + reserve[i]) // P) - -(-n // P)):
                free.pop(0)
        return {"table": None, "length": None, "refs": None, "short": None, "k": s["k"], "v": s["v"]}
    ctx = s["ctx"].cpu().tolist()
    if kind == "compact":
        k, v = s["k"].float(), s["v"].float()
        path, accepted = s["path"].cpu().tolist(), s["accepted"].cpu().tolist()
        for i, n in enumerate(accepted):
            for j in range(n):  # ascending, and path[j] >= j: a source is read before it is written
                a, b = ctx[i] + path[i][j], ctx[i] + j
                k[:, table[i][b // P], :, b % P] = k[:, table[i][a // P], :, a % P].clone()
                to, of = b % P, a % P
                v[:, table[i][b // P], :, to // 16, :, to % 16] = v[:, table[i][a // P], :, of // 16, :, of % 16].clone()
        return {"k": k.to(s["k"].dtype), "v": v.to(s["v"].dtype)}
    start = s["start"].cpu().tolist()
    Hk, D = c["kv_heads"], c["dim"]
    if kind == "append":
        n, Hq = c["pairs"], c["q_heads"]
        x = s["qkv"].to(f64).view(-1, Hq + 2 * Hk, D)
        turn = s["pos"].to(f64)[:, s["axis"].long()] * s["inv_freq"].to(f64)
        z = torch.polar(torch.full_like(turn, s["factor"]), turn)[:, None]
        h = x[:, :Hq + Hk].clone()
        i = torch.arange(n, device=DEV)
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + n)
        w = torch.complex(h[..., a], h[..., b]) * z
        h[..., a], h[..., b] = w.real, w.imag
        if D * Hk * s["k"].shape[1] * P > 50_000_000:
            return None
        k, v = s["k"].to(f64), s["v"].to(f64)
        for i in range(c["lanes"]):
            for t in range(start[i + 1] - start[i]):
                r, at = start[i] + t, ctx[i] + t
                k[0, table[i][at // P], :, at % P] = h[r, Hq:] / s["ks"]
                v[0, table[i][at // P], :, at % P // 16, :, at % 16] = x[r, Hq + Hk:] / s["vs"]
        return {"q": h[:, :Hq].reshape(-1, Hq * D), "k": k, "v": v}
    G = c["q_heads"] // Hk
    outs, lses = [], []
    for i in range(c["lanes"]):
        t = start[i + 1] - start[i]
        n = ctx[i] + t
        pages = torch.tensor(table[i][:-(-n // P)], device=DEV)
        k = (s["k"][0].view(torch.uint8)[pages].view(s["k"].dtype).to(f64) * s["ks"]).transpose(1, 2).reshape(-1, Hk, D)[:n]
        v = (s["v"][0].view(torch.uint8)[pages].view(s["v"].dtype).to(f64) * s["vs"]).permute(0, 2, 4, 1, 3).reshape(-1, Hk, D)[:n]
        q = s["q"][start[i]:start[i + 1]].to(f64).view(t, Hk, G, D)
        words = s["mask"][start[i]:start[i + 1]].cpu().tolist()
        seen = torch.ones(t, n, dtype=torch.bool)
        for a, w in enumerate(words):
            for b in range(t):
                seen[a, ctx[i] + b] = bool((w >> b) & 1)
        o, z = [], []
        for h in range(Hk):
            x = (q[:, h].reshape(t * G, D) @ k[:, h].T.contiguous()) * D ** -0.5
            x = x.masked_fill(~seen.to(DEV).repeat_interleave(G, 0), NEG)
            z.append(torch.logsumexp(x, 1).view(t, G))
            o.append((torch.softmax(x, 1) @ v[:, h].contiguous()).view(t, G, D))
        outs.append(torch.stack(o, 1).reshape(t, -1))
        lses.append(torch.stack(z, 1).reshape(t, -1))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
