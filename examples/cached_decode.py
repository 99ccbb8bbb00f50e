"""Decoding with the paged cache: drafted trees and beam search on a small synthetic model.

A two-layer transformer with random NVFP4 weights runs on the library's products, SwiGLU,
cache append, tree attention, page-table update, compaction, top-k and beam selection; torch
does what is left (embedding, norms, residual sums).

    python examples/cached_decode.py

* ``speculate``: each round sends a tree of drafts per lane through the model in one pass,
  accepts the longest branch that the model itself would have taken, moves its keys and values to
  the front and goes on.  (The drafter is a stand-in: it knows a plain decode's answer and gets
  some of it wrong.)
* ``beam_search``: selection, reordering of the tables with copies of shared pages, and a step.

Both are checked by running the finished sequences through fresh pages in one pass.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import nvfp4_weight_streaming_amd as nv  # noqa: E402

LAYERS, HIDDEN, Q_HEADS, KV_HEADS, DIM, FFN, VOCAB = 2, 512, 8, 2, 64, 1024, 2000
PAGE, PAGES, WIDTH = 16, 256, 12  # tokens per page, pages of the pool, pages of a lane at most


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    def __init__(self, seed=0, cache_dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def matrix(n, k, std, out):
            w = nv.PackedWeight.quantize(std * torch.randn((n, k), generator=g, device="cuda"))
            return w, nv.Gemm(256, k, n, out)

        self.embed = torch.randn((VOCAB, HIDDEN), generator=g, device="cuda").to(torch.bfloat16)
        self.layers = [dict(qkv=matrix((Q_HEADS + 2 * KV_HEADS) * DIM, HIDDEN, 0.04, nv.OUT_BF16),
                            o=matrix(HIDDEN, Q_HEADS * DIM, 0.04, nv.OUT_BF16),
                            gate_up=matrix(2 * FFN, HIDDEN, 0.04, nv.OUT_BF16),
                            down=matrix(HIDDEN, FFN, 0.04, nv.OUT_BF16)) for _ in range(LAYERS)]
        self.head = matrix(VOCAB, HIDDEN, 0.12, nv.OUT_F32)
        self.inv_freq = (1e4 ** (-torch.arange(DIM // 2, device="cuda") / (DIM // 2))).float()
        k = torch.zeros((LAYERS, PAGES, KV_HEADS, PAGE, DIM), device="cuda").to(cache_dtype)
        v = torch.zeros((LAYERS, PAGES, KV_HEADS, PAGE // 16, DIM, 16), device="cuda").to(cache_dtype)
        scale = 0.02 if cache_dtype == torch.float8_e4m3fn else 1.0
        self.cache = nv.PagedCache(k, v, scale, scale)

    def _product(self, name, layer, x):
        w, gemm = layer[name] if layer else self.head
        out = torch.empty((x.shape[0], w.N), dtype=torch.float32 if name == "head" else torch.bfloat16, device="cuda")
        return gemm(w, x.contiguous(), out)

    @staticmethod
    def _norm(x):
        return (x * torch.rsqrt(x.pow(2).mean(1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def step(self, tokens, start, ctx, table, positions, mask, most):
        """fp32 logits of rows of drafted tokens over their lanes' contexts."""
        x = self.embed[tokens.long()].float()
        for i, layer in enumerate(self.layers):
            qkv = self._product("qkv", layer, self._norm(x))
            q = self.cache.append(i, qkv, Q_HEADS, start, ctx, table, positions, self.inv_freq)
            a = self.cache.attend(i, q, start, ctx, table, mask, most, DIM ** -0.5)
            x = x + self._product("o", layer, a).float()
            gate_up = self._product("gate_up", layer, self._norm(x))
            h = torch.empty((x.shape[0], FFN), dtype=torch.bfloat16, device="cuda")
            nv.nvfp4_swiglu(gate_up, x.shape[0], FFN, h)
            x = x + self._product("down", layer, h).float()
        return self._product("head", None, self._norm(x))


class Lanes:
    """Lanes of a model's cache: tables, lengths and page counts on the device."""

    def __init__(self, model, n):
        self.cache = model.cache
        self.table = torch.full((n, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.length = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")

    def update(self, parent, keep, room):
        n = parent.numel()
        self.table, self.length, self.refs, short = self.cache.update(
            self.table, self.length, self.refs, parent, keep, _i32([room] * n))
        assert int(short) == 0, "out of pages"


def run_trees(model, lanes, trees):
    """One pass over a tree of (tokens, parents) per lane; logits and each lane's first row."""
    rows = [len(t) for t, _ in trees]
    start = [0]
    for n in rows:
        start.append(start[-1] + n)
    words, depths = zip(*(nv.nvfp4_tree_mask(p) for _, p in trees))
    tokens = _i32([t for ts, _ in trees for t in ts])
    mask = torch.tensor([w for m in words for w in m], dtype=torch.int64, device="cuda")
    base = lanes.length.tolist()
    positions = _i32([[base[i] + d] for i, ds in enumerate(depths) for d in ds])
    logits = model.step(tokens, _i32(start), lanes.length, lanes.table, positions, mask, max(rows))
    return logits, start


def chain(n):
    return list(range(-1, n - 1))


def prefill(model, prompts, room):
    """Lanes that hold all but the last token of their prompts."""
    lanes = Lanes(model, len(prompts))
    lanes.update(_i32([-1] * len(prompts)), None, max(len(p) for p in prompts) + room)
    run_trees(model, lanes, [(p[:-1], chain(len(p) - 1)) for p in prompts])
    lanes.length = _i32([len(p) - 1 for p in prompts])
    return lanes


def greedy(model, prompts, count):
    """Plain decoding: the reference for the drafter."""
    lanes = prefill(model, prompts, count)
    out = [list(p) for p in prompts]
    for _ in range(count):
        logits, _ = run_trees(model, lanes, [([s[-1]], [-1]) for s in out])
        best, _ = nv.topk(logits, 1)
        lanes.length = lanes.length + 1
        for s, t in zip(out, best[:, 0].tolist()):
            s.append(t)
    return out


def speculate(model, prompts, count, answer, seed=1):
    """Sequences of at least `count` new tokens from rounds of drafted trees; rounds taken; lanes."""
    g = torch.Generator().manual_seed(seed)
    lanes = prefill(model, prompts, 0)
    out, rounds = [list(p) for p in prompts], 0
    while min(len(s) - len(p) for s, p in zip(out, prompts)) < count:
        rounds += 1
        trees = []
        for s, a in zip(out, answer):
            # the last token, then two branches of three drafts: one guesses right for a while
            right = (a[len(s):] + [0, 0, 0])[:3]
            right[int(torch.randint(0, 4, (1,), generator=g)) % 3] += int(torch.randint(0, 2, (1,), generator=g))
            wrong = [(t + 7) % VOCAB for t in right]
            trees.append(([s[-1]] + wrong[:1] + [t % VOCAB for t in right] + wrong[1:], [-1, 0, 0, 2, 3, 1, 5]))
        lanes.update(torch.arange(len(out), dtype=torch.int32, device="cuda"), None, len(trees[0][0]))
        logits, start = run_trees(model, lanes, trees)
        best = nv.topk(logits, 1)[0][:, 0].tolist()
        paths = []
        for i, (tokens, parents) in enumerate(trees):
            path, at = [0], 0
            while True:  # follow the branch that says what the model says
                nxt = [j for j, p in enumerate(parents) if p == at and tokens[j] == best[start[i] + at]]
                if not nxt:
                    break
                at = nxt[0]
                path.append(at)
            paths.append(path)
            out[i] += [tokens[j] for j in path[1:]] + [best[start[i] + at]]
        accepted = [len(p) for p in paths]
        wide = max(accepted)
        model.cache.compact(lanes.length, lanes.table, _i32([p + [0] * (wide - len(p)) for p in paths]), _i32(accepted))
        lanes.length = lanes.length + _i32(accepted)
    return out, rounds, lanes


def beam_search(model, prompt, beams, steps):
    """The best sequences and their scores after some steps of beam search."""
    lanes = prefill(model, [prompt] * beams, 0)
    # one prompt: all beams continue the first lane's pages
    lanes.update(_i32([0] * beams), None, 1)
    seqs = [list(prompt) for _ in range(beams)]
    score = torch.tensor([0.0] + [float("-inf")] * (beams - 1), device="cuda")
    for _ in range(steps):
        logits, _ = run_trees(model, lanes, [([s[-1]], [-1]) for s in seqs])
        lanes.length = lanes.length + 1
        score, parent, token, _ = nv.beam_select(logits, beams, score, beams)
        score, parent = score.flatten(), parent.flatten()
        seqs = [seqs[p] + [t] for p, t in zip(parent.tolist(), token.flatten().tolist())]
        lanes.update(parent, None, 1)
    return seqs, score.tolist(), lanes


def rescore(model, seqs):
    """fp32 logits of every position of each sequence, in one pass over fresh pages; the lanes."""
    lanes = Lanes(model, len(seqs))
    lanes.update(_i32([-1] * len(seqs)), None, max(len(s) for s in seqs))
    logits, start = run_trees(model, lanes, [(s[:-1], chain(len(s) - 1)) for s in seqs])
    lanes.length = _i32([len(s) - 1 for s in seqs])
    return [logits[start[i]:start[i + 1]] for i in range(len(seqs))], lanes


def cached(model, lanes, lane, n):
    """K and V of a lane's first n tokens, [layers, n, heads, dim] each."""
    c = model.cache
    k = torch.stack([c.k[:, lanes.table[lane, t // PAGE], :, t % PAGE].float() for t in range(n)], 1)
    v = torch.stack([c.v[:, lanes.table[lane, t // PAGE], :, t % PAGE // 16, :, t % 16].float() for t in range(n)], 1)
    return k, v


def main():
    model = Model()
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, VOCAB, (n,), generator=g).tolist() for n in (9, 21)]
    count = 20
    answer = greedy(model, prompts, count + 8)
    out, rounds, lanes = speculate(model, prompts, count, answer)
    tokens = sum(len(s) - len(p) for s, p in zip(out, prompts))
    held = [cached(model, lanes, i, len(s) - 1) for i, s in enumerate(out)]
    # what the products' two kernels round differently moves logits by about 1 in 100
    worst = moved = 0.0
    logits, fresh = rescore(model, out)
    for i, (s, p) in enumerate(zip(out, prompts)):
        new = logits[i][len(p) - 1:]
        chosen = new.gather(1, torch.tensor(s[len(p):], device="cuda")[:, None])[:, 0]
        worst = max(worst, float(((new.max(1).values - chosen) / new.std(1)).max()))
        for a, b in zip(held[i], cached(model, fresh, i, len(s) - 1)):
            moved = max(moved, float((a - b).norm() / b.norm()))
    print("drafted trees: %d tokens of %d lanes in %d rounds; furthest from the best logit %.3f deviations; cache within %.4f" % (
        tokens, len(out), rounds, worst, moved))
    seqs, scores, _ = beam_search(model, prompts[0], 4, 12)
    logits, _ = rescore(model, seqs)
    off = 0.0
    for s, c, x in zip(seqs, scores, logits):
        p = torch.log_softmax(x.double(), 1)[len(prompts[0]) - 1:]
        off = max(off, abs(float(p.gather(1, torch.tensor(s[len(prompts[0]):], device="cuda")[:, None]).sum()) - c))
    print("beam search: best score %.3f of %d beams; scores within %.3f of the sequences' own" % (scores[0], len(seqs), off))
    return dict(tokens=tokens, rounds=rounds, worst=worst, moved=moved, off=off, scores=scores, seqs=seqs)


if __name__ == "__main__":
    main()
