"""Cases of the operators around 8-bit matrices and the answer's probabilities, which a decode round needs beside its NVFP4 products.

* ``norm``: root-mean-square norm of x, or of x plus the residual stream, which is written back; in bf16 or fp32, or in 8 bits
  with one scale a row;
* ``quantise``: rows to 8 bits with one scale each, of x itself or of silu(gate) * up;
* ``gemm``: the product of 8-bit rows and 8-bit weights, with a scale for each row and each output channel;
* ``logprobs``: log probabilities of given tokens, the entropy, and the best tokens with theirs.

``run`` with ``own`` false computes them with elementary torch operations; with ``own`` true it makes the calls of
``nvfp4_weight_streaming_amd``.  ``exact`` computes them from their definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
NEG = float("-inf")
EPS = 1e-6


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # Between two projections of a decode round of 8 lanes: the smallest call, where latency counts.
        dict(name="norm 8 x 5120", kind="norm", rows=8, K=5120, x="bf16", residual="bf16", out="bf16"),
        # The same step of a prefill chunk.
        dict(name="norm 2048 x 5120", kind="norm", rows=2048, K=5120, x="bf16", residual="bf16", out="bf16"),
        # A verify round's rows (8 lanes x 8) in front of an 8-bit matrix, with a residual stream of 32 bits.
        dict(name="norm 64 x 5120, 8-bit", kind="norm", rows=64, K=5120, x="bf16", residual="f32", out="int8"),
        # In front of an 8-bit down matrix: decode.
        dict(name="swiglu 8 x 17408, 8-bit", kind="quantise", rows=8, K=17408, x="bf16", swiglu=True),
        # And a prefill chunk.
        dict(name="swiglu 2048 x 17408, 8-bit", kind="quantise", rows=2048, K=17408, x="bf16", swiglu=True),
        # An 8-bit qkv matrix in a decode round, with a bias.
        dict(name="gemm 8 x 5120 x 7168", kind="gemm", rows=8, K=5120, N=7168, out="bf16", bias=True),
        # An 8-bit down matrix in the widest verify round.
        dict(name="gemm 64 x 17408 x 5120", kind="gemm", rows=64, K=17408, N=5120, out="bf16", bias=False),
        # The output head, which recipes with 4-bit bodies keep in 8 bits.
        dict(name="head 8 x 5120 x 152064", kind="gemm", rows=8, K=5120, N=152064, out="f32", bias=False),
        # An 8-bit gate_up matrix over a prefill chunk: bound by arithmetic.
        dict(name="gemm 2048 x 5120 x 34816", kind="gemm", rows=2048, K=5120, N=34816, out="bf16", bias=False),
        # What a server answers a decode round of 8 lanes with: the taken token and 20 alternatives.
        dict(name="logprobs 8 x 152064", kind="logprobs", rows=8, V=152064, logits="f32", tokens=1, k=20, scale=1.0),
        # A verify round: each row's drafted tokens at a temperature; a vocabulary of odd size, so no row but the first is aligned.
        dict(name="logprobs 64 x 99991, bf16", kind="logprobs", rows=64, V=99991, logits="bf16", tokens=7, k=0, scale=1.25),
        # Scoring a prompt's chunk.
        dict(name="logprobs 1024 x 152064, bf16", kind="logprobs", rows=1024, V=152064, logits="bf16", tokens=1, k=8, scale=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "quantise", "gemm", "gemm", "gemm", "logprobs", "logprobs"])
    if kind in ("norm", "quantise"):
        K = _log(rng, 16, 17408)
        K = K if rng.random() < 0.3 else -(-K // 16) * 16
        rows = _log(rng, 1, min(4096, 2048 * 17408 // K))
        x = rng.choice(["bf16", "bf16", "f32"])
        if kind == "norm":
            return dict(kind=kind, rows=rows, K=K, x=x, residual=rng.choice(["none", "bf16", "f32"]), out=rng.choice(["bf16", "int8", "f32"]))
        return dict(kind=kind, rows=rows, K=K, x=x, swiglu=x == "bf16" and rng.random() < 0.6)
    if kind == "gemm":
        while True:
            rows, K, N = _log(rng, 1, 2048), 16 * _log(rng, 4, 1088), _log(rng, 16, 152064)
            N = N if rng.random() < 0.3 else -(-N // 16) * 16
            if K * N <= 5120 * 152064 and rows * K * N <= 2048 * 5120 * 17408:
                return dict(kind=kind, rows=rows, K=K, N=N, out=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5)
    V = _log(rng, 100, 152064)
    return dict(kind=kind, rows=_log(rng, 1, min(1024, 152064 * 512 // V)), V=V, logits=rng.choice(["f32", "bf16"]),
                tokens=_log(rng, 1, 8), k=rng.choice([0, 1, 5, 20, _log(rng, 1, 64)]), scale=rng.choice([1.0, 0.7, 1.25]))


_BYTES = {"none": 0, "bf16": 2, "f32": 4, "int8": 1}


def work(case):
    c = case
    rows = c["rows"]
    if c["kind"] == "norm":
        n = rows * c["K"]
        return {"bytes": n * (_BYTES[c["x"]] + 2 * _BYTES[c["residual"]] + _BYTES[c["out"]]) + 2 * c["K"] + (4 * rows if c["out"] == "int8" else 0),
                "flops": 6.0 * n}
    if c["kind"] == "quantise":
        n = rows * c["K"]
        return {"bytes": n * (_BYTES[c["x"]] * (2 if c["swiglu"] else 1) + 1) + 4 * rows, "flops": (8.0 if c["swiglu"] else 3.0) * n}
    if c["kind"] == "gemm":
        K, N = c["K"], c["N"]
        return {"bytes": rows * K + N * K + 4 * rows + 4 * N + (4 * N if c["bias"] else 0) + rows * N * _BYTES[c["out"]], "flops": 2.0 * rows * K * N}
    return {"bytes": rows * (c["V"] * _BYTES[c["logits"]] + 8 * c["tokens"] + 4 + 8 * c["k"]), "flops": 6.0 * rows * c["V"]}


# ---- inputs --------------------------------------------------------------------

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8}


def _codes(g, *shape):
    """Codes as rows of normal draws quantise to: a largest value of 127, most of them below 100."""
    x = torch.empty(shape, dtype=torch.int8, device=DEV)
    step = max(1, (1 << 26) // shape[1])
    for i in range(0, shape[0], step):
        n = min(step, shape[0] - i)
        x[i:i + n] = (torch.randn(n, shape[1], generator=g, device=DEV) * 30).round_().clamp_(-127, 127).to(torch.int8)
    x[:, 0] = 127
    return x


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    s = {"c": c}
    rows = c["rows"]
    if c["kind"] == "norm":
        K = c["K"]
        s["x"] = (0.5 * torch.randn(rows, K, generator=g, device=DEV)).to(_TYPES[c["x"]])
        s["weight"] = (1.0 + 0.2 * torch.randn(K, generator=g, device=DEV)).to(torch.bfloat16)
        s["residual"] = None
        if c["residual"] != "none":  # a stream with a few channels that stand out
            r = 2.0 * torch.randn(rows, K, generator=g, device=DEV)
            r[:, torch.randint(0, K, (4,), generator=g, device=DEV)] *= 12.0
            s["residual"] = r.to(_TYPES[c["residual"]])
    elif c["kind"] == "quantise":
        s["x"] = torch.randn(rows, c["K"] * (2 if c["swiglu"] else 1), generator=g, device=DEV).to(_TYPES[c["x"]])
    elif c["kind"] == "gemm":
        K, N = c["K"], c["N"]
        s["a"], s["w"] = _codes(g, rows, K), _codes(g, N, K)
        s["a_scale"] = 0.02 + 0.02 * torch.rand(rows, generator=g, device=DEV)
        s["w_scale"] = (0.5 + torch.rand(N, generator=g, device=DEV)) / (30.0 * math.sqrt(K))
        s["bias"] = torch.randn(N, generator=g, device=DEV) if c["bias"] else None
        if own:
            import nvfp4_weight_streaming_amd as nv
            s["weight"] = nv.Int8Weight.from_canonical(s["w"], s["w_scale"])
            del s["w"]
    else:
        V = c["V"]
        x = torch.randn(rows, V, generator=g, device=DEV, dtype=torch.float32) * 3.0
        x[torch.arange(rows, device=DEV), torch.randint(0, V, (rows,), generator=g, device=DEV)] += 9.0
        x[3::8, : V // 3] = NEG  # rows of constrained decoding
        s["logits"] = x.to(_TYPES[c["logits"]])
        s["tokens"] = torch.randint(0, V, (rows, c["tokens"]), generator=g, device=DEV).to(torch.int32)
        s["tokens"][:, 0] = torch.where(torch.rand(rows, generator=g, device=DEV) < 0.8, x.argmax(1).to(torch.int32), s["tokens"][:, 0])
    return s


# ---- one pass --------------------------------------------------------------------

def run(state):
    s, c = state, state["c"]
    kind = c["kind"]
    if not own:
        return _PLAIN[kind](s, c)
    import nvfp4_weight_streaming_amd as nv
    if kind == "norm":
        got = nv.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], dtype=_TYPES[c["out"]])
        got = list(got) if isinstance(got, tuple) else [got]
        if c["out"] == "int8":
            got[:2] = [got[0] * got[1][:, None], got[1]]  # the values that the codes stand for
        return got
    if kind == "quantise":
        q, scale = nv.int8_quantize(s["x"], swiglu=c["swiglu"])
        return [q * scale[:, None], scale]
    if kind == "gemm":
        return nv.int8_gemm(s["a"], s["a_scale"], s["weight"], dtype=_TYPES[c["out"]], bias=s["bias"])
    logprob, entropy, token, top = nv.logprobs(s["logits"], s["tokens"], k=c["k"], scale=c["scale"])
    return {"logprob": logprob, "entropy": entropy, "token": token, "top": top} if c["k"] else {"logprob": logprob, "entropy": entropy}


# ---- plain forms -------------------------------------------------------------------

def _to_codes(y):
    """[the values that y's codes stand for, scale]: in 64 bits, as a value next to a border takes one code or the other."""
    scale = (y.abs().amax(1) / 127.0).float()
    q = torch.round(y / scale.double()[:, None]).to(torch.int8)
    return [q * scale[:, None], scale]


def _plain_norm(s, c):
    wide = torch.float64 if c["out"] == "int8" else torch.float32
    h, more = s["x"].float(), []
    if s["residual"] is not None:
        h = (h + s["residual"].float()).to(s["residual"].dtype)
        more = [h]
    h = h.to(wide)
    y = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * s["weight"].to(wide)
    return (_to_codes(y) if c["out"] == "int8" else [y.to(_TYPES[c["out"]])]) + more


def _plain_quantise(s, c):
    y = s["x"].double()
    if c["swiglu"]:
        gate, up = y[:, :c["K"]], y[:, c["K"]:]
        y = gate * up / (1.0 + torch.exp(-gate))
    return _to_codes(y)


def _plain_gemm(s, c):
    y = torch.matmul(s["a"].float(), s["w"].float().t())
    y = y * s["a_scale"][:, None] * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(_TYPES[c["out"]])


def _order(x):
    """Whole numbers in the order of the values of x, which are not NaN; both zeros are equal."""
    b = (x + 0.0).view(torch.int32).long()
    return torch.where(b < 0, -(b & 0x7FFFFFFF), b)


def _plain_logprobs(s, c):
    x = s["logits"].float()
    d = (x - x.amax(1, keepdim=True)) * c["scale"]
    e = torch.exp(d)
    z = e.sum(1, keepdim=True)
    entropy = z[:, 0].log() - (e * d.clamp(min=-1e30)).sum(1) / z[:, 0]
    lp = lambda at: d.gather(1, at) - z.log()  # noqa: E731
    out = {"logprob": lp(s["tokens"].long()), "entropy": entropy}
    if c["k"]:
        V = c["V"]
        token = torch.topk((_order(x) << 32) + (V - 1 - torch.arange(V, device=DEV)), c["k"], 1).indices  # equal logits: by token
        out |= {"token": token.to(torch.int32), "top": lp(token)}
    return out


_PLAIN = {"norm": _plain_norm, "quantise": _plain_quantise, "gemm": _plain_gemm, "logprobs": _plain_logprobs}


# ---- from the definitions, in 64 bits ------------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, f64 = s["c"], torch.float64
    if c["kind"] == "gemm":
        a, out = s["a"].to(f64) * s["a_scale"].to(f64)[:, None], []
        for i in range(0, c["N"], 16384):  # channels by blocks
            w = s["w"][i:i + 16384].to(f64) * s["w_scale"][i:i + 16384].to(f64)[:, None]
            out.append((w @ a.t().contiguous()).t())
        y = torch.cat(out, 1)
        return y if s["bias"] is None else y + s["bias"].to(f64)
    if c["kind"] == "logprobs":
        lp, ent, token, top = [], [], [], []
        for i in range(0, c["rows"], 64):
            p = torch.log_softmax(s["logits"][i:i + 64].to(f64) * c["scale"], 1)
            lp.append(torch.take_along_dim(p, s["tokens"][i:i + 64].long(), 1))
            ent.append(-torch.xlogy(p.exp(), p.exp()).sum(1))
            if c["k"]:
                v, j = torch.sort(s["logits"][i:i + 64].to(f64), dim=1, descending=True, stable=True)
                token.append(j[:, :c["k"]].to(torch.int32))
                top.append(torch.take_along_dim(p, j[:, :c["k"]], 1))
        out = {"logprob": torch.cat(lp), "entropy": torch.cat(ent)}
        return out | {"token": torch.cat(token), "top": torch.cat(top)} if c["k"] else out
    more, x = [], s["x"].to(f64)
    if c["kind"] == "norm":
        if s["residual"] is not None:
            x = x + s["residual"].to(f64)
            more = [x]
            x = x.to(s["residual"].dtype).to(f64)  # the norm is of the stream as it is stored
        y = x / torch.sqrt(torch.sum(x * x, 1, keepdim=True) / c["K"] + EPS) * s["weight"].to(f64)
        if c["out"] != "int8":
            return [y] + more
    else:
        y = torch.nn.functional.silu(x[:, :c["K"]]) * x[:, c["K"]:] if c["swiglu"] else x
    scale = (torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 127).to(torch.float32).to(f64)
    return [torch.round(y / scale[:, None]) * scale[:, None], scale] + more
