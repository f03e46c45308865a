"""Cases of what many requests bring to a step: projections of any number of tokens through a block-quantized matrix with
low-rank adapters beside it (mul), and tokens sampled from their logits (sample).

A matrix is GGUF blocks: Q8_0, 34 bytes for 32 values (fp16 scale d, int8 codes q: d q), or Q4_0, 18 bytes (d, nibbles c: the
low ones values 0..15, the high ones 16..31: d (c - 8)).
"""

import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------
def _mul(name, w, rows, cols, tokens, dtype, slots, rank, run):
    """`slots` adapters of rank up to `rank` (0: none); a request has `run` tokens of the call, each its own adapter or none."""
    return dict(name=name, op="mul", w=w, rows=rows, cols=cols, tokens=tokens, dtype=dtype, slots=slots, rank=rank, run=run)


def _sample(name, requests, vocab, dtype, mode, mask):
    return dict(name=name, op="sample", requests=requests, vocab=vocab, dtype=dtype, mode=mode, mask=mask)


def listed():
    return [
        # a single request of the 135M shape, fp32 as in the framework's own step, with its adapter
        _mul("mul_1_576_f32", "q8_0", 576, 576, 1, "f32", 4, 8, 1),
        # one step of 16 requests of the 8B shape, each with another adapter
        _mul("mul_16_4096_bf16", "q8_0", 4096, 4096, 16, "bf16", 16, 16, 1),
        # a larger batch through a 7B shape's 4-bit gate projection, an odd count, fewer adapters than requests
        _mul("mul_61_11008_f16", "q4_0", 11008, 4096, 61, "f16", 9, 32, 1),
        # the 8B shape's head for 16 requests, without adapters
        _mul("mul_head_16_f32", "q8_0", 128256, 4096, 16, "f32", 0, 0, 1),
        # chunks of prompts beside each other, in fp32
        _mul("mul_500_4096_f32", "q8_0", 4096, 4096, 500, "f32", 3, 64, 130),
        # a long prompt through the 8B shape's widest product, several requests with adapters
        _mul("mul_8192_down_bf16", "q8_0", 4096, 14336, 8192, "bf16", 5, 16, 1500),
        # a single request, every filter
        _sample("sample_1_f32", 1, 49152, "f32", "all", "none"),
        # one step of 16 requests with parameters of their own
        _sample("sample_16_f32", 16, 128256, "f32", "mixed", "none"),
        # a grammar's mask leaves few tokens; 16-bit logits with many ties
        _sample("sample_61_bf16", 61, 32000, "bf16", "mixed", "grammar"),
        # temperature alone over the whole vocabulary
        _sample("sample_128_temperature", 128, 128256, "f32", "temperature", "none"),
        # the largest batch: top-k and top-p
        _sample("sample_512_f32", 512, 128256, "f32", "all", "none"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.55:
        rows, cols = rng.choice([(576, 576), (1536, 576), (576, 1536), (4096, 4096), (1024, 4096), (11008, 4096), (4096, 11008),
                                 (14336, 4096), (4096, 14336), (49152, 576), (32000, 4096), (992, 96), (4100, 2080)])
        most = min(8192, 8192 * 14336 * 4096 // (rows * cols), 2 ** 30 // rows)
        tokens = _log(rng, 1, most) if rng.random() < 0.6 else rng.randint(1, 64)
        slots = rng.choice([0, 1, 3, rng.randint(2, 64)])
        run = 1 if tokens <= 64 else _log(rng, 2, tokens)
        dtype = rng.choice(["f32", "f16", "bf16"])
        if dtype == "f32":  # (its products take longer: no more than the largest listed case's time)
            tokens = min(tokens, 2048)
        rank = rng.choice([1, 8, 16, 33, 64, 128]) if slots else 0
        while slots > 1 and tokens * slots * rank * (rows + cols) > 2 ** 37:  # (the plain form multiplies by every adapter)
            slots //= 2
        c = _mul("", rng.choice(["q8_0", "q4_0"]), rows, cols, tokens, dtype, slots, rank, run)
    else:
        vocab = rng.choice([49152, 32000, 128256, 1000, 50257, 151936, _log(rng, 2, 200000)])
        requests = min(_log(rng, 1, 512), 512 * 128256 // vocab)
        c = _sample("", requests, vocab, rng.choice(["f32", "f32", "bf16", "f16"]),
                    rng.choice(["temperature", "topk", "topp", "all", "mixed"]), rng.choice(["none", "none", "grammar"]))
    del c["name"]
    return c


def _ranks(c):
    """The adapters' ranks: the largest one first, smaller ones among the others."""
    return [max(1, c["rank"] - 5 * (i % 3)) for i in range(c["slots"])]


def _ids(c):
    """The adapter of each token (-1: none): a request's tokens share one, neighbours hardly ever do."""
    out, i = [], 0
    r = random.Random(c["tokens"] * 31 + c["slots"])
    while len(out) < c["tokens"]:
        n = 1 if c["run"] == 1 else r.randint(1, c["run"])
        out += [(-1 if c["slots"] == 0 or r.random() < 0.1 else (i * 7 + 3) % c["slots"] if c["slots"] % 7 else i % c["slots"])] * n
        i += 1
    return out[: c["tokens"]]


def work(c):
    if c["op"] == "mul":
        n, rows, cols, s = c["tokens"], c["rows"], c["cols"], SIZES[c["dtype"]]
        ids, ranks = _ids(c), _ranks(c)
        used = sum(ranks[i] for i in set(ids) if i >= 0)
        per = sum(ranks[i] for i in ids if i >= 0)
        w = rows * cols // 32 * (34 if c["w"] == "q8_0" else 18)
        return {"bytes": w + n * s * (rows + cols) + 2 * used * (rows + cols) + 4 * n, "flops": 2 * n * rows * cols + 2 * per * (rows + cols)}
    n = c["requests"] * c["vocab"]
    return {"bytes": n * SIZES[c["dtype"]] + c["requests"] * 28, "flops": 4 * n}


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _blocks(g, c):
    """Weights of about 1 / sqrt(cols), a scale for each 32: GGUF bytes [rows, cols / 32, 34 or 18]."""
    rows, nb = c["rows"], c["cols"] // 32
    top = 127 if c["w"] == "q8_0" else 8
    d = ((0.6 + 0.8 * _rand(g, rows, nb)) * 3.0 / (math.sqrt(c["cols"]) * top)).half()
    d = torch.where(_rand(g, rows, nb) < 0.5, -d, d) if c["w"] == "q4_0" else d  # a Q4_0 scale has its largest value's sign
    head = d.view(torch.uint8).view(rows, nb, 2)
    if c["w"] == "q8_0":
        q = (_randn(g, rows, nb, 32) * 42).round_().clamp_(-127, 127).to(torch.int8)
        return torch.cat([head, q.view(torch.uint8)], 2).contiguous()
    q = (_randn(g, rows, nb, 32) * 2.7).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
    return torch.cat([head, q[..., :16] | q[..., 16:] << 4], 2).contiguous()


def prepare(c, seed):
    g = _gen(seed)
    s = {"case": c, "seed": seed}
    if c["op"] == "sample":
        return s | _logits(g, c)
    dt, n, rows, cols = DTYPES[c["dtype"]], c["tokens"], c["rows"], c["cols"]
    s["blocks"] = _blocks(g, c)
    x = _randn(g, n, cols)
    x[:, torch.randint(0, cols, (3,), generator=g, device="cuda")] *= 12.0  # a few dims carry large activations
    s["x"] = x.to(dt)
    s["out"] = torch.empty((n, rows), dtype=dt, device="cuda")
    if c["slots"]:
        # adapters come in 16 bits: bf16, or fp16 where the rows are
        at = torch.float16 if c["dtype"] == "f16" else torch.bfloat16
        s["ranks"] = _ranks(c)
        s["a"] = [(_randn(g, r, cols) / math.sqrt(cols)).to(at) for r in s["ranks"]]
        s["b"] = [(_randn(g, rows, r) * 0.1).to(at) for r in s["ranks"]]
        s["scale"] = [2.0 * c["rank"] / r for r in s["ranks"]]
        shift = int(torch.randint(0, c["slots"], (1,), generator=g, device="cuda"))
        s["ids"] = torch.tensor([(i + shift) % c["slots"] if i >= 0 else -1 for i in _ids(c)], dtype=torch.int32, device="cuda")
        # the plain form's: every adapter below the other, zeros up to the largest rank
        big = torch.zeros((c["slots"], c["rank"], cols), dtype=at, device="cuda")
        bbig = torch.zeros((c["slots"], c["rank"], rows), dtype=at, device="cuda")
        for i, r in enumerate(s["ranks"]):
            big[i, :r], bbig[i, :r] = s["a"][i], s["b"][i].T
        s["a_all"], s["b_all"], s["scales"] = big.flatten(0, 1), bbig.flatten(0, 1), torch.tensor(s["scale"], device="cuda")
    return s


def _logits(g, c):
    n, v = c["requests"], c["vocab"]
    # a wide bulk far below a few dozen likely tokens, as a model's logits are; how far differs by request
    x = _randn(g, n, v).mul_(1.2 + 1.3 * _rand(g, n, 1))
    k = min(v, 48)
    step = v // k  # (places that no two share: one in each k-th of the vocabulary, turned)
    at = torch.randint(0, v, (n, 1), generator=g, device="cuda") + torch.arange(k, device="cuda") * step
    at = (at + torch.randint(0, step, (n, k), generator=g, device="cuda")) % v
    x.scatter_(1, at, 4.0 + _rand(g, n, 1) * 12.0 + 2.0 * _randn(g, n, k))
    if c["mask"] == "grammar":
        drop = _rand(g, n, v) < 0.97
        drop[:, int(torch.randint(0, v, (1,), generator=g, device="cuda"))] = False
        low = torch.where(torch.arange(n, device="cuda") % 2 == 0, -math.inf, torch.finfo(DTYPES[c["dtype"]]).min)
        x = torch.where(drop, low[:, None], x)
    row = torch.arange(n, device="cuda")

    def pick(values, step, on):
        t = torch.tensor(values, device="cuda")
        return t[(row * step + int(torch.randint(0, len(values), (1,), generator=g, device="cuda"))) % len(values)].contiguous() if on else None

    m = c["mode"]
    return dict(logits=x.to(DTYPES[c["dtype"]]).contiguous(), uniform=_rand(g, n),
                temperature=pick([0.7, 1.0, 0.0, 1.3, 0.2] if m == "mixed" else [0.8, 1.0, 1.2], 1, True),
                top_k=pick([50, 0, 1, 40, 1000, 7] if m == "mixed" else [50, 20, 200], 5, m in ("topk", "all", "mixed")),
                top_p=pick([0.9, 1.0, 0.95, 0.5] if m == "mixed" else [0.9, 0.95], 3, m in ("topp", "all", "mixed")),
                min_p=pick([0.0, 0.05, 0.0, 0.1, 0.0, 0.0, 0.2], 2, m == "mixed") if m != "all" else pick([0.02, 0.0], 1, True),
                tokens=torch.empty(n, dtype=torch.int32, device="cuda"), logprobs=torch.empty(n, device="cuda"))


# ---------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        return _own_mul(s, c) if c["op"] == "mul" else _own_sample(s, c)
    return _plain_mul(s, c) if c["op"] == "mul" else _plain_sample(s, c)


def _own_mul(s, c):
    if "matrix" not in s:  # the matrix and the adapters that a program keeps: made in a state's first pass
        from block_quantized_token_gb300 import runtime
        s["matrix"] = runtime.Matrix(c["w"], c["rows"], c["cols"], s["blocks"])
        s["adapters"] = None
        if c["slots"]:
            s["adapters"] = runtime.Adapters(c["rows"], c["cols"], c["slots"], c["rank"], s["a"][0].dtype)
            for i in range(c["slots"]):
                s["adapters"].set(i, s["a"][i], s["b"][i], s["scale"][i])
    s["matrix"].mul(s["x"], s["out"], adapters=s["adapters"], ids=s.get("ids"))
    return s["out"]


def _own_sample(s, c):
    from block_quantized_token_gb300 import runtime
    runtime.sample(s["logits"], s["uniform"], s["tokens"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                   min_p=s["min_p"], logprobs=s["logprobs"])
    return [s["tokens"], s["logprobs"]]


def _dequantize(blocks, w):
    """GGUF bytes -> fp32 [rows, cols] (every value exact)."""
    d = blocks[..., :2].contiguous().view(torch.float16).float()
    q = blocks[..., 2:]
    if w == "q8_0":
        v = q.contiguous().view(torch.int8).float()
    else:
        v = torch.cat([q & 15, q >> 4], 2).float() - 8
    return (v * d).flatten(1)


def _plain_mul(s, c):
    x = s["x"].float()
    y = torch.matmul(x, _dequantize(s["blocks"], c["w"]).T)
    if c["slots"]:
        v = torch.matmul(x, s["a_all"].float().T).view(len(x), c["slots"], -1)
        mine = (s["ids"][:, None] == torch.arange(c["slots"], device="cuda")).float() * s["scales"]
        y += torch.matmul((v * mine[..., None]).flatten(1), s["b_all"].float())
    return y.to(s["x"].dtype)


def _plain_sample(s, c):
    n, v = s["logits"].shape
    x = s["logits"].double()  # tokens are decided next to borders
    top = x.amax(1, keepdim=True)
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    z = torch.where(torch.isinf(x) & (x < 0), x, (x - top) / torch.where(greedy, torch.ones_like(t), t))
    z, order = torch.sort(z, dim=1, descending=True, stable=True)
    e = torch.exp(z)
    rank = torch.arange(v, device="cuda")[None]
    keep = rank < torch.where(greedy, 1, v)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep = keep & (rank < torch.where(k <= 0, v, k))
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        within = e * keep
        before = torch.cumsum(within, 1) - within
        keep = keep & ((before < p * within.sum(1, keepdim=True)) | (rank == 0) | (p >= 1))
    if s["min_p"] is not None:
        keep = keep & ((e >= s["min_p"].double()[:, None]) | (rank == 0))
    e = torch.zeros_like(e).scatter_(1, order, e * keep)  # in the vocabulary's order
    cum = torch.cumsum(e, 1)
    total = cum[:, -1:]
    token = (cum <= s["uniform"].double()[:, None] * total).sum(1).clamp(max=v - 1)
    z = torch.log(e.gather(1, token[:, None])[:, 0]) - torch.log(total[:, 0])
    return [token.int(), z.float()]


# ---------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------
def _exact_mul(c, seed):
    if 2 * c["tokens"] * c["rows"] * c["cols"] > 2e12:
        return None
    s = prepare(c, seed)
    x, rows = s["x"].double(), c["rows"]
    out = torch.empty((c["tokens"], rows), dtype=torch.float64, device="cuda")
    for r in range(0, rows, 4096):
        b = s["blocks"][r:r + 4096]
        d = (b[..., 0].int() | b[..., 1].int() << 8).to(torch.int16).view(torch.float16).double()[..., None]
        if c["w"] == "q8_0":
            q = b[..., 2:].double()
            q = torch.where(q > 127, q - 256, q)
        else:
            q = torch.cat([b[..., 2:].double() % 16, torch.floor(b[..., 2:].double() / 16)], 2) - 8
        out[:, r:r + 4096] = torch.einsum("nk,rk->nr", x, (d * q).reshape(len(b), -1))
    for i in range(c["slots"]):
        at = (s["ids"] == i).nonzero()[:, 0]
        if len(at):
            out[at] += s["scale"][i] * torch.einsum("nj,rj->nr", torch.einsum("nk,jk->nj", x[at], s["a"][i].double()), s["b"][i].double())
    return out


def _exact_sample(c, seed):
    s = prepare(c, seed)
    out = []
    for i in range(c["requests"]):
        x = s["logits"][i].double()
        t = float(s["temperature"][i])
        if t <= 0:
            out.append(0.0)
            continue
        at = torch.argsort(-x, stable=True)
        z = x[at] / t
        if s["top_k"] is not None and int(s["top_k"][i]) > 0:
            at, z = at[: int(s["top_k"][i])], z[: int(s["top_k"][i])]
        w = torch.softmax(z, 0)
        n = len(w)
        if s["top_p"] is not None and float(s["top_p"][i]) < 1:
            n = 1 + int((torch.cumsum(w, 0)[:-1] < float(s["top_p"][i])).sum())
        if s["min_p"] is not None:
            n = min(n, max(1, int((w >= float(s["min_p"][i]) * w[0]).sum())))
        at, w = at[:n], w[:n]
        by, order = torch.sort(at)
        cum = torch.cumsum(w[order], 0)
        j = min(int((cum <= float(s["uniform"][i]) * cum[-1]).sum()), n - 1)
        out.append(float(torch.log(w[order][j] / cum[-1])))
    return [None, torch.tensor(out, dtype=torch.float64, device="cuda")]


def exact(c, seed):
    return _exact_mul(c, seed) if c["op"] == "mul" else _exact_sample(c, seed)
