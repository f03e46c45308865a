"""Cases of the paged 4-bit K/V cache: its block tables (plan), its rows (append) and the attention over it (attend).

The cache is a pool of pages; page p of KV head h holds `page_rows` rows as whole tiles of 16 rows, each tile 18 * hd
bytes: K codes [8 hd], K scales [hd], V codes [8 hd], V scales [hd].  A row is hd / 32 blocks; a value is d * (c - 8)
with an fp16 scale d and a 4-bit code c.  `pack` below writes a tile and `unpack` reads one.
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
def _plan(name, seqs, lo, hi, new_lo, new_hi, page):
    return dict(name=name, op="plan", seqs=seqs, len_lo=lo, len_hi=hi, new_lo=new_lo, new_hi=new_hi, page=page)


def _append(name, heads, kv, hd, tokens, dtype, page, norm, style):
    return dict(name=name, op="append", heads=heads, kv=kv, hd=hd, tokens=tokens, dtype=dtype, page=page, norm=norm,
                style=style)


def _attend(name, heads, kv, hd, seqs, lo, hi, new_lo, new_hi, dtype, page, window=0):
    return dict(name=name, op="attend", heads=heads, kv=kv, hd=hd, seqs=seqs, len_lo=lo, len_hi=hi, new_lo=new_lo,
                new_hi=new_hi, dtype=dtype, page=page, window=window)


def listed():
    return [
        # one decode step of the 16-sequence workload: a token each, positions around 8192
        _plan("plan_step_16", 16, 8100, 8250, 1, 1, 16),
        # admission of a full batch: prompts of every length next to running requests
        _plan("plan_prompts_512", 512, 0, 900, 0, 250, 16),
        # the rows of one decode step of 16 sequences, 32 query heads on 8 K/V heads
        _append("append_step_16", 32, 8, 128, 16, "bf16", 16, True, "pairs"),
        # a ragged chunk of the 9/3-head shape in the framework's fp32 activations, no norms
        _append("append_f32_1000", 9, 3, 64, 1000, "f32", 32, False, "pairs"),
        # a whole prompt of 8192 tokens
        _append("append_prompt_8192", 32, 8, 128, 8192, "bf16", 16, True, "halves"),
        # single-sequence decode of the 135M shape at context 2048, fp32 activations
        _attend("decode_1x2048_f32", 9, 3, 64, 1, 2049, 2049, 1, 1, "f32", 16),
        # single-sequence decode with as many K/V heads as query heads at context 4096
        _attend("decode_1x4096_f16", 32, 32, 128, 1, 4097, 4097, 1, 1, "f16", 64),
        # a serving batch: ragged contexts, some requests empty, a sliding window
        _attend("decode_61_ragged_bf16", 32, 8, 128, 61, 0, 4001, 1, 1, "bf16", 16, window=1500),
        # the 16-sequence workload at context 8192
        _attend("decode_16x8192_bf16", 32, 8, 128, 16, 8193, 8193, 1, 1, "bf16", 16),
        # the same in fp32, the type of the framework's own step
        _attend("decode_16x8192_f32", 32, 8, 128, 16, 8193, 8193, 1, 1, "f32", 16),
        # chunks of four prompts on top of what is cached
        _attend("chunks_4x500_f32", 32, 8, 128, 4, 900, 4100, 300, 500, "f32", 16),
        # a whole prompt
        _attend("prompt_8192_bf16", 32, 8, 128, 1, 8192, 8192, 8192, 8192, "bf16", 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    heads, kv, hd = rng.choice([(9, 3, 64), (32, 8, 128), (32, 32, 128), (8, 1, 64), (32, 8, 64), (5, 5, 128)])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "plan":
        hi = _log(rng, 16, 8000)
        c = _plan("", _log(rng, 1, 512), rng.randrange(0, hi), hi, 0, _log(rng, 1, 250), page)
    elif op == "append":
        c = _append("", heads, kv, hd, _log(rng, 1, 32000 // (heads + kv)), dtype, page, rng.random() < 0.6, rng.choice(["pairs", "halves"]))
    elif rng.random() < 0.6:  # decode, one token each or a few
        seqs = _log(rng, 1, 64)
        hi = min(_log(rng, 1, 16000), 16 * 8192 * 8 // (seqs * kv))
        c = _attend("", heads, kv, hd, seqs, rng.choice([0, hi // 2, hi]), hi, 1, rng.choice([1, 1, 1, 4]), dtype, page,
                    rng.choice([0, 0, 0, _log(rng, 1, 4000)]))
    else:  # prompts and chunks
        new = _log(rng, 17, 3000)
        seqs = rng.randint(1, max(1, min(8, 6000 // new)))
        hi = new + _log(rng, 1, 3000)
        c = _attend("", heads, kv, hd, seqs, rng.choice([new, hi]), hi, rng.randint(1, new), new, dtype, page,
                    rng.choice([0, 0, 0, _log(rng, 16, 2000)]))
    del c["name"]
    return c


def _spread(n, lo, hi, at):
    """n whole numbers over [lo, hi], both ends among them where n > 1."""
    if n == 1:
        return [hi]
    order = list(range(n))
    random.Random(at).shuffle(order)
    return [lo + (hi - lo) * k // (n - 1) for k in order]


def _lengths(c):
    """What each request holds before the call (plan) or after its new tokens are in (attend), and its new tokens."""
    return _spread(c["seqs"], c["len_lo"], c["len_hi"], 1), _spread(c["seqs"], c["new_lo"], c["new_hi"], 2)


def _attended(c):
    """Pairs of a token and a row that it attends, and rows that any token attends, over all sequences."""
    every = [(n, max(0, n - t), c["window"] or n + 1) for n, t in zip(*_lengths(c))]
    pairs = sum(min(w, p + 1) for n, first, w in every for p in range(first, n))
    return pairs, sum(n - max(0, first - w + 1) for n, first, w in every if n)


def work(c):
    if c["op"] == "plan":
        lens, new = _lengths(c)
        pages = sum(-(-(a + b) // c["page"]) - -(-a // c["page"]) for a, b in zip(lens, new))
        return {"bytes": 4 * (4 * c["seqs"] + 2 * pages + 3 * sum(new)), "flops": 0}
    if c["op"] == "append":
        s, t = SIZES[c["dtype"]], c["tokens"]
        row, kvd = c["heads"] * c["hd"], c["kv"] * c["hd"]
        # q, k, v in; q out; the cache's rows out and, as the pass returns them, back as values
        return {"bytes": t * (2 * s * row + 2 * s * kvd + 2 * kvd * 9 // 16 * 2 + 2 * s * kvd + 4 * c["hd"] + 8), "flops": t * (row + kvd) * 8}
    pairs, rows = _attended(c)
    s, t = SIZES[c["dtype"]], sum(_lengths(c)[1])
    return {"bytes": rows * c["kv"] * c["hd"] * 9 // 8 + t * c["heads"] * (2 * s * c["hd"] + 4), "flops": 4 * pairs * c["heads"] * c["hd"]}


# ---------------------------------------------------------------------------------------------------
# the pool's bytes
# ---------------------------------------------------------------------------------------------------
def _halves(d):
    return d.contiguous().view(torch.uint8)


def quantize(x):
    """fp32 [..., n] -> codes uint8 [..., n], scales fp16 [..., n / 32]: m the first value of the largest size,
    d = fp16(bf16(-m / 8)) within +-2720, c = clamp(round(x / d) + 8, 0, 15), halves away from zero; 8 where d is 0."""
    b = x.unflatten(-1, (-1, 32))
    at = b.abs().argmax(-1, keepdim=True)
    d = (b.gather(-1, at)[..., 0] * -0.125).bfloat16().float().clamp(-2720.0, 2720.0).half()
    r = b / d.float()[..., None]
    r = torch.where(d[..., None] == 0, torch.zeros_like(r), r).double()
    r = torch.sign(r) * torch.floor(r.abs() + 0.5)
    return (r + 8).clamp(0, 15).to(torch.uint8).flatten(-2), d


def pack(kc, kd, vc, vd):
    """Codes [tiles, 16, hd] and scales [tiles, 16, hd / 32] of K and V -> tiles' bytes [tiles, 18 hd]."""
    n, _, hd = kc.shape
    k = kc.view(n, 16, hd // 32, 4, 4, 2).permute(0, 1, 3, 2, 5, 4).reshape(n, 8 * hd, 2)
    v = vc.view(n, 2, 4, 2, hd // 64, 4, 2, 8).permute(0, 4, 7, 2, 5, 3, 1, 6).reshape(n, 8 * hd, 2)
    vs = vd.view(n, 2, 4, 2, hd // 32).permute(0, 2, 4, 1, 3).reshape(n, hd // 2)
    return torch.cat([k[..., 0] | k[..., 1] << 4, _halves(kd.reshape(n, hd // 2)), v[..., 0] | v[..., 1] << 4, _halves(vs)], 1)


def unpack(tiles):
    """Tiles' bytes [tiles, 18 hd] -> K and V values fp32 [tiles, 16, hd] (every one exact)."""
    n, hd = tiles.shape[0], tiles.shape[1] // 18
    kc, ks, vc, vs = tiles.split([8 * hd, hd, 8 * hd, hd], 1)
    k = torch.stack([kc & 15, kc >> 4], -1).view(n, 16, 4, hd // 32, 2, 4).permute(0, 1, 3, 2, 5, 4)
    v = torch.stack([vc & 15, vc >> 4], -1).view(n, hd // 64, 8, 4, 4, 2, 2, 2).permute(0, 6, 3, 5, 1, 4, 7, 2)
    kd = ks.contiguous().view(torch.float16).view(n, 16, hd // 32, 1)
    vd = vs.contiguous().view(torch.float16).view(n, 4, hd // 32, 2, 2).permute(0, 3, 1, 4, 2).reshape(n, 16, hd // 32, 1)
    return ((k.reshape(n, 16, hd // 32, 32).float() - 8) * kd.float()).flatten(2), ((v.reshape(n, 16, hd // 32, 32).float() - 8) * vd.float()).flatten(2)


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(g, blocks, page_count, stride):
    """A block table [seqs, stride] of pages in random order, -1 past each request's own, and the free pages."""
    order = torch.randperm(page_count, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(blocks, device="cuda")
    at = torch.arange(stride, device="cuda")[None, :]
    first = (n.cumsum(0) - n)[:, None]
    used = int(sum(blocks))
    t = torch.where(at < n[:, None], order[(first + at).clamp(max=page_count - 1)], torch.full_like(order[:1], -1))
    return t.contiguous(), order[used:].contiguous()


def _rows(c, seed):
    """The cached rows of an attend case: per sequence and K/V head, padded to whole pages of the longest."""
    g = _gen(seed)
    lens, _ = _lengths(c)
    blocks = [-(-n // c["page"]) for n in lens]
    top = max(1, max(blocks)) * c["page"]
    shape = (c["seqs"], c["kv"], top, c["hd"])
    # keys of unit size, as after their norm; values somewhat smaller
    kc, kd = quantize(torch.randn(shape, generator=g, device="cuda"))
    vc, vd = quantize(torch.randn(shape, generator=g, device="cuda").mul_(0.7))
    t = sum(_lengths(c)[1])
    q = torch.randn((t, c["heads"], c["hd"]), generator=g, device="cuda").to(DTYPES[c["dtype"]])
    return g, (kc, kd, vc, vd), q, blocks, top


def _append_inputs(c, seed):
    g = _gen(seed)
    t, h, kv, hd = c["tokens"], c["heads"], c["kv"], c["hd"]
    # one row of the fused projection a token: the queries, then the keys, then the values
    qkv = (torch.randn((t, (h + 2 * kv) * hd), generator=g, device="cuda") * 1.5).to(DTYPES[c["dtype"]])
    gains = [1 + 0.1 * torch.randn(hd, generator=g, device="cuda") for _ in range(2)]
    return g, qkv, gains


def _rope(hd, n):
    i = torch.arange(hd // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"), -2.0 * i / hd)
    return torch.stack([torch.cos(a), torch.sin(a)], -1).float().contiguous()


def prepare(c, seed):
    s = {"case": c, "seed": seed}
    if c["op"] == "plan":
        lens, new = _lengths(c)
        g = _gen(seed)
        # another seed has other lengths: the same ones in another order
        order = torch.randperm(c["seqs"], generator=g, device="cuda").tolist()
        lens, new = [lens[i] for i in order], [new[i] for i in order]
        if c["seqs"] == 1:
            lens = [max(0, lens[0] - seed % 7)]
        blocks = [-(-n // c["page"]) for n in lens]
        most = sum(-(-(a + b) // c["page"]) for a, b in zip(lens, new))
        pages = most + most // 4 + 16
        stride = -(-(c["len_hi"] + c["new_hi"]) // c["page"])
        tables, free = _tables(g, blocks, pages, stride)
        tokens = max(1, sum(_lengths(c)[1]))
        full = torch.zeros(pages, dtype=torch.int32, device="cuda")
        full[: len(free)] = free
        s |= dict(lens=_ints(lens), new=_ints(new), tables=tables, free=full, count=_ints([len(free)]), pages=pages,
                  tokens=tokens, lens_out=_ints(lens), count_out=_ints([0]), q_start=_ints([0] * (c["seqs"] + 1)),
                  positions=_ints([0] * tokens), slots=_ints([0] * tokens), seqs=_ints([0] * tokens))
        return s
    if c["op"] == "append":
        g, qkv, gains = _append_inputs(c, seed)
        t, h, kv, hd, page = c["tokens"], c["heads"], c["kv"], c["hd"], c["page"]
        start = 37 if t > 64 else 2000  # prompts start inside a page, steps far on
        pages = -(-(t + start) // page) + 3
        step = t <= 64
        if step:  # one token of each of t sequences, each in a page of its own
            pages = t + 3
            order = torch.randperm(pages, generator=g, device="cuda")[:t]
            slots = order * page + torch.randint(0, page, (t,), generator=g, device="cuda")
            pos = start + torch.randint(0, 4000, (t,), generator=g, device="cuda")
        else:
            order = torch.randperm(pages, generator=g, device="cuda")
            pos = start + torch.arange(t, device="cuda")
            slots = order[pos // page] * page + pos % page
        dt = DTYPES[c["dtype"]]
        return s | dict(qkv=qkv, q=qkv[:, : h * hd].view(t, h, hd), k=qkv[:, h * hd:(h + kv) * hd].view(t, kv, hd),
                        v=qkv[:, (h + kv) * hd:].view(t, kv, hd), q_gain=gains[0] if c["norm"] else None,
                        k_gain=gains[1] if c["norm"] else None, rope=_rope(hd, int(pos.max()) + 1),
                        positions=pos.int().contiguous(), slots=slots.int().contiguous(), pages=pages,
                        pool=torch.zeros((pages, kv, page // 16, 18 * hd), dtype=torch.uint8, device="cuda"),
                        q_out=torch.empty((t, h, hd), dtype=dt, device="cuda"),
                        k_out=torch.empty((t, kv, hd), dtype=dt, device="cuda"),
                        v_out=torch.empty((t, kv, hd), dtype=dt, device="cuda"))
    g, (kc, kd, vc, vd), q, blocks, top = _rows(c, seed)
    page, kv, hd = c["page"], c["kv"], c["hd"]
    pages = sum(blocks) + 2
    tables, _ = _tables(g, blocks, pages, top // page)
    pool = torch.randint(0, 256, (pages, kv, page // 16 * 18 * hd), dtype=torch.uint8, generator=g, device="cuda")
    per = 16 * max(1, 2 ** 24 // (kv * hd * 16))
    for b in range(c["seqs"]):  # a page's rows past the request's length hold what the row maker drew for them
        n = blocks[b] * page
        for r in range(0, n, per * page):
            e = min(n, r + per * page)
            tiles = pack(*(x[b, :, r:e].reshape(kv * (e - r) // 16, 16, -1) for x in (kc, kd, vc, vd)))
            tiles = tiles.view(kv, (e - r) // page, -1).transpose(0, 1)
            pool[tables[b, r // page:e // page].long()] = tiles
    lens, new = _lengths(c)
    start = [sum(new[:b]) for b in range(len(new) + 1)]
    return s | dict(pool=pool, tables=tables, lens=_ints(lens), q_start=_ints(start), q=q, out=torch.empty_like(q), pages=pages,
                    lse=torch.empty(q.shape[:2], dtype=torch.float32, device="cuda"))


# ---------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        return {"plan": _own_plan, "append": _own_append, "attend": _own_attend}[c["op"]](s, c)
    return {"plan": _plain_plan, "append": _plain_append, "attend": _plain_attend}[c["op"]](s, c)


def _cache(s, c, kv, hd):
    """The handle that a program keeps: made in a state's first pass."""
    if "cache" not in s:
        from block_quantized_token_gb300 import runtime
        s["cache"] = runtime.PagedCache(1, s["pages"], c["page"], kv, hd, pool=s.get("pool"))
    return s["cache"]


def _own_plan(s, c):
    _cache(s, c, 1, 64).plan(s["lens"], s["new"], s["tables"], s["free"], s["count"], s["lens_out"], s["count_out"],
                             s["q_start"], s["positions"], s["slots"], s["seqs"])
    return [s[k] for k in ("lens_out", "count_out", "tables", "q_start", "positions", "slots", "seqs")]


def _own_append(s, c):
    cache = _cache(s, c, c["kv"], c["hd"])
    cache.append(0, s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"], q_gain=s["q_gain"], k_gain=s["k_gain"],
                 eps=1e-5, rope=s["rope"], rope_style=c["style"])
    cache.read(0, s["slots"], s["k_out"], s["v_out"])
    return [s["q_out"], s["k_out"], s["v_out"]]


def _own_attend(s, c):
    _cache(s, c, c["kv"], c["hd"]).attention(0, s["q"], s["out"], s["q_start"], s["lens"], s["tables"], window=c["window"], lse=s["lse"])
    return [s["out"], s["lse"]]


def _plain_plan(s, c):
    lens, new, page = s["lens"].long(), s["new"].long(), c["page"]
    have = (lens + page - 1) // page
    need = (lens + new + page - 1) // page - have
    count = s["count"].long()
    fits = (need.cumsum(0) <= count) & (new.cumsum(0) <= s["tokens"])
    new, need = new * fits, need * fits
    first = need.cumsum(0) - need
    at = torch.arange(s["tables"].shape[1], device="cuda")[None, :] - have[:, None]
    got = (at >= 0) & (at < need[:, None])
    taken = s["free"][(count - 1 - first[:, None] - at).clamp(min=0, max=len(s["free"]) - 1)]
    tables = torch.where(got, taken, s["tables"])
    end = new.cumsum(0)
    q_start = torch.cat([torch.zeros_like(end[:1]), end])
    row = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(end, row, right=True)
    there = row < end[-1]
    of = seq.clamp(max=c["seqs"] - 1)
    pos = lens[of] + row - q_start[of]
    slot = tables[of, (pos // page).clamp(max=tables.shape[1] - 1)] * page + pos % page
    left = [(lens + new).int(), (count - need.sum()).int(), tables, q_start.int()]
    return left + [torch.where(there, pos, 0).int(), torch.where(there, slot, -1).int(), torch.where(there, of, -1).int()]


def _turn(x, cs, style):
    """Rotates the pairs of x [t, h, hd] by (cos, sin) [t, hd / 2, 2] in x's type."""
    cos, sin = cs[:, None, :, 0].to(x.dtype), cs[:, None, :, 1].to(x.dtype)
    a, b = (x[..., 0::2], x[..., 1::2]) if style == "pairs" else x.chunk(2, -1)
    y = a * cos - b * sin, b * cos + a * sin
    return torch.stack(y, -1).flatten(-2) if style == "pairs" else torch.cat(y, -1)


def _plain_append(s, c):
    cs = s["rope"][s["positions"].long()]
    q, k = s["q"].float(), s["k"].double()  # keys in 64 bits: their codes are decided next to borders
    if c["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + 1e-5) * s["q_gain"]
        k = k / torch.sqrt((k * k).mean(-1, keepdim=True) + 1e-5) * s["k_gain"].double()
    q, k = _turn(q, cs, c["style"]), _turn(k, cs, c["style"]).float()
    code, d = quantize(torch.stack([k, s["v"].float()]))
    k, v = ((code.unflatten(-1, (-1, 32)).float() - 8) * d.float()[..., None]).flatten(-2).to(s["q_out"].dtype)
    return [q.to(s["q_out"].dtype), k, v]


def _plain_attend(s, c):
    kv, hd, page, b = c["kv"], c["hd"], c["page"], c["seqs"]
    g = c["heads"] // kv
    tables = s["tables"].long().clamp(min=0)
    n = tables.shape[1] * page
    tiles = s["pool"][tables].view(b, -1, kv, page // 16, 18 * hd).transpose(1, 2).reshape(-1, 18 * hd)
    k, v = (x.view(b, kv, n, hd) for x in unpack(tiles))
    start, lens = s["q_start"].long(), s["lens"].long()
    new = start[1:] - start[:-1]
    most = c["new_hi"]
    i = torch.arange(most, device="cuda")
    at = (start[:-1, None] + i).clamp(max=len(s["q"]) - 1)
    real = i < new[:, None]
    q = s["q"].float()[at].view(b, most, kv, g, hd).permute(0, 2, 3, 1, 4).reshape(b, kv, g * most, hd)
    p = (lens - new)[:, None] + i  # positions of the tokens
    row = torch.arange(n, device="cuda")
    see = (row <= p[..., None]) & (row < lens[:, None, None])
    if c["window"]:
        see = see & (row > p[..., None] - c["window"])
    x = torch.matmul(q, k.transpose(2, 3)).mul_(1 / math.sqrt(hd)).view(b, kv, g, most, n)
    x.masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = x.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(b, kv, g * most, n), v).view(b, kv, g, most, hd) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total))[..., 0]
    pick = real.flatten().nonzero()[:, 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(b * most, c["heads"], hd)[pick]
    return [o.to(s["q"].dtype), lse.permute(0, 3, 1, 2).reshape(b * most, c["heads"])[pick]]


# ---------------------------------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence and head by head
# ---------------------------------------------------------------------------------------------------
def _value(code, d):
    return (code.double() - 8) * torch.repeat_interleave(d.double(), 32, -1)


def _stored(y):
    """What the cache holds of y (64 bits) [..., n]."""
    b = y.float().double().unflatten(-1, (-1, 32))  # the row in fp32 is what is quantised
    hi, lo = b.amax(-1), -b.amin(-1)
    first = (b == hi[..., None]).double().argmax(-1) < (b == -lo[..., None]).double().argmax(-1)
    m = torch.where((hi > lo) | ((hi == lo) & first), hi, -lo)
    f, e = torch.frexp(m / -8)
    d = torch.ldexp(torch.round(f * 256), e - 8).clamp(-2720, 2720)  # 8 significant bits
    d = (torch.round(d * 2 ** 24) / 2 ** 24)[..., None]  # fp16's smallest step
    r = torch.where(d == 0, torch.zeros_like(b), b / torch.where(d == 0, torch.ones_like(d), d))
    c = torch.where(r < 0, torch.ceil(r - 0.5), torch.floor(r + 0.5)).clamp(-8, 7)
    return (c * d).flatten(-2)


def exact(c, seed):
    if c["op"] == "plan":
        return None  # whole numbers
    if c["op"] == "append":
        s = prepare(c, seed)
        hd, pos = c["hd"], s["positions"].long()
        angle = s["rope"].double()[pos]
        z = torch.complex(angle[..., 0], angle[..., 1])[:, None]
        out = []
        for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"]), (s["v"], None)):
            y = x.double()
            if x is not s["v"]:
                if gain is not None:
                    y = y * (gain.double() / torch.sqrt(torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / hd + 1e-5))
                if c["style"] == "pairs":
                    y = torch.view_as_real(torch.view_as_complex(y.reshape(*y.shape[:-1], hd // 2, 2).contiguous()) * z).flatten(-2)
                else:
                    w = torch.complex(y[..., : hd // 2].contiguous(), y[..., hd // 2:].contiguous()) * z
                    y = torch.cat([w.real, w.imag], -1)
            if x is not s["q"]:
                y = _stored(y)
            out.append(y)
        return out
    g, (kc, kd, vc, vd), q, _, _ = _rows(c, seed)
    lens, new = _lengths(c)
    t, group = len(q), c["heads"] // c["kv"]
    if 4 * _attended(c)[0] * c["heads"] * c["hd"] > 3e12:
        return None
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        for h in range(c["heads"] if n and m else 0):
            k, v = _value(kc[b, h // group, :n], kd[b, h // group, :n]), _value(vc[b, h // group, :n], vd[b, h // group, :n])
            p = torch.arange(n - m, n, device="cuda")[:, None]
            r = torch.arange(n, device="cuda")[None]
            seen = (r <= p) & ((r > p - c["window"]) if c["window"] else (r >= 0))
            x = (q[at:at + m, h].double() @ k.T) / math.sqrt(c["hd"])
            x = x.masked_fill(~seen, -math.inf)
            z = torch.logsumexp(x, -1)
            w = torch.where(seen, torch.exp(x - z.masked_fill(torch.isinf(z), 0.0)[:, None]), torch.zeros_like(x))
            o[at:at + m, h], lse[at:at + m, h] = w @ v, z
        at += m
    return [o, lse]
