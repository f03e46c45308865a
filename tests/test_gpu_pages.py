"""The paged 4-bit K/V cache on the GPU (er_pages_*) against its float64 oracle (oracle/pages.py).

Tolerances, u = 2^-24 (float32's half step), h = half a step of the output type (2^-24, 2^-11, 2^-8):
* cache codes and scales, block tables, slots: equal.
* append's queries: the norm and the rotation take at most 16 float32 roundings of |a| + |b| of a pair; then h.
* attention.  A score: the queries' two halves carry 22 bits (2^-22 of the row's largest, sqrt(hd) of it at most of
  sum |q||k| for these inputs: counted as 2^-21 of S = scale sum |q||k|) and hd / 16 products of 16 terms are
  added with float32 truncation (2^-23 each): together below hd / 16 * 2^-23 S + 2^-21 S <= 2^-19 S for hd = 128.
  A probability is off by twice that (its own score and the maximum's), by 2^-21 from its exponential and by
  2^-21 from its two halves; o and l add up to N / 16 + 64 products with 2^-23 each.  With |v| <= vmax:
      |out - exact| <= vmax (4 S 2^-19 + 2^-19 + 2 (N / 16 + 64) 2^-23) + h |exact|.
  16-bit types whose probabilities enter as one half: 2 * 2^-11 vmax more.  lse: the score's 2^-19 S, l's
  (N / 16 + 64) 2^-23 + 2^-20, and 4 u |lse|.
"""

from __future__ import annotations

import numpy as np
import pytest

from oracle import pages as op

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def host(t):
    return t.detach().cpu().double().numpy()


def paged(n_pages, page_rows, kv, hd, layers=1, fill=None, pool=None):
    from block_quantized_token_gb300 import runtime
    c = runtime.PagedCache(layers, n_pages, page_rows, kv, hd, pool=pool)
    if fill is not None:
        c.pool.copy_(fill(c.pool.numel()))
    return c


def noise(seed):
    def make(n):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda", generator=g)
    return make


def fine(cache, want=0):
    _, code = cache.error()
    assert code == want, code


# ------------------------------------------------------------------------------------------------------------------
# plan and release
# ------------------------------------------------------------------------------------------------------------------
def run_plan(cache, lens, new, tables, free, count, max_tokens, alias=False):
    n = len(lens)
    d = dict(lens=ints(lens), new=ints(new), tables=ints(tables), free=ints(free), count=ints([count]),
             q=ints([-7] * (n + 1)), pos=ints([-7] * max_tokens), slot=ints([-7] * max_tokens), seq=ints([-7] * max_tokens))
    lo, co = (d["lens"], d["count"]) if alias else (ints([-7] * n), ints([-7]))
    cache.plan(d["lens"], d["new"], d["tables"], d["free"], d["count"], lo, co, d["q"], d["pos"], d["slot"], d["seq"])
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (lo, co, d["tables"], d["q"], d["pos"], d["slot"], d["seq"])]


@pytest.mark.parametrize("n,page,top,new_top,room", [(1, 16, 40, 1, 1.0), (16, 16, 8000, 2, 1.0), (3, 48, 100, 64, 1.0),
                                                     (257, 64, 900, 9, 1.0), (1024, 16, 60, 40, 1.0),
                                                     (300, 16, 500, 200, 0.6), (64, 32, 0, 0, 1.0)])
@pytest.mark.parametrize("alias", [False, True])
def test_plan(n, page, top, new_top, room, alias):
    rng = np.random.default_rng(n + page)
    lens, new = rng.integers(0, top + 1, n), rng.integers(0, new_top + 1, n)
    if n > 3:
        lens[1] = new[2] = 0
    if n > 200:
        lens[50], new[60] = -3, -1  # refused by themselves
    stride = -(-(top + new_top + 1) // page)
    have = [-(-max(0, int(x)) // page) for x in lens]
    extra = sum(-(-max(0, int(a) + int(b)) // page) for a, b in zip(lens, new))
    total = sum(have) + int(extra * room) + 3
    order = rng.permutation(total)
    tables, at = np.full((n, stride), -1), 0
    for b in range(n):
        tables[b, :have[b]] = order[at:at + have[b]]
        at += have[b]
    count = max(1, int((total - at) * (0.5 if room < 1 else 1.0)))
    free = np.zeros(total, int)
    free[:total - at] = order[at:]
    rows = max(1, int(new.clip(0).sum() * (0.9 if room < 1 else 1.0)))
    cache = paged(total, page, 1, 64)
    got = run_plan(cache, lens, new, tables, free, count, rows, alias)
    *want, flags = op.plan(lens, new, tables, free, count, rows, page)
    for name, g, w in zip(("lens", "count", "tables", "q_start", "positions", "slots", "seqs"), got, want):
        np.testing.assert_array_equal(g.reshape(-1), np.asarray(w).reshape(-1), err_msg=name)
    fine(cache, flags)


def test_plan_refuses_by_table_and_bad_pages():
    cache = paged(20, 16, 1, 64)
    # request 1's rows pass its table of 2 pages; request 2 holds a page outside the pool
    tables = np.array([[3, -1], [4, 5], [99, -1]])
    got = run_plan(cache, [16, 32, 5], [1, 1, 2], tables, list(range(20)), 10, 8)
    assert list(got[0]) == [17, 32, 7] and list(got[3]) == [0, 1, 1, 3]
    assert list(got[5]) == [9 * 16, -1, -1] + [-1] * 5 and got[1][0] == 9
    fine(cache, 2)


def test_release_gives_pages_back_in_order():
    cache = paged(40, 16, 1, 64)
    rng = np.random.default_rng(5)
    lens = np.array([33, 0, 16, 100, 5, 64])
    tables, order, at = np.full((6, 8), -1), rng.permutation(40), 0
    for b, n in enumerate(lens):
        k = -(-n // 16)
        tables[b, :k] = order[at:at + k]
        at += k
    free = np.full(40, -9)
    free[:40 - at] = order[at:]
    d = [ints(x) for x in ([1, 1, 0, 1, 0, 1], lens, tables, free, [40 - at])]
    cache.release(*d)
    want = [p for b in (0, 3, 5) for p in tables[b] if p >= 0]
    n = 40 - at
    assert d[4].item() == n + len(want)
    assert list(d[3][n:n + len(want)].cpu().numpy()) == want
    assert list(d[1].cpu().numpy()) == [0, 0, 16, 0, 5, 0]
    assert (d[2][[0, 1, 3, 5]] == -1).all() and (d[2][2, :1].cpu().numpy() == tables[2, :1]).all()
    fine(cache)
    # bad entries and a full list are dropped and flagged
    d = [ints(x) for x in ([1], [48], [[2, 77, 3]], [0] * 40, [39])]
    cache.release(*d)
    assert d[4].item() == 40 and d[3][39].item() == 2
    fine(cache, 2)


def test_plan_release_chain_returns_every_page():
    rng = np.random.default_rng(1)
    P, R, B = 200, 16, 12
    cache = paged(P, R, 1, 64)
    lens, tables, free, count = ints([0] * B), ints(np.full((B, 40), -1)), ints(np.arange(P)), ints([P])
    q, row = ints([0] * (B + 1)), [ints([0] * 700) for _ in range(3)]
    for step in range(30):
        cache.plan(lens, ints(rng.integers(0, 30, B)), tables, free, count, lens, count, q, *row)
        t, n = tables.cpu().numpy(), lens.cpu().numpy()
        used = [p for b in range(B) for p in t[b, :-(-n[b] // R)]]
        assert len(set(used)) == len(used) and min(used) >= 0
        assert sorted(used + list(free[:count.item()].cpu().numpy())) == list(range(P))
        cache.release(ints(rng.integers(0, 4, B) == 0), lens, tables, free, count)
    cache.release(ints([1] * B), lens, tables, free, count)
    assert sorted(free.cpu().numpy()) == list(range(P)) and count.item() == P


# ------------------------------------------------------------------------------------------------------------------
# rows in and out
# ------------------------------------------------------------------------------------------------------------------
def make_rows(rng, n, heads, hd, dtype, pad=0, scale=1.5):
    """[n, heads, hd] on the device inside a wider buffer (pad values more a row, odd starts) and its values."""
    width = heads * hd + pad
    x = torch.tensor(rng.standard_normal((n * width + pad,)) * scale, device="cuda").to(DT[dtype])
    return x[pad:].as_strided((n, heads, hd), (width, hd, 1))


def check_queries(got, x, gain, eps, cs, style, dtype):
    want = op.norm_rope(host(x), gain, eps, cs, style)
    size = np.abs(op.norm_rope(host(x), gain, eps, None, style))
    hd = size.shape[-1]
    a, b = (slice(0, hd, 2), slice(1, hd, 2)) if style == "pairs" else (slice(0, hd // 2), slice(hd // 2, hd))
    pair = np.empty_like(size)
    pair[..., a] = pair[..., b] = size[..., a] + size[..., b]
    tol = 16 * 2.0 ** -24 * pair + HALF[dtype] * np.abs(want) * 1.001 + 1e-7 * (dtype == "f16")
    assert (np.abs(host(got) - want) <= tol).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("heads,kv,hd,page,n,norm,rope,style,pad", [
    (9, 3, 64, 16, 1, True, True, "pairs", 0), (9, 3, 64, 48, 37, True, True, "halves", 3),
    (8, 2, 128, 16, 65, True, True, "halves", 0), (4, 4, 128, 64, 70, True, True, "pairs", 8),
    (5, 1, 128, 32, 33, False, True, "halves", 1), (0, 2, 64, 16, 40, False, False, "pairs", 0),
    (2, 2, 128, 16, 19, True, False, "pairs", 5), (16, 8, 128, 128, 300, True, True, "halves", 0)])
def test_append_and_read(dtype, heads, kv, hd, page, n, norm, rope, style, pad):
    rng = np.random.default_rng(heads * 100 + n)
    pages = n // page + 5
    cache = paged(pages, page, kv, hd, layers=2, fill=noise(1))
    before = cache.pool.clone()
    k, v = make_rows(rng, n, kv, hd, dtype, pad), make_rows(rng, n, kv, hd, dtype, pad, 0.6)
    q = make_rows(rng, n, heads, hd, dtype, pad) if heads else None
    q_out = torch.full((n, heads, hd), 7.0, dtype=DT[dtype], device="cuda") if heads else None
    gains = [(1 + 0.2 * rng.standard_normal(hd)).astype(np.float32) for _ in range(2)] if norm else [None, None]
    positions = rng.integers(0, 5000, n)
    from block_quantized_token_gb300 import runtime
    table = runtime.rope_table(hd, 10000.0, 5000) if rope else None
    cs = host(table)[positions] if rope else None
    # half of the rows in order from inside a page on, the others anywhere
    slots = rng.permutation(pages * page)[:n]
    m = n // 2
    start = 5
    slots[:m] = np.arange(start, start + m)
    slots[m:] = rng.permutation(np.setdiff1d(np.arange(pages * page), slots[:m]))[:n - m]
    gd = [None if g is None else torch.tensor(g, device="cuda") for g in gains]
    cache.append(1, q, k, v, ints(positions), ints(slots), q_out, q_gain=gd[0], k_gain=gd[1], eps=1e-5, rope=table,
                 rope_style=style)
    if heads:
        check_queries(q_out, q, gains[0], 1e-5, cs, style, dtype)
    want_k = op.quantize_kv_q4_0(op.norm_rope(host(k), gains[1], 1e-5, cs, style).astype(np.float32))
    want_v = op.quantize_kv_q4_0(host(v).astype(np.float32))
    out = [torch.empty((n, kv, hd), dtype=torch.float32, device="cuda") for _ in range(2)]
    cache.read(1, ints(slots), *out)
    np.testing.assert_array_equal(host(out[0]), op.dequant_kv_q4_0(*want_k))
    np.testing.assert_array_equal(host(out[1]), op.dequant_kv_q4_0(*want_v))
    # fp16 values are exact too
    half = [torch.empty((n, kv, hd), dtype=torch.float16, device="cuda") for _ in range(2)]
    cache.read(1, ints(slots), *half)
    np.testing.assert_array_equal(host(half[0]), host(out[0]))
    # nothing else of the pool moved: put the old bytes of the written rows back
    fine(cache)
    mask = written_bytes(pages, page, kv, hd, slots, layers=2, layer=1)
    np.testing.assert_array_equal(cache.pool.cpu().numpy()[~mask], before.cpu().numpy()[~mask])


def written_bytes(pages, page, kv, hd, slots, layers, layer):
    """Which bytes of the pool belong to rows `slots` of `layer`."""
    ones, none = np.full((16, hd), 15, np.uint8), np.zeros((16, hd), np.uint8)
    full, zero = np.full((16, hd // 32), -1, np.int16).view(np.float16), np.zeros((16, hd // 32), np.float16)
    mask = np.zeros((layers, pages, kv, page // 16, 18 * hd), bool)
    per_row = []
    for r in range(16):
        pick = np.arange(16)[:, None] == r
        c, d = np.where(pick, ones, none), np.where(pick, full.view(np.int16), zero.view(np.int16)).view(np.float16)
        per_row.append(op.pack_tile(c, d, c, d) != 0)
    for s in slots:
        mask[layer, s // page, :, (s % page) // 16] |= per_row[s % 16]
    return mask.reshape(-1)


@pytest.mark.parametrize("hd", [64, 128])
def test_append_special_blocks(hd):
    """Zeros, ties of sizes, saturation, subnormal values, infinities and NaN; keys with neither norm nor rotation."""
    n = 40
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((n, 1, hd)) * 3).astype(np.float32)
    x[0] = 0
    x[1, 0, 5], x[1, 0, 9] = -40, 40
    x[2, 0, 5], x[2, 0, 9] = 40, -40
    x[3] = 1e5 * np.sign(x[3])
    x[4] *= 1e-8
    x[5] *= 1e-30
    x[6, 0, 3] = np.inf
    x[7, 0, 33] = np.nan
    x[8, 0, 2], x[8, 0, 7] = -np.inf, np.nan
    x[9] = np.arange(hd) / 2 - 16  # exact halves
    cache = paged(3, 16, 1, hd, fill=noise(2))
    t = torch.tensor(x, device="cuda")
    cache.append(0, None, t, t, None, ints(np.arange(n)))
    out = [torch.empty((n, 1, hd), device="cuda") for _ in range(2)]
    cache.read(0, ints(np.arange(n)), *out)
    want = op.dequant_kv_q4_0(*op.quantize_kv_q4_0(x))
    for o in out:
        np.testing.assert_array_equal(host(o), want)
    fine(cache)


@pytest.mark.parametrize("style", ["pairs", "halves"])
def test_append_keys_next_to_borders(style):
    """Keys whose normed and rotated values fall on or next to borders between codes and between scales: equal rows
    with quarter turns give exact ties, tiny steps around them the nearest misses."""
    n, hd = 512, 128
    rng = np.random.default_rng(8)
    base = rng.integers(-8, 9, (n, 1, hd)) / 2.0
    x = (base * (1 + rng.integers(-3, 4, (n, 1, hd)) * 2.0 ** -23)).astype(np.float32)
    cs = np.zeros((4, hd // 2, 2), np.float32)
    cs[:, :, 0], cs[:, :, 1] = [[1], [0], [-1], [0]], [[0], [1], [0], [-1]]
    cache = paged(n // 16, 16, 1, hd)
    t, pos = torch.tensor(x, device="cuda"), np.arange(n) % 4
    gain = np.ones(hd, np.float32)
    cache.append(0, None, t, t, ints(pos), ints(np.arange(n)), k_gain=torch.tensor(gain, device="cuda"), eps=0.0,
                 rope=torch.tensor(cs, device="cuda"), rope_style=style)
    out = torch.empty((n, 1, hd), device="cuda")
    cache.read(0, ints(np.arange(n)), out, None)
    y = op.norm_rope(x, gain, 0.0, cs[pos], style).astype(np.float32)
    np.testing.assert_array_equal(host(out), op.dequant_kv_q4_0(*op.quantize_kv_q4_0(y)))


def test_append_skips_and_flags():
    rng = np.random.default_rng(4)
    cache = paged(4, 16, 2, 64, fill=noise(3))
    before = cache.pool.clone()
    k, q = make_rows(rng, 5, 2, 64, "f32"), make_rows(rng, 5, 4, 64, "f32")
    q_out = torch.full((5, 4, 64), 7.0, device="cuda")
    from block_quantized_token_gb300 import runtime
    table = runtime.rope_table(64, 10000.0, 10)
    cache.append(0, q, k, k, ints([0, 1, 2, 3, 4]), ints([-1] * 5), q_out, rope=table)
    assert (q_out == 7).all() and torch.equal(cache.pool, before)
    fine(cache)
    cache.append(0, q, k, k, ints([0, 1, 10, -1, 4]), ints([64, -5, 3, 4, 5]), q_out, rope=table)
    assert (q_out[:4] == 7).all() and not (q_out[4] == 7).any()
    mask = written_bytes(4, 16, 2, 64, [5], 1, 0)
    np.testing.assert_array_equal(cache.pool.cpu().numpy()[~mask], before.cpu().numpy()[~mask])
    fine(cache, 2)
    out = torch.full((3, 2, 64), 7.0, device="cuda")
    cache.read(0, ints([64, -1, 5]), out, None)
    assert (out[:2] == 7).all() and not (out[2] == 7).all()
    fine(cache, 2)


def test_append_in_place_queries():
    rng = np.random.default_rng(6)
    cache = paged(2, 16, 2, 128)
    k, q = make_rows(rng, 9, 2, 128, "bf16"), make_rows(rng, 9, 6, 128, "bf16", pad=16)
    from block_quantized_token_gb300 import runtime
    table = runtime.rope_table(128, 500000.0, 100)
    a = torch.empty((9, 6, 128), dtype=torch.bfloat16, device="cuda")
    cache.append(0, q, k, k, ints(np.arange(9)), ints(np.arange(9)), a, rope=table, rope_style="halves")
    cache.append(0, q, k, k, ints(np.arange(9)), ints(np.arange(9)), q, rope=table, rope_style="halves")
    assert torch.equal(a, q)


def test_rope_table():
    from block_quantized_token_gb300 import runtime
    n, hd, base = 100003, 64, 500000.0
    t = host(runtime.rope_table(hd, base, n))
    a = np.arange(n, dtype=np.float64)[:, None] * np.power(base, -2.0 * np.arange(hd // 2) / hd)
    # float64 angles up to 1e5 are off by at most 2^-36 (an ulp of the power, times the position); then float32
    np.testing.assert_allclose(t[..., 0], np.cos(a), rtol=2.0 ** -24, atol=2.0 ** -34)
    np.testing.assert_allclose(t[..., 1], np.sin(a), rtol=2.0 ** -24, atol=2.0 ** -34)


# ------------------------------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------------------------------
class Batch:
    """Sequences with cached rows in shuffled pages; pages and rows that belong to nobody hold noise (NaN scales)."""

    def __init__(self, lens, new, heads, kv, hd, page, dtype, seed=0, pad=0, tail=0, scale=0.0, window=0, sharp=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.new, self.heads, self.kv, self.hd = list(lens), list(new), heads, kv, hd
        self.dtype, self.window, self.page = dtype, window, page
        self.scale = scale
        blocks = [-(-max(0, n) // page) for n in lens]
        self.pages = sum(blocks) + 3
        self.cache = paged(self.pages, page, kv, hd, fill=noise(seed + 1))
        order, at = rng.permutation(self.pages), 0
        stride = max([1] + blocks) + 2
        self.tables = np.full((len(lens), stride), -1)
        for b, n in enumerate(blocks):
            self.tables[b, :n] = order[at:at + n]
            at += n
        self.k, self.v = [], []
        for b, n in enumerate(lens):
            if n <= 0:
                self.k.append(np.zeros((0, kv, hd)))
                self.v.append(np.zeros((0, kv, hd)))
                continue
            k = torch.tensor(rng.standard_normal((n, kv, hd)) * sharp, dtype=torch.float32, device="cuda")
            v = torch.tensor(rng.standard_normal((n, kv, hd)) * 0.7, dtype=torch.float32, device="cuda")
            pos = np.arange(n)
            slots = ints(self.tables[b, pos // page] * page + pos % page)
            self.cache.append(0, None, k, v, None, slots)
            out = [torch.empty_like(k) for _ in range(2)]
            self.cache.read(0, slots, *out)
            self.k.append(host(out[0]))
            self.v.append(host(out[1]))
        self.start = np.concatenate([[0], np.cumsum(new)])
        self.q = make_rows(rng, int(self.start[-1]) + tail, heads, hd, dtype, pad, 1.0)
        self.tail = tail

    def args(self):
        return ints(self.start), ints(self.lens), ints(self.tables)

    def run(self, out=None, lse=None, cache=None, q=None):
        q = self.q if q is None else q
        out = torch.full(tuple(q.shape), 7.0, dtype=q.dtype, device="cuda") if out is None else out
        lse = torch.full(tuple(q.shape[:2]), 7.0, device="cuda") if lse is None else lse
        (cache or self.cache).attention(0, q, out, *self.args(), scale=self.scale, window=self.window, lse=lse)
        return out, lse

    def check(self, out, lse, seqs=None):
        q, o, z = host(self.q), host(out), host(lse)
        scale = self.scale or self.hd ** -0.5
        for b, n in enumerate(self.lens):
            if seqs is not None and b not in seqs:
                continue
            a, e = self.start[b], self.start[b + 1]
            want, wz = op.attention(q[a:e], self.k[b], self.v[b], n, scale, self.window)
            if n <= 0 or a == e:
                assert (o[a:e] == 0).all() and (z[a:e] == -np.inf).all()
                continue
            S = abs(scale) * (np.abs(q[a:e]).sum(-1).max() * np.abs(self.k[b]).max())
            S = min(S, abs(scale) * np.linalg.norm(q[a:e], axis=-1).max() * np.linalg.norm(self.k[b], axis=-1).max())
            vmax, steps = np.abs(self.v[b]).max(), n / 16 + 64
            tol = vmax * (4 * S * 2.0 ** -19 + 2.0 ** -19 + 2 * steps * 2.0 ** -23) + HALF[self.dtype] * np.abs(want)
            if self.dtype != "f32":
                tol = tol + 2 * 2.0 ** -11 * vmax
            bad = np.abs(o[a:e] - want) > tol
            assert not bad.any(), (b, n, np.abs(o[a:e] - want).max(), tol.min())
            empty = np.isneginf(wz)
            assert (np.isneginf(z[a:e]) == empty).all() and (o[a:e][empty] == 0).all()
            zt = S * 2.0 ** -19 + steps * 2.0 ** -23 + 2.0 ** -20 + 4 * 2.0 ** -24 * np.abs(wz[~empty])
            assert (np.abs(z[a:e][~empty] - wz[~empty]) <= zt).all()
        if self.tail:
            assert (o[self.start[-1]:] == 7).all() and (z[self.start[-1]:] == 7).all()


SHAPES = [(9, 3, 64), (8, 2, 128), (4, 4, 128), (2, 2, 64), (16, 1, 128), (12, 1, 64), (20, 1, 128)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("heads,kv,hd", SHAPES)
@pytest.mark.parametrize("page", [16, 48, 128])
def test_decode(dtype, heads, kv, hd, page):
    """One token each over lengths from none to several pages, in one call."""
    lens = [1, 0, 2, 15, 16, 17, 31, 33, 64, 100, 129, 257, 500]
    b = Batch(lens, [1] * len(lens), heads, kv, hd, page, dtype, seed=heads + page, pad=4, tail=3)
    b.check(*b.run())
    fine(b.cache)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,hd,n", [(9, 3, 64, 2049), (8, 8, 128, 5000), (8, 1, 128, 9001), (4, 1, 64, 20011)])
def test_decode_one_long(dtype, heads, kv, hd, n):
    """A single sequence: its rows are split over the whole GPU and joined."""
    b = Batch([n], [1], heads, kv, hd, 16, dtype, seed=n)
    b.check(*b.run())
    fine(b.cache)


@pytest.mark.parametrize("window", [1, 5, 16, 100, 4000])
@pytest.mark.parametrize("dtype,new", [("f32", 1), ("bf16", 1), ("f32", 40), ("bf16", 40), ("f16", 150)])
def test_window(window, dtype, new):
    lens = [new, 17 + new, 300, 301, 1000]
    b = Batch(lens, [min(n, new) for n in lens], 8, 2, 128, 32, dtype, seed=window, window=window)
    b.check(*b.run())
    fine(b.cache)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("heads,kv,hd,page", [(9, 3, 64, 16), (8, 2, 128, 16), (4, 4, 128, 64), (16, 1, 64, 48),
                                              (12, 1, 128, 32)])
def test_prompts(dtype, heads, kv, hd, page):
    """Prompts, chunks on cached rows, single tokens and absent ones in one call."""
    new = [130, 1, 0, 64, 7, 33, 257, 128]
    lens = [130, 200, 50, 64, 300, 34, 600, 127]  # the last: its first token has no row at all
    b = Batch(lens, new, heads, kv, hd, page, dtype, seed=heads, pad=8, tail=2)
    b.check(*b.run())
    fine(b.cache)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_prompt(dtype):
    b = Batch([1500], [1100], 4, 1, 128, 16, dtype, seed=2)
    b.check(*b.run())
    b = Batch([900], [900], 6, 3, 64, 64, dtype, seed=3, pad=1)
    b.check(*b.run())


@pytest.mark.parametrize("dtype,new", [("f32", 1), ("bf16", 1), ("f32", 70), ("bf16", 140)])
def test_empty_rows_and_lengths_below_new(dtype, new):
    """Lengths of zero, and lengths shorter than the new tokens: the first tokens attend nothing."""
    lens = [0, new // 2, 0, new, 3 * new + 1, 0]
    b = Batch(lens, [new] * 6, 4, 2, 128, 16, dtype, seed=4)
    b.check(*b.run())
    fine(b.cache)


@pytest.mark.parametrize("dtype,new", [("f32", 1), ("f16", 1), ("bf16", 100)])
def test_sharp_and_flat_scores(dtype, new):
    """Scores that one row dominates, and a scale that makes all alike; scale below 0."""
    for scale, sharp in ((1.0, 2.0), (1e-4, 1.0), (-0.3, 1.0)):
        b = Batch([400, 90 + new], [new, new], 4, 2, 64, 16, dtype, seed=5, scale=scale, sharp=sharp)
        b.check(*b.run())


def test_wide_range_queries():
    """bf16 queries beyond fp16's range and tiny ones beside them: heads are scaled on their own."""
    for new in (1, 100):
        b = Batch([200], [new], 4, 2, 128, 16, "bf16", seed=9, scale=1e-7)
        b.q[:, 0] *= 3e6
        b.q[:, 1] *= 1e-6
        b.check(*b.run())


def test_shared_pages_and_strides():
    """Two sequences whose tables share a prefix's pages; table rows wider than needed; output into the queries."""
    b = Batch([64, 64], [1, 1], 8, 2, 128, 16, "f32", seed=7, pad=3)
    b.tables[1, :3] = b.tables[0, :3]
    b.k[1] = np.concatenate([b.k[0][:48], b.k[1][48:]])
    b.v[1] = np.concatenate([b.v[0][:48], b.v[1][48:]])
    out, lse = b.run()
    b.check(out, lse)
    q = b.q.clone()
    dense = torch.empty_like(b.q).copy_(b.q)
    b.q.copy_(q)
    o2, l2 = b.run(out=dense, q=dense, lse=torch.empty_like(lse))
    assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("dtype,new", [("f32", 1), ("bf16", 1), ("f32", 90), ("bf16", 300)])
def test_repeatable(dtype, new):
    lens = [2000 + 7 * i for i in range(5)]
    b = Batch(lens, [new] * 5, 8, 2, 128, 16, dtype, seed=11)
    first = b.run()
    for _ in range(5):
        again = b.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_nan_stays_in_its_sequence():
    """A NaN row makes its own sequence's outputs NaN; rows past a length may hold anything."""
    b = Batch([40, 40], [1, 1], 4, 2, 64, 16, "f32", seed=12)
    bad = torch.full((1, 2, 64), float("nan"), device="cuda")
    slot = ints([b.tables[0, 1] * 16 + 3])
    b.cache.append(0, None, bad, bad, None, slot)
    out, lse = b.run()
    assert torch.isnan(out[0]).all()
    b.check(out, lse, seqs=[1])


@pytest.mark.parametrize("new", [1, 100])
def test_bad_tables_and_lengths_are_flagged(new):
    b = Batch([120, 200, 150, 140], [new] * 4, 4, 2, 64, 16, "bf16" if new > 1 else "f32", seed=13)
    good = [b.tables.copy(), list(b.lens)]
    for page in (-1, b.pages, 1 << 30, -(1 << 31)):
        b.tables[1, 4] = page
        out, lse = b.run()
        fine(b.cache, 2)
        b.check(out, lse, seqs=[0, 2, 3])
        b.tables = good[0].copy()
    for n in (-1, b.tables.shape[1] * 16 + 1, 1 << 30):
        b.lens[2] = n
        out, lse = b.run()
        fine(b.cache, 2)
        b.lens = list(good[1])
        b.check(out, lse, seqs=[0, 1, 3])
    start = b.start.copy()
    b.start = np.array([0, new, 0, 3 * new, 4 * new])
    b.run()
    fine(b.cache, 2)
    b.start = np.array([0, new, 2 * new, 3 * new, 4 * new + 1])
    out, lse = b.run()
    fine(b.cache, 2)
    b.start = start
    b.check(out, lse, seqs=[0, 1, 2])
    fine(b.cache)


def test_two_handles_over_one_pool_on_two_streams():
    from block_quantized_token_gb300 import runtime
    b = Batch([3000, 2500], [1, 1], 8, 2, 128, 16, "f32", seed=14)
    other = runtime.PagedCache(1, b.pages, 16, 2, 128, pool=b.cache.pool)
    want = b.run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    args = b.args()
    torch.cuda.synchronize()
    for _ in range(10):
        for i, c in enumerate((b.cache, other)):
            with torch.cuda.stream(streams[i]):
                o, z = torch.empty(b.q.shape, device="cuda"), torch.empty(b.q.shape[:2], device="cuda")
                c.attention(0, b.q, o, *args, lse=z)
                outs[i].append((o, z))
    torch.cuda.synchronize()
    for o, z in outs[0] + outs[1]:
        assert torch.equal(o, want[0]) and torch.equal(z, want[1])


def test_captured_step_replays_with_new_lengths():
    """plan, append, read and attention captured once, replayed while lengths, pages and rows change."""
    from block_quantized_token_gb300 import runtime
    B, H, KV, hd, R, P, T = 3, 8, 2, 128, 16, 60, 8
    rng = np.random.default_rng(15)
    cache = paged(P, R, KV, hd, fill=noise(9))
    lens, new = ints([0] * B), ints([0] * B)
    tables, free, count = ints(np.full((B, 20), -1)), ints(rng.permutation(P)), ints([P])
    q_start, pos, slots, seqs = ints([0] * (B + 1)), ints([0] * T), ints([0] * T), ints([0] * T)
    qkv = torch.zeros((T, (H + 2 * KV) * hd), device="cuda")
    q, k, v = (x.unflatten(1, (-1, hd)) for x in qkv.split([H * hd, KV * hd, KV * hd], 1))
    q_out, out = torch.zeros((T, H, hd), device="cuda"), torch.zeros((T, H, hd), device="cuda")
    kv_out = [torch.zeros((T, KV, hd), device="cuda") for _ in range(2)]
    table = runtime.rope_table(hd, 10000.0, 400)

    def step():
        cache.plan(lens, new, tables, free, count, lens, count, q_start, pos, slots, seqs)
        cache.append(0, q, k, v, pos, slots, q_out, rope=table)
        cache.read(0, slots, *kv_out)
        cache.attention(0, q_out, out, q_start, lens, tables)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # no new tokens: changes nothing
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held = [([], []) for _ in range(B)]
    have = [0] * B
    for n in ([5, 1, 0], [1, 1, 1], [0, 3, 5], [1, 1, 1], [8, 0, 0], [1, 1, 1]):
        qkv.copy_(torch.tensor(rng.standard_normal(tuple(qkv.shape)), dtype=torch.float32))
        new.copy_(ints(n))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        at = 0
        for b in range(B):
            if n[b]:
                held[b][0].append(host(kv_out[0][at:at + n[b]]))
                held[b][1].append(host(kv_out[1][at:at + n[b]]))
                have[b] += n[b]
                ks, vs = (np.concatenate(x) for x in held[b])
                want, _ = op.attention(host(q_out[at:at + n[b]]), ks, vs, have[b], hd ** -0.5)
                np.testing.assert_allclose(host(out[at:at + n[b]]), want, atol=2e-4)
            at += n[b]
        assert (out[at:] == 7).all()
    assert lens.cpu().tolist() == have
    fine(cache)


# ------------------------------------------------------------------------------------------------------------------
# all of them as a decoder layer uses them
# ------------------------------------------------------------------------------------------------------------------
def test_layer_with_quantised_projections():
    """A layer's attention over several steps: projections by er_matrix_gemv (Q8_0 weights), plan, append with norms
    and rotation, attention, the output projection, release; against the same in float64 on the same cache values."""
    import oracle
    import synth
    from block_quantized_token_gb300 import er, runtime
    D, H, KV, hd, R, B, P = 256, 4, 2, 64, 16, 3, 40
    rng = np.random.default_rng(16)

    def matrix(rows, cols):
        raw = synth.quantize((0.06 * rng.standard_normal((rows, cols))).astype(np.float32), "q8_0")
        dev = torch.from_numpy(raw).cuda()
        return er.er_matrix_create(er.ER_Q8_0, rows, cols, dev.data_ptr()), oracle.dequant(raw, "q8_0", rows, cols)

    wqkv, fqkv = matrix((H + 2 * KV) * hd, D)
    wo, fo = matrix(D, H * hd)
    gains = [(1 + 0.1 * rng.standard_normal(hd)).astype(np.float32) for _ in range(2)]
    gd = [torch.tensor(g, device="cuda") for g in gains]
    cache = paged(P, R, KV, hd, fill=noise(10))
    table = runtime.rope_table(hd, 10000.0, 300)
    cs = host(table)
    lens, tables, free, count = ints([0] * B), ints(np.full((B, 12), -1)), ints(np.arange(P)), ints([P])
    T = 16
    q_start, pos, slots, seqs = ints([0] * (B + 1)), ints([0] * T), ints([0] * T), ints([0] * T)
    have, held = [0] * B, [[np.zeros((0, KV, hd)), np.zeros((0, KV, hd))] for _ in range(B)]
    try:
        for n in ([9, 0, 7], [1, 14, 1], [1, 1, 1], [12, 1, 3], [1, 1, 1]):
            t = sum(n)
            x = torch.tensor(rng.standard_normal((T, D)), dtype=torch.float32, device="cuda")
            qkv = torch.zeros((T, (H + 2 * KV) * hd), device="cuda")
            er.er_matrix_gemv(wqkv, x.data_ptr(), T, qkv.data_ptr(), torch.cuda.current_stream().cuda_stream)
            q, k, v = (y.unflatten(1, (-1, hd)) for y in qkv.split([H * hd, KV * hd, KV * hd], 1))
            cache.plan(lens, ints(n), tables, free, count, lens, count, q_start, pos, slots, seqs)
            q_out, out = torch.zeros((T, H, hd), device="cuda"), torch.zeros((T, H, hd), device="cuda")
            cache.append(0, q, k, v, pos, slots, q_out, q_gain=gd[0], k_gain=gd[1], rope=table, rope_style="halves")
            cache.attention(0, q_out, out, q_start, lens, tables)
            y = torch.zeros((T, D), device="cuda")
            er.er_matrix_gemv(wo, out.data_ptr(), T, y.data_ptr(), torch.cuda.current_stream().cuda_stream)
            kv = [torch.zeros((t, KV, hd), device="cuda") for _ in range(2)]
            cache.read(0, slots[:t].contiguous(), *kv)
            f = (host(x)[:t] @ fqkv.T).reshape(t, -1, hd)
            np.testing.assert_allclose(host(qkv)[:t].reshape(t, -1, hd), f, atol=2e-5)
            at = 0
            for b in range(B):
                if not n[b]:
                    continue
                s = slice(at, at + n[b])
                c = cs[have[b]:have[b] + n[b]]
                fq = op.norm_rope(f[s, :H], gains[0], 1e-5, c, "halves")
                for i, (rows, g) in enumerate(((host(k)[s], gains[1]), (host(v)[s], None))):
                    want = op.norm_rope(rows, g, 1e-5, c if i == 0 else None, "halves").astype(np.float32)
                    want = op.dequant_kv_q4_0(*op.quantize_kv_q4_0(want))
                    np.testing.assert_array_equal(host(kv[i])[s], want)
                    held[b][i] = np.concatenate([held[b][i], want])
                have[b] += n[b]
                o, _ = op.attention(fq, held[b][0], held[b][1], have[b], hd ** -0.5)
                np.testing.assert_allclose(host(y)[s], o.reshape(n[b], -1) @ fo.T, atol=2e-4)
                at += n[b]
            if n == [1, 14, 1]:  # the first request ends: its pages and its place are free again
                cache.release(ints([1, 0, 0]), lens, tables, free, count)
                have[0], held[0] = 0, [np.zeros((0, KV, hd)), np.zeros((0, KV, hd))]
        fine(cache)
        assert lens.cpu().tolist() == have
    finally:
        er.er_matrix_destroy(wqkv)
        er.er_matrix_destroy(wo)


# ------------------------------------------------------------------------------------------------------------------
# refusals
# ------------------------------------------------------------------------------------------------------------------
def test_refusals_leave_everything_alone():
    from block_quantized_token_gb300 import er
    cache = paged(4, 16, 2, 64, layers=2, fill=noise(20))
    before = cache.pool.clone()
    x = torch.zeros((4, 2, 64), device="cuda")
    i = ints([0, 0, 0, 0])
    p, ip = x.data_ptr(), i.data_ptr()

    def attend(**kw):
        f = dict(n_seqs=1, n_tokens=4, n_heads=2, type=er.ER_F32, table_stride=4, window=0, q=p, out=p, lse=None,
                 q_stride=128, out_stride=128, q_start=ip, lens=ip, tables=ip, scale=0.0)
        layer = kw.pop("layer", 0)
        f.update(kw)
        er.er_pages_attention(cache.handle, layer, er.er_pages_attention_args(**f))

    def append(**kw):
        f = dict(n_tokens=4, n_heads=2, type=er.ER_F32, rope_style=0, rope_positions=0, q=p, k=p, v=p, q_out=p,
                 q_stride=128, k_stride=128, v_stride=128, q_out_stride=128, q_gain=None, k_gain=None, rope=None,
                 positions=None, slots=ip, eps=1e-5)
        layer = kw.pop("layer", 0)
        f.update(kw)
        er.er_pages_append(cache.handle, layer, er.er_pages_append_args(**f))

    def plan(**kw):
        f = dict(n_seqs=1, max_tokens=4, table_stride=4, lens=ip, new_=ip, free=ip, free_count=ip, tables=ip, lens_out=ip,
                 free_count_out=ip, q_start=ip, positions=ip, slots=ip, seqs=ip)
        f.update(kw)
        er.er_pages_plan(cache.handle, er.er_pages_plan_args(**f))

    bad = [(attend, kw) for kw in (
        dict(layer=2), dict(layer=-1), dict(type=er.ER_Q4_0), dict(n_seqs=0), dict(n_seqs=1025), dict(n_tokens=-1),
        dict(table_stride=0), dict(window=-1), dict(n_heads=3), dict(n_heads=0), dict(n_heads=130), dict(q=None),
        dict(out=None), dict(q_start=None), dict(lens=None), dict(tables=None), dict(q_stride=127), dict(out_stride=64),
        dict(scale=float("nan")), dict(scale=float("inf")), dict(q=p + 2), dict(lse=p + 2), dict(out_stride=256))]
    bad += [(append, kw) for kw in (
        dict(layer=2), dict(type=er.ER_Q8_0), dict(n_tokens=-1), dict(k=None), dict(v=None), dict(slots=None),
        dict(q=None), dict(q_out=None), dict(n_heads=0), dict(rope_style=2), dict(rope=p), dict(rope=p, positions=ip),
        dict(rope=p + 4, positions=ip, rope_positions=1), dict(eps=-1.0), dict(eps=float("nan")), dict(q_stride=64),
        dict(k_stride=127), dict(v_stride=0), dict(k=p + 1), dict(q_out_stride=256))]
    bad += [(plan, kw) for kw in (
        dict(n_seqs=0), dict(n_seqs=1025), dict(max_tokens=-1), dict(table_stride=0), dict(lens=None), dict(new_=None),
        dict(free=None), dict(free_count=None), dict(tables=None), dict(lens_out=None), dict(q_start=None),
        dict(slots=None))]
    bad += [(lambda **kw: er.er_pages_read(cache.handle, **kw), kw) for kw in (
        dict(layer=2, n=1, slots=ip, type=er.ER_F32, k_out=p, v_out=p), dict(layer=0, n=-1, slots=ip, type=0, k_out=p, v_out=p),
        dict(layer=0, n=1, slots=None, type=0, k_out=p, v_out=p), dict(layer=0, n=1, slots=ip, type=2, k_out=p, v_out=p),
        dict(layer=0, n=1, slots=ip, type=0, k_out=p + 2, v_out=None))]
    for call, kw in bad:
        with pytest.raises(er.ErError) as e:
            call(**kw)
        assert e.value.status == er.ER_EINVAL, (call, kw)
    # nothing to do is done
    attend(n_tokens=0)
    append(n_tokens=0)
    er.er_pages_read(cache.handle, 0, 0, None, er.ER_F32, p, p)
    er.er_pages_read(cache.handle, 0, 4, ip, er.ER_F32, None, None)
    torch.cuda.synchronize()
    assert (x == 0).all() and torch.equal(cache.pool, before)
    fine(cache)


def test_runtime_refuses_wrong_tensors():
    cache = paged(4, 16, 2, 64)
    x, i = torch.zeros((4, 2, 64), device="cuda"), ints([0] * 8)
    t = ints([[0, 0]])
    for call in (lambda: cache.append(0, None, x.cpu(), x, None, i), lambda: cache.append(0, None, x, x.half(), None, i),
                 lambda: cache.append(0, x, x, x, None, i), lambda: cache.append(0, None, x, x, None, i.long()),
                 lambda: cache.append(0, None, x.double(), x.double(), None, i),
                 lambda: cache.append(0, None, x.transpose(1, 2), x, None, i),
                 lambda: cache.append(0, None, x, x, None, i[:2]),
                 lambda: cache.attention(0, x, x[:, :, :32], i, i[:1], t),
                 lambda: cache.attention(0, x, x, i[:1], i[:1], t), lambda: cache.attention(0, x, x, i, i, t),
                 lambda: cache.attention(0, x, x.half(), i, i[:1], t), lambda: cache.read(0, i, x, None)):
        with pytest.raises(ValueError):
            call()
    from block_quantized_token_gb300 import runtime
    with pytest.raises(ValueError):
        runtime.PagedCache(1, 4, 16, 2, 64, pool=torch.zeros(10, dtype=torch.uint8, device="cuda"))


def test_handles_free_what_they_allocate():
    from block_quantized_token_gb300 import er, runtime
    n = er.er_debug_live_allocations()
    c = runtime.PagedCache(1, 4, 16, 2, 64)
    assert er.er_debug_live_allocations() > n
    c.close()
    assert er.er_debug_live_allocations() == n
    pool = torch.zeros(4 * 2 * 18 * 64, dtype=torch.uint8, device="cuda")
    i = 0
    while True:
        er.er_debug_fail_allocation(i)
        try:
            c = runtime.PagedCache(1, 4, 16, 2, 64, pool=pool)
        except er.ErError as e:
            assert e.status == er.ER_ENOMEM
            assert er.er_debug_live_allocations() == n
            i += 1
            continue
        finally:
            er.er_debug_fail_allocation(-1)
        c.close()
        break
    assert i >= 1 and er.er_debug_live_allocations() == n


# ------------------------------------------------------------------------------------------------------------------
# sizes and contents at the edges of what the header allows
# ------------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,new", [("f32", 1), ("bf16", 9), ("f32", 70), ("f16", 140)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 20])
def test_window_past_every_length(dtype, new, window):
    """The widest windows, with tokens before row 0: position - window must not wrap."""
    b = Batch([new // 2, 300, new], [new] * 3, 4, 2, 64, 16, dtype, seed=31, window=window)
    b.check(*b.run())
    fine(b.cache)


def test_lengths_next_to_2_31_are_flagged():
    from block_quantized_token_gb300 import er
    cache = paged(4, 16, 1, 64, fill=noise(32))
    stride = 1 << 28  # (the table has one entry; nothing may look further)
    one, out = ints([0]), torch.full((2, 1, 64), 7.0, device="cuda")
    for n in (2 ** 31 - 1, 2 ** 31 - 1024):
        lens, start, new = ints([n]), ints([0, 2]), ints([0])
        er.er_pages_attention(cache.handle, 0, er.er_pages_attention_args(
            1, 2, 1, er.ER_F32, stride, 0, out.data_ptr(), out.data_ptr(), None, 64, 64, start.data_ptr(),
            lens.data_ptr(), one.data_ptr(), 0.0))
        fine(cache, 2)
        lo, co, q, t = ints([-7]), ints([-7]), ints([-7, -7]), [ints([-7] * 4) for _ in range(3)]
        er.er_pages_plan(cache.handle, er.er_pages_plan_args(
            1, 4, stride, lens.data_ptr(), new.data_ptr(), one.data_ptr(), ints([1]).data_ptr(), one.data_ptr(),
            lo.data_ptr(), co.data_ptr(), q.data_ptr(), *(x.data_ptr() for x in t)))
        fine(cache, 2)
        assert lo.item() == n and co.item() == 1 and q.tolist() == [0, 0] and t[1].tolist() == [-1] * 4


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("new", [1, 5, 100])
@pytest.mark.parametrize("row", [0, 31, 130, 255, 256, 287, 290, 299])
def test_nan_values_reach_the_tokens_that_attend_them(dtype, new, row):
    """A NaN in 32 dims of one cached V row: in those dims of every token that attends it, in no token that does not; a
    single token's other dims stay as they were."""
    b = Batch([300], [new], 4, 2, 128, 16, dtype, seed=33)
    v = torch.tensor(b.v[0][row:row + 1], dtype=torch.float32, device="cuda")
    v[:, 0, 40] = float("nan")
    k = torch.tensor(b.k[0][row:row + 1], dtype=torch.float32, device="cuda")
    clean, zc = b.run()
    b.cache.append(0, None, k, v, None, ints([b.tables[0, row // 16] * 16 + row % 16]))
    out, lse = b.run()
    attends = torch.arange(300 - new, 300, device="cuda") >= row
    bad = torch.isnan(out)
    assert bad[attends][:, :2, 32:64].all() and not bad[~attends].any() and not bad[:, 2:].any()
    assert torch.equal(out[:, 2:], clean[:, 2:]) and torch.equal(lse[:, 2:], zc[:, 2:])
    if new == 1:
        assert not bad[..., :32].any() and not bad[..., 64:].any() and torch.isfinite(lse).all()
        other = [d for d in range(128) if not 32 <= d < 64]
        assert torch.equal(out[..., other], clean[..., other]) and torch.equal(lse, zc)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("row", [3, 19967, 19968, 19999, 20000, 20007, 20009])
@pytest.mark.parametrize("new", [1, 5])
def test_nan_value_in_a_long_sequence(dtype, row, new):
    """The same where warps walk several blocks of rows, the last of them not whole: before it, in it, far from it."""
    b = Batch([20010], [new], 8, 8, 128, 16, dtype, seed=42)
    k, v = (torch.tensor(x[0][row:row + 1], dtype=torch.float32, device="cuda") for x in (b.k, b.v))
    v[:, :, 100] = float("nan")
    b.cache.append(0, None, k, v, None, ints([b.tables[0, row // 16] * 16 + row % 16]))
    bad = torch.isnan(b.run()[0])
    attends = torch.arange(20010 - new, 20010, device="cuda") >= row
    assert bad[attends][..., 96:].all() and not bad[~attends].any()
    if new == 1:
        assert not bad[..., :96].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,hd,page", [(64, 1, 128, 16), (64, 1, 64, 1024), (34, 2, 64, 112), (63, 1, 128, 32)])
@pytest.mark.parametrize("new", [[1], [1, 1, 0, 1], [3, 0, 1, 40]])
def test_wide_groups_and_large_pages(dtype, heads, kv, hd, page, new):
    b = Batch([1 + 700 * i for i in range(1, len(new) + 1)], new, heads, kv, hd, page, dtype, seed=34, tail=2)
    b.check(*b.run())
    fine(b.cache)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mixed", [False, True])
def test_many_sequences(dtype, mixed):
    """More sequences than one launch lists, single tokens alone and among prompts."""
    rng = np.random.default_rng(35)
    lens, new = rng.integers(0, 60, 700), np.ones(700, int)
    new[::7] = 0
    if mixed:
        for i in (0, 31, 32, 511, 512, 690):
            lens[i], new[i] = 150 + i % 90, 40 + i % 70
    b = Batch(lens.tolist(), new.tolist(), 4, 2, 64, 16, dtype, seed=36, tail=3)
    b.check(*b.run())
    fine(b.cache)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("new", [1, 100])
def test_rows_at_odd_addresses(dtype, new):
    """Queries and outputs one value past an aligned address, and a stride of an odd number of values."""
    b = Batch([333, 40 + new], [new, new], 4, 2, 64, 16, dtype, seed=37)
    out, lse = b.run()
    n = b.q.shape[0]
    def odd(fill):
        flat = torch.full((n * 261 + 1,), fill, dtype=b.q.dtype, device="cuda")
        return flat, flat[1:].view(n, 261)[:, :256].view(n, 4, 64)
    (_, q), (flat, o) = odd(0.0), odd(7.0)
    q.copy_(b.q)
    o2, l2 = b.run(out=o, q=q)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    assert flat[0] == 7 and (flat[1:].view(n, 261)[:, 256:] == 7).all()
    o3, l3 = b.run(out=q, q=q)  # over the queries themselves
    assert torch.equal(o3, out) and torch.equal(l3, lse)


@pytest.mark.parametrize("dtype,new", [("f32", 1), ("bf16", 1), ("f32", 50), ("bf16", 100)])
def test_window_leaves_earlier_pages_unread(dtype, new):
    """Pages before every token's window may be given back: their entries are not looked at.  Another layer's rows."""
    b = Batch([700, 900], [new, new], 4, 2, 64, 16, dtype, seed=38, window=100)
    first = b.run()
    b.check(*first)
    for i, n in enumerate(b.lens):
        b.tables[i, :(n - new - 100 + 1) // 16] = -1
    again = b.run()
    fine(b.cache)
    three = paged(b.pages, 16, 2, 64, layers=3, fill=noise(39))
    three.pool.view(3, -1)[2].copy_(b.cache.pool)
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    three.attention(2, b.q, out, *b.args(), window=100, lse=lse)
    for o, z in (again, (out, lse)):
        assert torch.equal(o, first[0]) and torch.equal(z, first[1])
    with pytest.raises(Exception):
        three.attention(3, b.q, out, *b.args())


def test_two_graphs_of_one_handle_in_turn():
    """A decode step and a prompt captured apart; replayed one after the other they share the handle's scratch."""
    small, large = (Batch(l, n, 8, 2, 128, 16, "bf16", seed=40) for l, n in (([5000, 90], [1, 1]), ([700, 300], [200, 1])))
    want, graphs = [small.run(), large.run()], []
    pool = torch.cat([small.cache.pool, large.cache.pool])
    cache = paged(small.pages + large.pages, 16, 2, 128, pool=pool)
    large.tables = np.where(large.tables >= 0, large.tables + small.pages, large.tables)
    side = torch.cuda.Stream()
    for b in (small, large):
        args = b.args()
        out, lse = torch.zeros_like(b.q), torch.zeros(tuple(b.q.shape[:2]), device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            cache.attention(0, b.q, out, *args, lse=lse)
        graphs.append((g, out, lse, args))
    for _ in range(4):
        for (g, out, lse, _), w in zip(graphs, want):
            out.zero_()
            g.replay()
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])
    fine(cache)


def test_more_refusals():
    from block_quantized_token_gb300 import er
    cache = paged(4, 16, 2, 64, fill=noise(41))
    x, i = torch.zeros((4, 2, 64), device="cuda"), ints([0] * 8)
    p, ip = x.data_ptr(), i.data_ptr()
    base = dict(n_seqs=1, n_tokens=4, n_heads=2, type=er.ER_F32, table_stride=4, window=0, q=p, out=p, lse=None,
                q_stride=128, out_stride=128, q_start=ip, lens=ip, tables=ip, scale=0.0)
    calls = [lambda kw=kw: er.er_pages_attention(cache.handle, 0, er.er_pages_attention_args(**{**base, **kw}))
             for kw in (dict(q_start=ip + 1), dict(lens=ip + 2), dict(tables=ip + 3), dict(n_tokens=2 ** 31 - 1),
                        dict(n_tokens=1 << 26, n_heads=128, q_stride=8192, out_stride=8192))]
    base_p = dict(n_seqs=1, max_tokens=4, table_stride=4, lens=ip, new_=ip, free=ip, free_count=ip, tables=ip, lens_out=ip,
                  free_count_out=ip, q_start=ip, positions=ip, slots=ip, seqs=ip)
    calls += [lambda n=n: er.er_pages_plan(cache.handle, er.er_pages_plan_args(**{**base_p, n: ip + 2}))
              for n in ("lens", "new_", "free", "free_count", "tables", "lens_out", "free_count_out", "q_start", "positions",
                        "slots", "seqs")]
    base_a = dict(n_tokens=4, n_heads=2, type=er.ER_F32, rope_style=0, rope_positions=0, q=p, k=p, v=p, q_out=p,
                  q_stride=128, k_stride=128, v_stride=128, q_out_stride=128, q_gain=None, k_gain=None, rope=None,
                  positions=None, slots=ip, eps=1e-5)
    calls += [lambda kw=kw: er.er_pages_append(cache.handle, 0, er.er_pages_append_args(**{**base_a, **kw}))
              for kw in (dict(slots=ip + 1), dict(q_gain=p + 2), dict(k_gain=p + 1),
                         dict(rope=p, rope_positions=1, positions=ip + 2))]
    calls += [lambda: er.er_pages_read(cache.handle, 0, 1, ip + 2, er.ER_F32, p, p),
              lambda: er.er_pages_release(cache.handle, 1, ip + 1, ip, ip, 1, ip, ip),
              lambda: er.er_pages_release(cache.handle, 1, ip, ip, ip + 2, 1, ip, ip),
              lambda: er.er_pages_release(cache.handle, 0, ip, ip, ip, 1, ip, ip),
              lambda: er.er_pages_release(cache.handle, 1, ip, ip, ip, 0, ip, ip)]
    for call in calls:
        with pytest.raises(er.ErError) as e:
            call()
        assert e.value.status == er.ER_EINVAL
    torch.cuda.synchronize()
    assert (x == 0).all() and (i == 0).all()
    fine(cache)


@pytest.mark.parametrize("dtype,new", [("f32", 1), ("bf16", 1), ("f32", 60), ("bf16", 200)])
def test_pool_past_4_gib(dtype, new):
    """Pages and a layer whose bytes start past 32 bits: rows written, read and attended there as in a small pool."""
    b = Batch([500, 260], [new, new], 8, 8, 128, 128, dtype, seed=43)
    want, wz = b.run()
    page_bytes = b.cache.pool.numel() // b.pages
    pages = (9 << 29) // page_bytes  # 4.5 GiB a layer
    big = paged(pages, 128, 8, 128, layers=2)
    high = pages - b.pages
    big.pool.view(2, pages, page_bytes)[1, high:].copy_(b.cache.pool.view(b.pages, page_bytes))
    tables = ints(np.where(b.tables >= 0, b.tables + high, b.tables))
    out, lse = torch.empty_like(want), torch.empty_like(wz)
    big.attention(1, b.q, out, ints(b.start), ints(b.lens), tables, lse=lse)
    assert torch.equal(out, want) and torch.equal(lse, wz)
    rng = np.random.default_rng(44)
    k, v = (make_rows(rng, 40, 8, 128, dtype) for _ in range(2))
    slots = ints((pages - 1) * 128 + np.arange(60, 100))
    big.append(1, None, k, v, None, slots)
    small = paged(1, 128, 8, 128)
    small.append(0, None, k, v, None, ints(np.arange(60, 100)))
    got = [torch.empty((40, 8, 128), dtype=k.dtype, device="cuda") for _ in range(4)]
    big.read(1, slots, *got[:2])
    small.read(0, ints(np.arange(60, 100)), *got[2:])
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])
    fine(big)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_among_many_idle_sequences(dtype):
    """Fewer tokens than sequences, all of them one sequence's; and a padded batch whose rows end far before its tensors."""
    b = Batch([40] * 75 + [300] + [0] * 74, [0] * 75 + [100] + [0] * 74, 16, 2, 64, 32, dtype, seed=45, tail=30)
    b.check(*b.run())
    b = Batch([70, 130, 9], [70, 3, 0], 4, 2, 128, 16, dtype, seed=46, tail=500)
    b.check(*b.run())
    fine(b.cache)
