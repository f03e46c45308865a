"""The paged 4-bit K/V cache on the GPU: rows at the ends of the float range, waits that give up, flags between streams."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import pages as op

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from test_gpu_pages import HALF, Batch, fine, host, ints, noise, paged  # noqa: E402

LEAST = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half the smallest step of a type


@pytest.mark.parametrize("style", ["pairs", "halves"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype,sizes", [("f32", (1e-44, 1e-38, 1e-30, 1e-22, 1e-15, 1e-9, 1e9, 1e18, 1e25, 1e37)),
                                         ("bf16", (1e-38, 1e-30, 1e-22, 1e-15, 1e18, 1e30, 1e37)), ("f16", (1e-7, 1e-3, 1e4))])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-30, 1e-5])
def test_norm_of_rows_at_the_ends_of_the_range(style, hd, dtype, sizes, eps):
    """The norm takes a row's size away whatever it is: squares below fp32's smallest and above its largest number (queries: the
    latter only with an eps up to 2^-90, and zeros else).  Queries
    within 16 roundings of a pair and the output's own, keys with the codes of the float64 formula."""
    from block_quantized_token_gb300 import runtime
    rng = np.random.default_rng(80)
    n, heads, kv = 3 * len(sizes), 5, 3
    size = np.repeat(sizes, 3)[rng.permutation(n), None, None]  # neighbours of other sizes
    def rows(h):
        x = torch.tensor(np.clip(rng.standard_normal((n, h, hd)), -3, 3) * size, device="cuda")
        return x.to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype])
    q, k = rows(heads), rows(kv)
    gains = [(1 + 0.2 * rng.standard_normal(hd)).astype(np.float32) for _ in range(2)]
    gd = [torch.tensor(g, device="cuda") for g in gains]
    positions = rng.integers(0, 500, n)
    table = runtime.rope_table(hd, 10000.0, 500)
    cs = host(table)[positions]
    cache = paged(n // 16 + 1, 16, kv, hd, fill=noise(81))
    q_out = torch.empty_like(q)
    cache.append(0, q, k, k, ints(positions), ints(np.arange(n)), q_out, q_gain=gd[0], k_gain=gd[1], eps=eps, rope=table,
                 rope_style=style)
    out = torch.empty((n, kv, hd), device="cuda")
    cache.read(0, ints(np.arange(n)), out, None)
    want = op.norm_rope(host(k), gains[1], eps, cs, style).astype(np.float32)
    np.testing.assert_array_equal(host(out), op.dequant_kv_q4_0(*op.quantize_kv_q4_0(want)))
    want, flat = op.norm_rope(host(q), gains[0], eps, cs, style), np.abs(op.norm_rope(host(q), gains[0], eps, None, style))
    a, b = (slice(0, hd, 2), slice(1, hd, 2)) if style == "pairs" else (slice(0, hd // 2), slice(hd // 2, hd))
    pair = np.empty_like(flat)
    pair[..., a] = pair[..., b] = flat[..., a] + flat[..., b]
    # below fp32's smallest normal number a rounding is 2^-150 whatever the value: three of them times 1 / sqrt(mean square),
    # and the output's own
    low = 4 * 2.0 ** -150 / np.sqrt(max(eps, 2.0 ** -90)) + LEAST[dtype]
    tol = 16 * 2.0 ** -24 * pair + HALF[dtype] * np.abs(want) * 1.001 + low
    squares = (host(q) ** 2).sum(-1, keepdims=True)
    zero = (squares > 2.0 ** 127) & (eps > 2.0 ** -90)
    assert (host(q_out)[np.broadcast_to(zero & (squares > 2.0 ** 129), q.shape)] == 0).all()
    assert (np.abs(host(q_out) - want) <= tol)[np.broadcast_to(~zero, q.shape)].all()
    # over the queries themselves
    same = q.clone()
    cache.append(0, same, k, k, ints(positions), ints(np.arange(n)), same, q_gain=gd[0], k_gain=gd[1], eps=eps, rope=table,
                 rope_style=style)
    assert torch.equal(same, q_out)
    fine(cache)


def _batch(kind):
    """A call of each attention kernel: a long sequence over all CTAs, and prompts of several blocks of rows."""
    dtype, lens, new = {"decode_f32": ("f32", [9000, 70], [1, 1]), "decode_bf16": ("bf16", [9000, 70], [1, 1]),
                        "prompt_f32": ("f32", [900, 300, 40], [400, 300, 1]),
                        "prompt_bf16": ("bf16", [900, 300, 40], [400, 300, 1])}[kind]
    return Batch(lens, new, 8, 2, 128, 16, dtype, seed=90)


KINDS = ["decode_f32", "decode_bf16", "prompt_f32", "prompt_bf16"]


@pytest.mark.parametrize("kind", KINDS)
def test_shortest_wait_limit(kind):
    """Waits that give up at the first look: the result is right or flag bit 2 says that it is not, copies and products in
    flight are waited for all the same, and after er_pages_error the next call is right."""
    from block_quantized_token_gb300 import er
    b = _batch(kind)
    want, wz = b.run()
    fine(b.cache)
    er.er_set_wait_limit_ns(1)
    try:
        for _ in range(20):
            out, lse = b.run()
            _, code = b.cache.error()
            assert code in (0, 4), code
            assert code == 4 or torch.equal(out, want) and torch.equal(lse, wz)
    finally:
        er.er_set_wait_limit_ns(0)
    out, lse = b.run()
    assert torch.equal(out, want) and torch.equal(lse, wz)
    fine(b.cache)


@pytest.mark.parametrize("kind", KINDS)
def test_wait_gives_up_and_the_next_call_is_right(kind):
    """One CTA's wait runs out: every kernel returns, bit 2 is reported, and er_pages_error puts right what the CTAs that
    shared a sequence with it had counted."""
    import time

    from block_quantized_token_gb300 import er
    b = _batch(kind)
    want, wz = b.run()
    fine(b.cache)
    er.er_set_wait_limit_ns(5_000_000)
    er.er_pages_inject_wait_shortfall(b.cache.handle, 1)
    try:
        for _ in range(3):
            t0 = time.perf_counter()
            b.run()
            torch.cuda.synchronize()
            elapsed = time.perf_counter() - t0
            st, code = b.cache.error()
            assert st == er.ER_EDEVICE and code == 4, (st, code)
            assert elapsed < 0.5, f"gave up after {elapsed:.3f} s with a 5 ms limit"
    finally:
        er.er_pages_inject_wait_shortfall(b.cache.handle, 0)
        er.er_set_wait_limit_ns(0)
    for _ in range(3):
        out, lse = b.run()
        assert torch.equal(out, want) and torch.equal(lse, wz)
    fine(b.cache)


def test_shortfall_refusals():
    from block_quantized_token_gb300 import er
    cache = paged(4, 16, 2, 64)
    for handle, extra in ((cache.handle, -1), (cache.handle, 1025), (None, 0)):
        with pytest.raises(er.ErError) as e:
            er.er_pages_inject_wait_shortfall(handle, extra)
        assert e.value.status == er.ER_EINVAL


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window", [0, 161])
def test_prompt_whose_first_rows_come_late(dtype, window):
    """Copies of cached rows land in any order: every prompt's first 64 rows lie in a page far from the others, out of L2 and
    of the address cache, the rows after them close together.  Every run is the first one's."""
    n, kv, hd, page = 12, 8, 128, 64
    lens, new = [400 + 37 * i for i in range(n)], [300 + 11 * i for i in range(n)]
    b = Batch(lens, new, kv, kv, hd, page, dtype, seed=91, window=window)
    want, wz = b.run()
    b.check(want, wz, seqs=[0, n - 1])
    page_bytes = b.cache.pool.numel() // b.pages
    far = (1 << 31) // page_bytes  # 2 GiB on
    big = paged(far + n * 4099, page, kv, hd)
    pages, small = big.pool.view(-1, page_bytes), b.cache.pool.view(-1, page_bytes)
    pages[:b.pages].copy_(small)
    tables = b.tables.copy()
    for i in range(n):
        at = far + i * 4099
        pages[at].copy_(small[tables[i, 0]])
        tables[i, 0] = at
    args = ints(b.start), ints(b.lens), ints(tables)
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(want), torch.empty_like(wz)
    bad = torch.zeros((), device="cuda")
    for i in range(200):
        flush.fill_(i)
        small_rows = pages[:b.pages].sum()  # the close pages are in L2
        big.attention(0, b.q, out, *args, window=window, lse=lse)
        bad += (out != want).any() | (lse != wz).any()
    assert bad.item() == 0 and small_rows.item() >= 0
    fine(big)
