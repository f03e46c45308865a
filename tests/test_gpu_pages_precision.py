"""How near paged attention (er_pages_attention) comes to the 64-bit result, row by row, on inputs made to show a part that
works in fewer bits than it should.

Bounds, u = 2^-24.  A = scale sum |q||k| of a (token, row) pair.
* a score is off by at most 2^-19 A (hd / 16 products of 16 terms, each truncated at 2^-23, the scale and the exponential's
  argument; fp32 queries enter as two halves, 2^-22 of the query row's largest value, which these inputs keep below that);
* a probability by its score, 2^-21 of its exponential, 2^-21 of its two halves, relative to itself, and 2^-32 of the largest
  (fp16's smallest step against p >= 2^7);
* o and l are sums of N / 16 + 64 products of 16 terms at most (64: states joined and rescaled), each truncated at 2^-23.
      |out - exact| <= W (2 e + 2 (N / 16 + 64) 2^-23) + N 2^-32 vmax + half a step of the output's type there,
  W = sum w |v|, e = 2^-19 max A + 2^-20.  lse: 2^-19 max A + (N / 16 + 64) 2^-23 + 2^-20 + 4 u |lse|.
"""

from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from test_gpu_pages import Batch, fine, host, ints  # noqa: E402

BITS = {"f32": 24, "f16": 11, "bf16": 8}  # significant bits
LEAST = {"f32": -150, "f16": -25, "bf16": -134}  # exponent of half the smallest step


def half_step(x, dtype):
    """Half a step of the type at sizes x."""
    e = np.floor(np.log2(np.maximum(x, 1e-300)))
    return 2.0 ** np.maximum(e - BITS[dtype], LEAST[dtype])


def rewrite(b, seq, k, v):
    """Puts new rows into a sequence's slots and reads back what the cache holds of them."""
    n = b.lens[seq]
    pos = np.arange(n)
    slots = ints(b.tables[seq, pos // b.page] * b.page + pos % b.page)
    k, v = (torch.tensor(x, dtype=torch.float32, device="cuda") for x in (k, v))
    b.cache.append(0, None, k, v, None, slots)
    out = [torch.empty_like(k) for _ in range(2)]
    b.cache.read(0, slots, *out)
    b.k[seq], b.v[seq] = host(out[0]), host(out[1])


def check(b, out, lse):
    q, o, z = host(b.q), host(out), host(lse)
    scale, group = b.scale or b.hd ** -0.5, b.heads // b.kv
    for s, n in enumerate(b.lens):
        a, e = b.start[s], b.start[s + 1]
        p = np.arange(n - (e - a), n)
        seen = np.arange(n)[None] <= p[:, None]
        none = p < 0  # tokens before the first row
        steps = n / 16 + 64
        for h in range(b.heads):
            k, v = b.k[s][:, h // group], b.v[s][:, h // group]
            x = np.where(seen, scale * (q[a:e, h] @ k.T), -np.inf)
            top = x.max(-1, keepdims=True)
            w = np.exp(x - np.where(none[:, None], 0, top))
            total = np.where(none[:, None], 1, w.sum(-1, keepdims=True))
            want, wz = w @ v / total, (top + np.log(total))[:, 0]
            A = np.where(seen, abs(scale) * (np.abs(q[a:e, h]) @ np.abs(k).T), 0).max(-1)
            W = w @ np.abs(v) / total
            err = W * (2 * (2.0 ** -19 * A + 2.0 ** -20) + 2 * steps * 2.0 ** -23)[:, None] + n * 2.0 ** -32 * np.abs(v).max()
            off = np.abs(o[a:e, h] - want) - err - half_step(np.abs(want) + err, b.dtype)
            assert (off <= 0).all(), (s, h, off.max(), err.max())
            zt = 2.0 ** -19 * A + steps * 2.0 ** -23 + 2.0 ** -20 + 4 * 2.0 ** -24 * np.abs(np.where(none, 0, wz))
            assert (np.isneginf(z[a:e, h]) == none).all() and (o[a:e, h][none] == 0).all()
            miss = np.abs(z[a:e, h][~none] - wz[~none])
            assert (miss <= zt[~none]).all(), (s, h, miss.max(), zt.max())
    fine(b.cache)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("heads,kv,hd", [(8, 2, 128), (9, 3, 64)])
@pytest.mark.parametrize("new", [1, 3, 100])
def test_blocks_of_one_large_value(dtype, heads, kv, hd, new):
    """Keys with a value in each block far above its others, where the queries have nothing: the scores are sums of small
    code steps or none, and the size of the block's scale must not show in them."""
    rng = np.random.default_rng(50 + new)
    b = Batch([300, 170], [new, new], heads, kv, hd, 16, dtype, seed=50)
    for s, small in enumerate((3.0, 10.0)):  # below half a code's step of 100 / 8: all zeros; about one step
        n = b.lens[s]
        k = rng.uniform(-small, small, (n, kv, hd))
        k[..., 7::32] = 100.0
        rewrite(b, s, k, rng.standard_normal((n, kv, hd)))
    b.q *= 3
    b.q[..., 7::32] = 0
    check(b, *b.run())


@pytest.mark.parametrize("dtype,new", [("f16", 1), ("bf16", 1), ("f16", 100), ("bf16", 100)])
def test_small_queries_beside_a_large_one(dtype, new):
    """16-bit queries enter exactly: one value of a row is 2^20 times the others and meets keys of zero."""
    rng = np.random.default_rng(60)
    b = Batch([250], [new], 8, 2, 128, 16, dtype, seed=51, scale=2.0 ** 17)
    k = rng.standard_normal((250, 2, 128))
    k[..., :32] = 0
    rewrite(b, 0, k, rng.standard_normal((250, 2, 128)))
    b.q *= 2.0 ** -20
    b.q[..., 5] = 1.0
    check(b, *b.run())


@pytest.mark.parametrize("dtype,new", [("f32", 1), ("f16", 1), ("bf16", 1), ("f32", 100), ("f16", 100), ("bf16", 100), ("f16", 300)])
@pytest.mark.parametrize("heads,kv,hd", [(8, 2, 128), (8, 4, 64)])
def test_probabilities_all_alike(dtype, new, heads, kv, hd):
    """One row scores above all others, which score the same: whatever a probability loses on its way to the values' product
    is the same in every row and does not average out."""
    rng = np.random.default_rng(70)
    for scale in (0.02, 0.031):
        b = Batch([400, 130], [new, new], heads, kv, hd, 16, dtype, seed=52, scale=scale)
        for s, n in enumerate(b.lens):
            k = np.full((n, kv, hd), 0.5)
            k[0] = 1.0
            rewrite(b, s, k, rng.uniform(0.5, 1.0, (n, kv, hd)))
        b.q.copy_(torch.tensor(rng.uniform(0.5, 2.0, tuple(b.q.shape)), device="cuda"))
        check(b, *b.run())
