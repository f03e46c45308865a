"""Float64 oracle of the paged 4-bit K/V cache: its quantiser, the pool's bytes, block tables, rows and attention
(test infrastructure; see package doc).  Written from the statement in include/er_pages.h: numpy, loops, no
sharing with the library."""

from __future__ import annotations

import numpy as np

D_MAX = 2720.0


def bf16(x: np.ndarray) -> np.ndarray:
    """float32 -> the nearest value of 8 significant bits (ties to even), as float32."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def quantize_kv_q4_0(x) -> tuple[np.ndarray, np.ndarray]:
    """float32 [..., n] -> (d fp16 [..., n / 32], c uint8 [..., n])."""
    x = np.asarray(x, np.float32)
    xb = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    bits = xb.view(np.uint32) & 0x7FFFFFFF  # sizes order as their bits, NaN last
    m = np.take_along_axis(xb, bits.argmax(-1)[..., None], -1)[..., 0]
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        d = np.clip(bf16(m * np.float32(-0.125)), -D_MAX, D_MAX).astype(np.float16)
        r = (xb / d.astype(np.float32)[..., None]).astype(np.float32).astype(np.float64)
        c = np.clip(np.sign(r) * np.floor(np.abs(r) + 0.5) + 8, 0, 15)
    zero = (d == 0) | np.isnan(d)
    return d, np.where(zero[..., None], 8, c).astype(np.uint8).reshape(x.shape)


def dequant_kv_q4_0(d, c) -> np.ndarray:
    c = np.asarray(c, np.float64)
    return ((c.reshape(c.shape[:-1] + (-1, 32)) - 8) * np.asarray(d, np.float64)[..., None]).reshape(c.shape)


def pack_tile(kc, kd, vc, vd) -> np.ndarray:
    """16 rows' codes [16, hd] and scales [16, hd / 32] of K and V -> the tile's 18 hd bytes, place by place."""
    hd = kc.shape[1]
    nb = hd // 32
    k = np.zeros((16, hd // 8), np.uint32)
    v = np.zeros((hd // 64, 8, 4, 4), np.uint32)
    vs = np.zeros((4, nb, 2, 2), np.float16)
    for r in range(16):
        t, e, i = (r % 8) // 2, r % 2, r // 8
        for dim in range(hd):
            b, j = dim // 32, dim % 32
            k[r, (j // 8) * nb + b] |= np.uint32(int(kc[r, dim]) << (4 * ((j % 8) // 2) + 16 * (j % 2)))
            q, u, g, high = dim // 64, (dim % 64) // 16, dim % 8, (dim // 8) % 2
            v[q, g, t, u] |= np.uint32(int(vc[r, dim]) << (8 * (i + 2 * e) + 4 * high))
        vs[t, :, i, e] = vd[r]
    parts = [k, np.asarray(kd, np.float16), v, vs]
    return np.concatenate([np.ascontiguousarray(p).reshape(-1).view(np.uint8) for p in parts])


def plan(lens, new, tables, free, count, max_tokens, page_rows):
    """(lens, count, tables, q_start, positions, slots, seqs, flags) after one step's plan."""
    lens, tables = [int(x) for x in lens], np.array(tables, np.int64)
    out_lens, q_start, flags = list(lens), [0], 0
    pos, slot, seq = [], [], []
    pages = toks = taken = 0
    open_ = True
    for b, (n, m) in enumerate(zip(lens, new)):
        m = int(m)
        if n < 0 or m < 0 or n + m > tables.shape[1] * page_rows:
            flags |= 2
            m = need = 0
        else:
            need = -(-(n + m) // page_rows) - -(-n // page_rows)
        pages, toks = pages + need, toks + m
        if pages > count or toks > max_tokens:
            open_ = False
        if not open_:
            flags |= 1
            m = need = 0
        have = -(-max(n, 0) // page_rows)
        for j in range(need):
            tables[b, have + j] = free[count - 1 - taken]
            taken += 1
        for p in range(n, n + m):
            pos.append(p)
            slot.append(tables[b, p // page_rows] * page_rows + p % page_rows)
            seq.append(b)
        out_lens[b] = n + m
        q_start.append(q_start[-1] + m)
    pad = max_tokens - len(pos)
    return (np.array(out_lens), count - taken, tables, np.array(q_start), np.array(pos + [0] * pad),
            np.array(slot + [-1] * pad), np.array(seq + [-1] * pad), flags)


def norm_rope(x, gain, eps, cs, style) -> np.ndarray:
    """x [n, heads, hd] normed per head and rotated by cs [n, hd / 2, 2] (either may be None), float64."""
    y = np.asarray(x, np.float64)
    hd = y.shape[-1]
    if gain is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(eps))) * np.asarray(gain, np.float64)
    if cs is None:
        return y
    c, s = (np.asarray(cs, np.float64)[:, None, :, i] for i in (0, 1))
    a, b = (slice(0, hd, 2), slice(1, hd, 2)) if style == "pairs" else (slice(0, hd // 2), slice(hd // 2, hd))
    out = np.empty_like(y)
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def attention(q, k, v, length, scale, window=0):
    """q [n, H, hd] the last n of `length` tokens over rows k, v [length, KV, hd] -> (o [n, H, hd], lse [n, H])."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, H, hd = q.shape
    o, lse = np.zeros((n, H, hd)), np.full((n, H), -np.inf)
    for i in range(n):
        p = length - n + i
        lo = max(0, p - window + 1) if window else 0
        if p < 0:
            continue
        for h in range(H):
            kv = h // (H // k.shape[1])
            s = scale * (k[lo:p + 1, kv] @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            o[i, h], lse[i, h] = e @ v[lo:p + 1, kv] / e.sum(), m + np.log(e.sum())
    return o, lse
