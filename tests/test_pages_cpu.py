"""The paged 4-bit K/V cache without a GPU: refusals that need no device, the oracle's own pins (quantiser, tile
bytes, plan) on hand-made cases."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import pages as op


@pytest.fixture(scope="module")
def er():
    from block_quantized_token_gb300 import build
    build.build()
    from block_quantized_token_gb300 import er as mod
    return mod


def _cfg(er, **kw):
    f = dict(n_layers=2, n_pages=10, page_rows=32, n_kv_heads=3, head_dim=64, kv_type=er.ER_Q4_0)
    f.update(kw)
    return er.er_pages_config(**f)


def test_pool_bytes(er):
    assert er.er_pages_pool_bytes(_cfg(er)) == 2 * 10 * 3 * 32 * 2 * (32 + 4)
    assert er.er_pages_pool_bytes(_cfg(er, head_dim=128)) == 2 * 10 * 3 * 32 * 2 * (64 + 8)
    # far past 32 bits
    assert er.er_pages_pool_bytes(_cfg(er, n_pages=1 << 20, page_rows=1024, head_dim=128)) == \
        2 * (1 << 20) * 3 * 1024 * 144


@pytest.mark.parametrize("field,value,status", [
    ("n_layers", 0, "ER_EINVAL"), ("n_pages", 0, "ER_EINVAL"), ("n_pages", -1, "ER_EINVAL"),
    ("page_rows", 0, "ER_EINVAL"), ("page_rows", 24, "ER_EINVAL"), ("page_rows", 2048, "ER_EINVAL"),
    ("n_kv_heads", 0, "ER_EINVAL"), ("head_dim", 96, "ER_EUNSUPPORTED"), ("head_dim", 0, "ER_EINVAL"),
    ("kv_type", 8, "ER_EUNSUPPORTED"), ("kv_type", 1, "ER_EUNSUPPORTED"), ("kv_type", 5, "ER_EINVAL"),
    ("n_pages", 1 << 27, "ER_EINVAL"), ("n_kv_heads", 1025, "ER_EINVAL"), ("n_layers", 65537, "ER_EINVAL")])
def test_config_refused(er, field, value, status):
    cfg = _cfg(er, **{field: value})
    assert er.er_pages_pool_bytes(cfg) == 0
    with pytest.raises(er.ErError) as e:
        er.er_pages_create(cfg, 4096)
    assert e.value.status == getattr(er, status)
    assert er.er_last_error()


def test_config_tiles_of_a_layer_fit_32_bits(er):
    for pages, kv in (((1 << 21) - 1, 17), (1 << 20, 32), (1 << 15, 1024)):
        cfg = _cfg(er, n_pages=pages, page_rows=1024, n_kv_heads=kv)
        assert er.er_pages_pool_bytes(cfg) == 0
        with pytest.raises(er.ErError) as e:
            er.er_pages_create(cfg, 4096)
        assert e.value.status == er.ER_EINVAL
    # the largest of all: past 32 bits everywhere, and inside 64
    assert er.er_pages_pool_bytes(_cfg(er, n_layers=65536, n_pages=(1 << 21) - 1, page_rows=1024, n_kv_heads=16, head_dim=128)) \
        == 65536 * ((1 << 21) - 1) * 64 * 16 * 18 * 128


def test_null_and_misaligned_refused(er):
    for call in (lambda: er.er_pages_create(_cfg(er), None), lambda: er.er_pages_create(_cfg(er), 4104),
                 lambda: er.er_pages_plan(None, er.er_pages_plan_args()),
                 lambda: er.er_pages_release(None, 1, 1, 1, 1, 1, 1, 1),
                 lambda: er.er_pages_append(None, 0, er.er_pages_append_args()),
                 lambda: er.er_pages_read(None, 0, 1, 1, er.ER_F32, None, None),
                 lambda: er.er_pages_attention(None, 0, er.er_pages_attention_args()),
                 lambda: er.er_pages_error(None),
                 lambda: er.er_rope_table(3, 10000.0, 1, 4096), lambda: er.er_rope_table(64, 0.0, 1, 4096),
                 lambda: er.er_rope_table(64, float("nan"), 1, 4096), lambda: er.er_rope_table(64, 1e4, -1, 4096),
                 lambda: er.er_rope_table(64, 1e4, 1, 4098)):
        with pytest.raises(er.ErError) as e:
            call()
        assert e.value.status == er.ER_EINVAL
    er.er_pages_destroy(None)


def test_quantiser_pins():
    x = np.zeros((6, 32), np.float32)
    x[1, 3] = -8.0                       # d = 1: codes 0 at the largest, halves away from zero
    x[1, 4:9] = [0.5, -0.5, 1.5, 6.5, 7.6]
    x[2, :2] = [4.0, -4.0]               # a tie of sizes: the first one's sign
    x[3, 0] = 1.0                        # d = -1/8: the largest is code 0
    x[4, 0] = 1e6                        # saturates
    x[5, 7] = np.nan
    d, c = op.quantize_kv_q4_0(x)
    assert d[0, 0] == 0 and (c[0] == 8).all()
    assert d[1, 0] == 1 and list(c[1, 3:9]) == [0, 9, 7, 10, 15, 15]
    assert d[2, 0] == -0.5 and list(c[2, :2]) == [0, 15]
    assert d[3, 0] == -0.125 and c[3, 0] == 0
    assert d[4, 0] == -2720 and op.dequant_kv_q4_0(d, c)[4, 0] == 21760
    assert np.isnan(d[5, 0]) and (c[5] == 8).all()


def test_every_value_is_fp16():
    """d has 8 significant bits, so d (c - 8) is an fp16 number, down to its smallest step."""
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((4000, 32)) * 10.0 ** rng.uniform(-9, 5, (4000, 1))).astype(np.float32)
    y = op.dequant_kv_q4_0(*op.quantize_kv_q4_0(x))
    assert (y.astype(np.float16).astype(np.float64) == y).all()
    big = np.abs(x).max(-1) > 1e-3
    ok = np.abs(x).max(-1) < 21000
    # at most half a code's step, and the last code of the side without an eighth one
    step = np.abs(x).max(-1, keepdims=True) / 8
    assert (np.abs(y - x) <= step * 1.01 + 1e-30)[big & ok].all()


@pytest.mark.parametrize("hd", [64, 128])
def test_tile_bytes(hd):
    """Hand-placed codes: a byte of V belongs to one row, a word of K to one row and 8 dims."""
    kc, vc = np.full((16, hd), 0, np.uint8), np.full((16, hd), 0, np.uint8)
    kd, vd = np.zeros((16, hd // 32), np.float16), np.zeros((16, hd // 32), np.float16)
    kc[3, 32 + 13] = 11        # b = 1, t = 1, j = 5: i = 2, e = 1
    vc[13, 16 + 8 + 5] = 9     # q = 0, u = 1, g = 5, high; row 13: t = 2, e = 1, i = 1
    kd[5, 1], vd[13, 1] = 1.0, 1.0
    tile = op.pack_tile(kc, kd, vc, vd)
    assert tile.shape == (18 * hd,)
    at = 3 * hd // 2 + 4 * (1 * (hd // 32) + 1)
    assert tile[at:at + 4].view(np.uint32)[0] == 11 << (8 + 16)
    at = 9 * hd + 4 * ((5 * 4 + 2) * 4 + 1)
    assert list(tile[at:at + 4]) == [0, 0, 0, 9 << 4]
    assert tile[8 * hd + 2 * (5 * hd // 32 + 1):][:2].view(np.float16)[0] == 1
    assert tile[17 * hd + 2 * ((2 * (hd // 32) + 1) * 4 + 2 + 1):][:2].view(np.float16)[0] == 1
    assert np.count_nonzero(tile) == 4


def test_plan_pins():
    tables = np.full((3, 4), -1)
    tables[0, :2] = [7, 5]
    lens, count, t, q, pos, slot, seq, flags = op.plan([20, 0, 3], [1, 17, -1], tables, [9, 8, 6], 3, 20, 16)
    assert list(lens) == [21, 17, 3] and count == 1 and list(q) == [0, 1, 18, 18] and flags == 2
    assert list(t[1]) == [6, 8, -1, -1] and slot[0] == 5 * 16 + 4 and slot[17] == 8 * 16 and list(slot[18:]) == [-1, -1]
    # the second does not fit any more: it and what follows get nothing
    lens, count, t, q, pos, slot, seq, flags = op.plan([0, 0, 0], [16, 17, 1], tables, [9, 8], 2, 64, 16)
    assert list(lens) == [16, 0, 0] and flags == 1 and count == 1
