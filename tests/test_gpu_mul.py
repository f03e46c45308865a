"""er_matrix_mul and er_adapters_* on the GPU against the float64 oracle (oracle/requests.py).

Tolerances, S = sum |w x| of an output's terms, h = half a step of the output type (2^-24, 2^-11, 2^-8), n = steps of 64
columns:
* Weights enter exactly, 16-bit rows too; fp32 rows as two fp16 halves, 2^-22 of a value, and the product of the two lo
  halves, 2^-22 of a term at most, is left out: 2^-21 S.
* The tensor cores add 16 products at a time to a running sum of at most S, cut off at 2^-23 of it: 8 such additions a
  step (fp32: 12), all n steps where the sum stays in tensor memory: 8 n 2^-23 S.  fp32 starts anew after two steps and adds up
  to nearest: 24 * 2^-23 S + n 2^-24 S.  Joining at most 152 CTAs' sums: 152 * 2^-24 S at most.
* Up to 16 tokens: sums of blocks of 32 in the tensor cores (fp32: 4 additions), two blocks a step, each added to nearest; 16
  warps' sums and at most 152 slices' joined: (8 n + n + 84) 2^-23 S.
      |y - exact| <= (12 n + 100) 2^-23 S + 2^-21 S + h |exact|   covers all.
* Adapters, T = sum |scale B A x|: v is an fp32 sum of K products in some order of at most K / 16 + 64 additions 2^-23 each;
  it enters as two bf16 pieces (2^-16 with what is left out), for fp32 as three (2^-23), or in fp32; r products are added:
      (K / 16 + 64 + r + 16) 2^-23 T + (2^-16 or 2^-22) T.
"""

from __future__ import annotations

import math

import numpy as np
import pytest

import oracle
import synth
from oracle import requests as orq

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def host(t):
    return t.detach().cpu().double().numpy()


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Case:
    """A matrix of seeded weights, adapters of seeded ranks, and what the oracle makes of rows."""

    def __init__(self, w_type, rows, cols, seed=0, ranks=(), adapter_type="bf16", slots=None, max_rank=None, weights=None):
        from block_quantized_token_gb300 import runtime
        self.rng = rng = np.random.default_rng([rows, cols, seed])
        w = weights if weights is not None else (rng.standard_normal((rows, cols)) * 0.05).astype(np.float32)
        raw = synth.quantize(w, w_type)
        self.rows, self.cols = rows, cols
        self.w = oracle.dequant(raw, w_type, rows, cols)
        self.m = runtime.Matrix(w_type, rows, cols, torch.from_numpy(raw).cuda())
        self.ad, self.known = None, {}
        self.at = DT[adapter_type]
        if ranks:
            self.ad = runtime.Adapters(rows, cols, slots or len(ranks), max_rank or max(ranks), self.at)
            for i, r in enumerate(ranks):
                self.put(i, r)

    def put(self, slot, rank, scale=None):
        rng = self.rng
        scale = float(rng.uniform(0.5, 2.0)) if scale is None else scale
        a = torch.tensor(rng.standard_normal((rank, self.cols)) / math.sqrt(self.cols)).to(self.at).cuda()
        b = torch.tensor(rng.standard_normal((self.rows, rank)) * 0.3).to(self.at).cuda()
        self.ad.set(slot, a, b, scale)
        self.known[slot] = (float(np.float32(scale)), host(a), host(b))

    def rows_of(self, n, dtype, size=1.0):
        return torch.tensor(self.rng.standard_normal((n, self.cols)) * size).to(DT[dtype]).cuda()

    def check(self, x, out, dtype, ids=None, rows=slice(None)):
        x, out = host(x)[rows], host(out)[rows]
        ids = None if ids is None else np.asarray(ids)[rows]
        y, (s, t) = orq.product(x, self.w, ids, self.known)
        n, r = -(-self.cols // 64), max((a.shape[0] for _, a, _ in self.known.values()), default=0)
        tol = ((12 * n + 100) * 2.0 ** -23 + 2.0 ** -21) * s + HALF[dtype] * np.abs(y) + 1e-30
        tol += ((self.cols / 16 + 80 + r) * 2.0 ** -23 + (2.0 ** -22 if dtype == "f32" else 2.0 ** -16)) * t
        bad = ~(np.abs(out - y) <= tol)
        assert not bad.any(), (int(bad.sum()), float((np.abs(out - y) / tol).max()), np.argwhere(bad)[:4])
        return y

    def fine(self, want=0):
        _, code = self.m.error()
        assert code == want, code

    def run(self, x, dtype, ids=None, **kw):
        out = torch.full((x.shape[0], self.rows), float("nan"), dtype=DT[dtype], device="cuda")
        self.m.mul(x, out, adapters=self.ad if ids is not None else None, ids=None if ids is None else ints(ids), **kw)
        return out


# tokens at every change of tile: 16 (adapters' two forms), 64 (warps), 128 (where sums lie), 256 (tiles)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("w_type,rows,cols", [("q8_0", 17, 32), ("q4_0", 130, 96), ("q8_0", 576, 576), ("q4_0", 1040, 1088)])
def test_products(w_type, rows, cols, dtype):
    c = Case(w_type, rows, cols)
    for n in (1, 2, 7, 16, 17, 33, 64, 65, 128, 129, 200, 256, 257, 300, 513):
        x = c.rows_of(n, dtype)
        out = c.run(x, dtype)
        c.check(x, out, dtype)
        assert torch.equal(out, c.run(x, dtype)), n
    c.fine()


@pytest.mark.parametrize("adapter_type", ["bf16", "f16"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_adapters(dtype, adapter_type):
    """Every form: few tokens, steps of their own, more kinds than those hold; ranks of odd sizes, tokens without any."""
    c = Case("q8_0", 200, 480, ranks=[1, 16, 33, 100, 8, 64, 128, 5], adapter_type=adapter_type)
    for n in (1, 5, 16, 17, 40, 64, 65, 128, 129, 260, 400):
        for pick in ([0], [2, -1], list(range(-1, 8)), [3, 3, 3, 6]):
            ids = c.rng.choice(pick, n)
            x = c.rows_of(n, dtype)
            out = c.run(x, dtype, ids)
            c.check(x, out, dtype, ids)
            assert torch.equal(out, c.run(x, dtype, ids)), (n, pick)
    c.fine()


@pytest.mark.parametrize("n", [12, 50, 120, 300])
def test_a_token_s_result_does_not_depend_on_its_neighbours_adapters(n):
    c = Case("q8_0", 96, 256, ranks=[16, 16, 48])
    x = c.rows_of(n, "f32")
    ids = np.full(n, -1)
    plain = c.run(x, "f32")
    ids[n // 2] = 2
    out = c.run(x, "f32", ids)
    others = np.arange(n) != n // 2
    assert torch.equal(out[others], plain[others]) and not torch.equal(out[n // 2], plain[n // 2])
    c.check(x, out, "f32", ids)


def test_wide_and_long():
    """Several tiles a CTA and shared ones, the widest products of the 8B shape."""
    c = Case("q8_0", 4096, 14336, ranks=[16, 64])
    for n, dtype in ((16, "bf16"), (700, "bf16"), (130, "f32")):
        ids = c.rng.integers(-1, 2, n)
        x = c.rows_of(n, dtype)
        c.check(x, c.run(x, dtype, ids), dtype, ids, rows=np.r_[0, 1, n // 2, n - 1])
    c.fine()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("w_type,rows,cols", [("q8_0", 70, 14336), ("q4_0", 1000, 4992), ("q8_0", 5000, 2560), ("q8_0", 33, 28672)])
def test_few_tokens_of_wide_matrices(w_type, rows, cols, dtype):
    """Columns in one slice and in several, warps without units, pairs of row groups that are not whole."""
    c = Case(w_type, rows, cols, ranks=[16, 40, 7])
    for n in (1, 3, 8, 9, 16):
        x, ids = c.rows_of(n, dtype), c.rng.integers(-1, 3, n)
        c.check(x, c.run(x, dtype), dtype)
        out = c.run(x, dtype, ids)
        c.check(x, out, dtype, ids)
        assert torch.equal(out, c.run(x, dtype, ids)), n
    c.fine()


def test_many_rows():
    c = Case("q4_0", 49152, 576)
    for n, dtype in ((1, "f32"), (61, "f16"), (300, "bf16")):
        x = c.rows_of(n, dtype)
        c.check(x, c.run(x, dtype), dtype, rows=np.r_[0, n - 1])
    c.fine()


def test_agrees_with_the_matrix_vector_product():
    from block_quantized_token_gb300 import er
    c = Case("q8_0", 1000, 1536)
    x = c.rows_of(16, "f32")
    want = torch.empty((16, 1000), device="cuda")
    er.er_matrix_gemv(c.m.handle, x.data_ptr(), 16, want.data_ptr(), torch.cuda.current_stream().cuda_stream)
    c.check(x, want, "f32")
    c.check(x, c.run(x, "f32"), "f32")


# ------------------------------------------------------------------------------------------------------------------
# values
# ------------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("n", [3, 40, 100, 200])
def test_scales_of_every_size(n):
    """Rows of W and of x whose sizes span what their types hold: each output is as near as its own terms allow."""
    rng = np.random.default_rng(5)
    w = (rng.standard_normal((150, 256)) * 2.0 ** rng.integers(-12, 13, (150, 1))).astype(np.float32)
    w[7] = 0
    w[:, 32:64] *= 2.0 ** -10  # a block far below its row's others
    c = Case("q8_0", 150, 256, weights=w, ranks=[16])
    for dtype, low, high in (("f32", -90, 90), ("bf16", -90, 90), ("f16", -8, 8)):
        x = c.rng.standard_normal((n, 256)) * 2.0 ** c.rng.integers(low, high, (n, 1))
        x[n // 2] = 0
        x = torch.tensor(x).to(DT[dtype]).cuda()
        ids = c.rng.integers(-1, 1, n)
        big = dtype == "f16"  # (large fp16 results pass the type's largest)
        out = c.run(x, dtype, ids)
        y, (s, t) = orq.product(host(x), c.w, ids, c.known)
        tol = ((12 * 4 + 100) * 2.0 ** -23 + 2.0 ** -20) * s + HALF[dtype] * np.abs(y) + 2.0 ** -15 * t + (2.0 ** -25 if big else 0)
        got = host(out)
        held = np.abs(y) < 60000 if big else np.ones_like(y, bool)
        assert (np.abs(got - y) <= tol)[held].all()
        assert (got[n // 2] == 0).all() and ((got[:, 7] == 0) | (np.asarray(ids) == 0)).all()
    c.fine()


@pytest.mark.parametrize("n", [5, 40, 100, 300])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_next_to_the_largest_number(n, dtype):
    """Outputs that the type holds, of rows up to 2^126: no sum on the way leaves float32's range."""
    rng = np.random.default_rng(7)
    c = Case("q8_0", 140, 1024, ranks=[16, 20], weights=(rng.standard_normal((140, 1024)) * 2.0 ** -20).astype(np.float32))
    for i, (scale, a, b) in list(c.known.items()):
        a, b = (torch.tensor(z).to(c.at).cuda() for z in (a * 2.0 ** -12, b))
        c.ad.set(i, a, b, scale)
        c.known[i] = (scale, host(a), host(b))
    x = c.rng.uniform(0.5, 1.0, (n, 1024)) * 2.0 ** c.rng.choice([0, 100, 126], (n, 1))
    x = torch.tensor(x).to(DT[dtype]).cuda()
    ids = c.rng.integers(-1, 2, n)
    c.check(x, c.run(x, dtype, ids), dtype, ids)
    c.fine()


@pytest.mark.parametrize("n", [5, 40, 100, 300])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinities_and_nan_stay_in_their_row(n, dtype):
    c = Case("q8_0", 140, 128, ranks=[16, 20])
    x = c.rows_of(n, dtype)
    ids = c.rng.integers(-1, 2, n)
    clean = c.run(x, dtype, ids)
    bad = [0, n // 2, n - 1]
    for t, v in zip(bad, (math.inf, math.nan, -math.inf)):
        x[t, 17] = v
    out = c.run(x, dtype, ids)
    assert out[bad].isnan().all()
    rest = np.setdiff1d(np.arange(n), bad)
    assert torch.equal(out[rest], clean[rest])
    c.fine()


@pytest.mark.parametrize("n", [5, 100, 300])
def test_a_nan_scale_stays_in_its_row_of_w(n):
    from block_quantized_token_gb300 import runtime
    rng = np.random.default_rng(6)
    raw = synth.quantize((rng.standard_normal((40, 96)) * 0.1).astype(np.float32), "q8_0").reshape(40, 3, 34).copy()
    raw[11, 1, :2] = np.array([math.nan], np.float16).view(np.uint8)
    raw[30, 2, :2] = np.array([math.inf], np.float16).view(np.uint8)
    w = oracle.dequant(raw.reshape(-1).copy(), "q8_0", 40, 96)
    m = runtime.Matrix("q8_0", 40, 96, torch.from_numpy(raw.reshape(-1).copy()).cuda())
    x = torch.tensor(rng.standard_normal((n, 96)), dtype=torch.float32, device="cuda")
    out = torch.empty((n, 40), device="cuda")
    m.mul(x, out)
    assert out[:, [11, 30]].isnan().all()
    rest = np.setdiff1d(np.arange(40), [11, 30])
    np.testing.assert_allclose(host(out)[:, rest], host(x) @ w[rest].T, atol=2e-5)


@pytest.mark.parametrize("w_type", ["q8_0", "q4_0"])
def test_weights_enter_exactly(w_type):
    """A row of x with a single power of two reads a column of W back, to the last bit, in fp32; 16-bit outputs are it rounded once."""
    c = Case(w_type, 300, 96)
    for n, dtype in ((96, "f32"), (3, "f32"), (96, "f16"), (200, "bf16")):
        x = torch.zeros((n, 96), dtype=DT[dtype], device="cuda")
        col = np.arange(n) % 96
        x[torch.arange(n), torch.tensor(col)] = 2.0
        want = torch.tensor(2 * c.w[:, col].T).float().to(DT[dtype])  # (fp32 holds every weight)
        assert torch.equal(c.run(x, dtype).cpu(), want), (n, dtype)


# ------------------------------------------------------------------------------------------------------------------
# memory
# ------------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [9, 70, 140, 290])
def test_strides_and_odd_addresses(n, dtype):
    c = Case("q4_0", 133, 160)
    for xo, yo, xp, yp in ((0, 0, 3, 5), (1, 1, 0, 0), (3, 2, 7, 1), (8, 4, 8, 8)):
        xb = torch.full((n * (160 + xp) + 16,), 9.0, dtype=DT[dtype], device="cuda")
        yb = torch.full((n * (133 + yp) + 16,), 7.0, dtype=DT[dtype], device="cuda")
        x = xb[xo:xo + n * (160 + xp)].view(n, 160 + xp)[:, :160]
        y = yb[yo:yo + n * (133 + yp)].view(n, 133 + yp)
        x.copy_(c.rows_of(n, dtype))
        c.m.mul(x, y[:, :133])
        c.check(x, y[:, :133], dtype)
        assert (y[:, 133:] == 7).all() and (yb[:yo] == 7).all() and (yb[yo + n * (133 + yp):] == 7).all()
    c.fine()


def test_outputs_past_2_31_elements():
    c = Case("q8_0", 128256, 32)
    n = 17000
    x = c.rows_of(n, "bf16")
    out = torch.empty((n, 128256), dtype=torch.bfloat16, device="cuda")
    c.m.mul(x, out)
    at = [0, 8191, 16743, 16744, n - 1]  # 16743 rows and a piece are 2^31 elements
    c.check(x[at], out[at], "bf16")
    c.fine()


def test_tokens_past_2_23():
    """256 threads a token: their numbers pass 31 bits.  Every row against fp32 sums (32 terms and 4 of an adapter: 36 2^-24 of the
    terms' size on both sides, 2^-16 of the adapter's, half a step of bf16)."""
    c = Case("q8_0", 17, 32, ranks=[4])
    n = 2 ** 23 + 300
    x = torch.randn((n, 32), device="cuda").bfloat16()
    w, f = torch.tensor(c.w, device="cuda").float(), x.float()
    out = torch.full((n, 17), float("nan"), dtype=torch.bfloat16, device="cuda")
    c.m.mul(x, out)
    y, s = f @ w.T, f.abs() @ w.abs().T
    assert bool(((out.float() - y).abs() <= 1e-5 * s + 2.0 ** -8 * y.abs()).all())
    c.check(x[-300:], out[-300:], "bf16")
    scale, a, b = c.known[0]
    a, b = torch.tensor(a, device="cuda").float() * scale, torch.tensor(b, device="cuda").float()
    ids = torch.arange(n, dtype=torch.int32, device="cuda") % 2 - 1
    c.m.mul(x, out, adapters=c.ad, ids=ids)
    mine = (ids == 0)[:, None]
    y += (f @ a.T) @ b.T * mine
    s += (f.abs() @ a.abs().T) @ b.abs().T * mine
    assert bool(((out.float() - y).abs() <= 3e-5 * s + 2.0 ** -8 * y.abs()).all())
    c.fine()


def test_no_rows_and_longer_buffers():
    c = Case("q8_0", 40, 64, ranks=[4])
    out = torch.full((8, 40), 7.0, device="cuda")
    c.m.mul(torch.empty((0, 64), device="cuda"), out)
    assert (out == 7).all()
    x = c.rows_of(5, "f32")
    ids = ints([0, -1, 0, 0, -1, 9, 9])  # what lies behind the tokens is not read
    c.m.mul(x, out, adapters=c.ad, ids=ids)
    c.check(x, out[:5], "f32", ids.cpu().numpy()[:5])
    assert (out[5:] == 7).all()
    c.fine()


# ------------------------------------------------------------------------------------------------------------------
# adapters come and go
# ------------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("n", [6, 40, 100, 300])
def test_slots_past_the_end_and_empty_ones(n):
    c = Case("q8_0", 64, 128, ranks=[8, 24], slots=4)
    x = c.rows_of(n, "f32")
    ids = c.rng.integers(-3, 4, n)  # 2 and 3 are empty
    c.check(x, c.run(x, "f32", ids), "f32", ids)
    c.fine()
    for far in (4, 2 ** 31 - 1):
        ids[n // 2] = far
        c.check(x, c.run(x, "f32", ids), "f32", ids)
        c.fine(2)
    c.fine()


def test_slots_are_filled_again_and_emptied_in_order():
    c = Case("q8_0", 64, 128, ranks=[32, 8])
    x = c.rows_of(20, "bf16")
    ids = c.rng.integers(-1, 2, 20)
    for rank in (1, 32, 7):
        c.put(0, rank)
        c.check(x, c.run(x, "bf16", ids), "bf16", ids)
    c.ad.clear(0)
    del c.known[0]
    c.check(x, c.run(x, "bf16", ids), "bf16", ids)
    c.put(0, 3, scale=0.0)
    c.check(x, c.run(x, "bf16", ids), "bf16", ids)
    c.fine()


@pytest.mark.parametrize("adapter_type", ["f16", "bf16"])
def test_adapters_of_every_size(adapter_type):
    c = Case("q8_0", 96, 128, ranks=[16], adapter_type=adapter_type)
    a = torch.tensor(c.rng.standard_normal((16, 128)) * 2.0 ** c.rng.integers(-10, 10, (16, 1))).to(c.at).cuda()
    b = torch.tensor(c.rng.standard_normal((96, 16)) * 2.0 ** c.rng.integers(-10, 6, (96, 1))).to(c.at).cuda()
    c.ad.set(0, a, b, 1.5)
    c.known[0] = (1.5, host(a), host(b))
    for n in (4, 30, 100, 300):
        for dtype in ("f32", "bf16"):
            x = c.rows_of(n, dtype)
            ids = c.rng.integers(-1, 1, n)
            c.check(x, c.run(x, dtype, ids), dtype, ids)


# ------------------------------------------------------------------------------------------------------------------
# streams and graphs
# ------------------------------------------------------------------------------------------------------------------
def test_calls_of_two_streams_at_once():
    c = Case("q8_0", 1024, 2048, ranks=[16, 8])
    xs = [c.rows_of(n, "bf16") for n in (16, 200)]
    ids = [c.rng.integers(-1, 2, len(x)) for x in xs]
    want = [c.run(x, "bf16", i) for x, i in zip(xs, ids)]
    outs = [torch.empty_like(w) for w in want]
    di = [ints(i) for i in ids]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(30):
        for s, x, o, i in zip(streams, xs, outs, di):
            with torch.cuda.stream(s):
                c.m.mul(x, o, adapters=c.ad, ids=i)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    c.fine()


@pytest.mark.parametrize("n", [5, 50, 150, 300])
def test_captured_call_replays_with_new_rows_and_adapters(n):
    c = Case("q8_0", 200, 256, ranks=[16, 8], max_rank=40)
    x, out, ids = c.rows_of(n, "bf16"), torch.empty((n, 200), dtype=torch.bfloat16, device="cuda"), ints(np.full(n, -1))
    c.m.mul(x, out, adapters=c.ad, ids=ids)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.m.mul(x, out, adapters=c.ad, ids=ids)
        c.m.mul(x, out, adapters=c.ad, ids=ids)
    for step in range(4):
        i = c.rng.integers(-1, 2, n)
        ids.copy_(ints(i))
        x.copy_(c.rows_of(n, "bf16"))
        c.put(0, [16, 40, 3, 17][step])
        out.fill_(7)
        g.replay()
        c.check(x, out, "bf16", i)
    c.fine()


def test_graphs_and_streams_have_scratch_of_their_own():
    """Two graphs captured on one stream and calls of that stream, all running at once; a larger call in between."""
    c = Case("q8_0", 2000, 1024, ranks=[16, 40])
    sets = []
    for n, dtype in ((16, "bf16"), (70, "f32"), (40, "f16")):
        x, ids = c.rows_of(n, dtype), c.rng.integers(-1, 2, n)
        sets.append((x, ints(ids), c.run(x, dtype, ids), torch.empty((n, 2000), dtype=DT[dtype], device="cuda")))
    big = c.rows_of(3000, "bf16")
    wanted_big, out_big = c.run(big, "bf16"), torch.empty((3000, 2000), dtype=torch.bfloat16, device="cuda")
    at, graphs = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    for x, ids, _, out in sets[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=at):
            c.m.mul(x, out, adapters=c.ad, ids=ids)
        graphs.append((g, torch.cuda.Stream()))
    for i in range(20):
        for g, st in graphs:
            with torch.cuda.stream(st):
                for _ in range(5):
                    g.replay()
        with torch.cuda.stream(at):
            for _ in range(5):
                c.m.mul(sets[2][0], sets[2][3], adapters=c.ad, ids=sets[2][1])
            if i % 5 == 0:
                c.m.mul(big, out_big)
        torch.cuda.synchronize()
        for _, _, want, out in sets:
            assert torch.equal(out, want)
            out.zero_()
    assert torch.equal(out_big, wanted_big)
    c.fine()


def test_rows_made_by_the_kernel_before():
    """Rows, numbers and results that the stream's neighbours write and read: every call sees the ones before it."""
    c = Case("q8_0", 256, 256, ranks=[16])
    n = 70
    x0 = c.rows_of(n, "f32")
    ids = ints(np.zeros(n))
    y = torch.empty((n, 256), device="cuda")
    for _ in range(50):
        x = x0 * 1.0
        c.m.mul(x, y, adapters=c.ad, ids=ids)
        z = y * 0.5
        c.m.mul(z, y, adapters=c.ad, ids=ids)
        ids.fill_(0)
    first = c.run(x0, "f32", np.zeros(n))
    assert torch.equal(c.run(first * 0.5, "f32", np.zeros(n)), y)


# ------------------------------------------------------------------------------------------------------------------
# waits that give up
# ------------------------------------------------------------------------------------------------------------------
GIVE_UP = [("f32", 30), ("bf16", 100), ("bf16", 300), ("f32", 200)]


@pytest.mark.parametrize("dtype,n", GIVE_UP)
def test_shortest_wait_limit(dtype, n):
    """Waits that give up at the first look: the result is right or flag bit 2 says that it is not; then all is well again."""
    from block_quantized_token_gb300 import er
    c = Case("q8_0", 600, 1024, ranks=[16, 40])
    x, ids = c.rows_of(n, dtype), c.rng.integers(-1, 2, n)
    want = c.run(x, dtype, ids)
    c.fine()
    er.er_set_wait_limit_ns(1)
    try:
        for _ in range(10):
            out = c.run(x, dtype, ids)
            _, code = c.m.error()
            assert code in (0, 4), code
            assert code == 4 or torch.equal(out, want)
    finally:
        er.er_set_wait_limit_ns(0)
    assert torch.equal(c.run(x, dtype, ids), want)
    c.fine()


@pytest.mark.parametrize("dtype,n", GIVE_UP)
def test_wait_gives_up_and_the_next_call_is_right(dtype, n):
    import time

    from block_quantized_token_gb300 import er
    c = Case("q4_0", 600, 1024, ranks=[16, 40])
    x, ids = c.rows_of(n, dtype), c.rng.integers(-1, 2, n)
    want = c.run(x, dtype, ids)
    c.fine()
    er.er_set_wait_limit_ns(5_000_000)
    er.er_matrix_mul_inject_wait_shortfall(c.m.handle, 1)
    try:
        for _ in range(3):
            t0 = time.perf_counter()
            c.run(x, dtype, ids)
            torch.cuda.synchronize()
            elapsed = time.perf_counter() - t0
            st, code = c.m.error()
            assert st == er.ER_EDEVICE and code == 4, (st, code)
            assert elapsed < 0.5, f"gave up after {elapsed:.3f} s with a 5 ms limit"
    finally:
        er.er_matrix_mul_inject_wait_shortfall(c.m.handle, 0)
        er.er_set_wait_limit_ns(0)
    for _ in range(3):
        assert torch.equal(c.run(x, dtype, ids), want)
    c.fine()


# ------------------------------------------------------------------------------------------------------------------
# refusals of the runtime
# ------------------------------------------------------------------------------------------------------------------
def test_runtime_refuses_wrong_tensors():
    from block_quantized_token_gb300 import er, runtime
    c = Case("q8_0", 40, 64, ranks=[4])
    x, out, ids = c.rows_of(3, "f32"), torch.empty((3, 40), device="cuda"), ints([0, 0, 0])
    for bad in (lambda: c.m.mul(x[:, :32], out), lambda: c.m.mul(x, out[:, :39]), lambda: c.m.mul(x, out[:2]),
                lambda: c.m.mul(x.half(), out), lambda: c.m.mul(x.double(), out.double()), lambda: c.m.mul(x.cpu(), out),
                lambda: c.m.mul(x, out.t().contiguous().t()), lambda: c.m.mul(x, out, adapters=c.ad),
                lambda: c.m.mul(x, out, ids=ids), lambda: c.m.mul(x, out, adapters=c.ad, ids=ids[:2]),
                lambda: c.m.mul(x, out, adapters=c.ad, ids=ids.long()), lambda: c.ad.set(0, torch.zeros(2, 64), torch.zeros(40, 2)),
                lambda: c.ad.set(0, torch.zeros(2, 32, device="cuda"), torch.zeros(40, 2, device="cuda")),
                lambda: runtime.Matrix("q8_0", 40, 64, torch.zeros(5, dtype=torch.uint8, device="cuda")),
                lambda: runtime.Matrix("f16", 40, 64, torch.zeros(5, dtype=torch.uint8, device="cuda")),
                lambda: runtime.Adapters(40, 64, 2, 4, torch.float32)):
        with pytest.raises(ValueError):
            bad()
    other = runtime.Adapters(40, 96, 1, 4)
    with pytest.raises(er.ErError) as e:
        c.m.mul(x, out, adapters=other, ids=ids)
    assert e.value.status == er.ER_EINVAL
    c.fine()


def test_handles_free_what_they_allocate():
    from block_quantized_token_gb300 import er
    live = er.er_debug_live_allocations()
    c = Case("q8_0", 40, 64, ranks=[4])
    assert c.ad.device_bytes >= 16 * (64 + 40) * 2
    c.run(c.rows_of(5, "f32"), "f32", [0] * 5)
    torch.cuda.synchronize()
    c.ad.close()
    c.m.close()
    assert er.er_debug_live_allocations() == live


# ------------------------------------------------------------------------------------------------------------------
# adapters that hold infinities and NaN
# ------------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan, 3e30])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [5, 17, 50, 120, 300])
def test_an_adapter_s_infinities_stay_with_its_tokens(n, dtype, value):
    """B of one slot holds a value that is no number (or one so large that it is none once W's row brings it up): tokens of other
    slots and of none do not see it, those of the slot get what the formula says.  A slot that is filled again is like any other."""
    rng = np.random.default_rng([n, 3])
    w = (rng.standard_normal((150, 256)) * 0.05).astype(np.float32)
    w[40:60] *= 2.0 ** -12
    c = Case("q8_0", 150, 256, weights=w, ranks=[16, 24, 8])
    x, ids = c.rows_of(n, dtype), c.rng.integers(-1, 3, n)
    ids[:4] = [0, 1, 2, -1]
    clean, plain = c.run(x, dtype, ids), c.run(x, dtype)
    scale, a, b = c.known[1]
    bad = b.copy()
    bad[45, 3], bad[120, 0] = value, value
    ta, tb = (torch.tensor(z).to(c.at).cuda() for z in (a, bad))
    c.ad.set(1, ta, tb, scale)
    out = c.run(x, dtype, ids)
    assert torch.equal(out[ids == -1], plain[ids == -1])
    others = ids != 1
    c.check(x, out, dtype, ids, rows=others)
    got, v = host(out)[~others], scale * host(x)[~others] @ a.T
    fine = np.setdiff1d(np.arange(150), [45, 120])
    np.testing.assert_allclose(got[:, fine], host(clean)[~others][:, fine], rtol=2 * HALF[dtype], atol=2e-4)
    for row, j in ((45, 3), (120, 0)):
        with np.errstate(over="ignore", invalid="ignore"):
            want = v[:, j] * value
        if math.isnan(value):
            assert np.isnan(got[:, row]).all()
        else:
            assert (np.sign(got[:, row]) == np.sign(want)).all() and (np.abs(got[:, row]) > 1e20).all()
    c.ad.set(1, ta, torch.tensor(b).to(c.at).cuda(), scale)
    assert torch.equal(c.run(x, dtype, ids), clean)
    c.fine()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [5, 17, 50, 120, 300])
def test_infinities_of_an_adapter_s_a_stay_with_its_tokens(n, dtype):
    c = Case("q8_0", 150, 256, ranks=[16, 24, 8], adapter_type="f16")
    x, ids = c.rows_of(n, dtype), c.rng.integers(-1, 3, n)
    ids[:4] = [0, 1, 2, -1]
    clean = c.run(x, dtype, ids)
    scale, a, b = c.known[1]
    a = a.copy()
    a[2, 10], a[20, 200] = math.inf, math.nan
    c.ad.set(1, torch.tensor(a).half().cuda(), torch.tensor(b).half().cuda(), scale)
    out = c.run(x, dtype, ids)
    assert torch.equal(out[ids != 1], clean[ids != 1]) and out[ids == 1].isnan().all()
    c.fine()


# ------------------------------------------------------------------------------------------------------------------
# host threads, streams of one's own
# ------------------------------------------------------------------------------------------------------------------
def test_two_host_threads_on_one_stream():
    """A call is several launches, and another thread's may come between them: each works on memory of its own."""
    import sys
    import threading
    cases = [Case("q8_0", 512, 1024, seed=i, ranks=[16]) for i in range(3)]
    xs = [c.rows_of(n, d) for c, n, d in zip(cases, (70, 40, 12), ("f32", "bf16", "f16"))]
    ids = [ints(c.rng.integers(-1, 1, len(x))) for c, x in zip(cases, xs)]
    want, wrong = [], [0, 0, 0]
    for c, x, i in zip(cases, xs, ids):
        want.append(torch.empty((len(x), 512), dtype=x.dtype, device="cuda"))
        c.m.mul(x, want[-1], adapters=c.ad, ids=i)
    torch.cuda.synchronize()
    begin = threading.Barrier(3)

    def work(t):
        outs = [torch.empty_like(want[t]) for _ in range(50)]
        begin.wait()
        for _ in range(8):
            for o in outs:
                cases[t].m.mul(xs[t], o, adapters=cases[t].ad, ids=ids[t])
            wrong[t] += sum(not torch.equal(o, want[t]) for o in outs)

    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=work, args=(t,)) for t in range(3)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(before)
    assert wrong == [0, 0, 0]
    for c in cases:
        c.fine()


def test_kept_scratch_is_bounded_and_goes_with_its_thread():
    import gc
    import threading
    c = Case("q8_0", 64, 4096)
    x, out = c.rows_of(2000, "bf16"), torch.empty((2000, 64), dtype=torch.bfloat16, device="cuda")  # some 16 MB of scratch
    torch.cuda.synchronize()
    gc.collect()
    before = torch.cuda.memory_allocated()

    def use():
        for s in [torch.cuda.Stream() for _ in range(30)]:
            with torch.cuda.stream(s):
                c.m.mul(x, out)
        torch.cuda.synchronize()
        peak.append(torch.cuda.memory_allocated())

    peak = []
    t = threading.Thread(target=use)
    t.start()
    t.join()
    gc.collect()
    assert peak[0] - before < 200 << 20
    assert torch.cuda.memory_allocated() == before


def _scratch_seen(monkeypatch):
    """(address, bytes) of the scratch of every call from here on."""
    from block_quantized_token_gb300 import er
    seen, call = [], er.er_matrix_mul

    def spy(mat, args, stream=0):
        seen.append((args.work, args.work_bytes))
        call(mat, args, stream)

    monkeypatch.setattr(er, "er_matrix_mul", spy)
    return seen


@pytest.mark.parametrize("n", [20, 20000])
def test_scratch_of_a_call_on_a_given_stream_is_not_given_away(n, monkeypatch):
    """mul(..., stream=s): while s still works on it, the current stream's allocations do not get the scratch."""
    c = Case("q8_0", 300, 1024, ranks=[16])
    x, ids = c.rows_of(n, "bf16"), ints(c.rng.integers(-1, 1, n))
    want, out = torch.empty((n, 300), dtype=torch.bfloat16, device="cuda"), torch.zeros((n, 300), dtype=torch.bfloat16, device="cuda")
    c.m.mul(x, want, adapters=c.ad, ids=ids)
    torch.cuda.synchronize()
    seen, s = _scratch_seen(monkeypatch), torch.cuda.Stream()
    for _ in range(3):
        done = torch.cuda.Event()
        with torch.cuda.stream(s):
            torch.cuda._sleep(200_000_000)
        c.m.mul(x, out, adapters=c.ad, ids=ids, stream=s.cuda_stream)
        done.record(s)
        at, size = seen[-1]
        held = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
        assert not done.query()  # (else nothing is shown)
        assert all(t.data_ptr() + size <= at or at + size <= t.data_ptr() for t in held)
        for t in held:
            t.fill_(255)
        s.synchronize()
        assert torch.equal(out, want)
        out.zero_()
        del held, t
    # the default stream by its number, and the current one by its own
    for number in (0, torch.cuda.current_stream().cuda_stream):
        c.m.mul(x, out, adapters=c.ad, ids=ids, stream=number)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        out.zero_()
    c.fine()


def test_a_call_on_a_given_stream_is_captured():
    """The stream that captures is another than the current one: the graph still owns its scratch."""
    c = Case("q8_0", 300, 1024, ranks=[16])
    x, ids = c.rows_of(50, "bf16"), ints(c.rng.integers(-1, 1, 50))
    want, out = c.run(x, "bf16", ids.cpu().numpy()), torch.zeros((50, 300), dtype=torch.bfloat16, device="cuda")
    s, g, other = torch.cuda.Stream(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        other.wait_stream(s)
        with torch.cuda.stream(other):
            c.m.mul(x, out, adapters=c.ad, ids=ids, stream=s.cuda_stream)
        s.wait_stream(other)
    c.m.mul(c.rows_of(70, "f32"), torch.empty((70, 300), device="cuda"), stream=s.cuda_stream)
    torch.cuda.synchronize()
    held = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    del held
    c.fine()


@pytest.mark.parametrize("n", [5, 40, 100, 300])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_next_to_the_least_number(n, dtype):
    """Rows whose largest value is below 2^-112 enter times 2^126: exactly (fp32 rows too: their least bit is 2^-149, 2^-23 then).
    Results are rounded to the type's least numbers, and so are A x's: 2^-150 of each at most, times B."""
    c = Case("q8_0", 140, 256, ranks=[16, 24])
    x = c.rng.uniform(0.5, 1.0, (n, 256)) * 2.0 ** c.rng.integers(-140, -105, (n, 1))
    x = torch.tensor(x).to(DT[dtype]).cuda()
    least = 2.0 ** -149 if dtype == "f32" else 2.0 ** -133
    for ids in (None, c.rng.integers(-1, 2, n)):
        out = c.run(x, dtype, ids)
        y, (s, t) = orq.product(host(x), c.w, ids, c.known)
        tol = ((12 * 4 + 100) * 2.0 ** -23 + 2.0 ** -21) * s + HALF[dtype] * np.abs(y) + least
        if ids is not None:
            tol += ((256 / 16 + 80 + 24) * 2.0 ** -23 + (2.0 ** -22 if dtype == "f32" else 2.0 ** -16)) * t
            tol += 2.0 ** -149 * max(np.abs(b).sum(1).max() for _, _, b in c.known.values())
        assert (np.abs(host(out) - y) <= tol).all(), float((np.abs(host(out) - y) / tol).max())
    c.fine()


@pytest.mark.parametrize("n", [3, 40, 300])
@pytest.mark.parametrize("w_type", ["q8_0", "q4_0"])
def test_scales_far_apart_in_a_row(w_type, n):
    """A row's scales from fp16's largest to its least.  Up to 16 tokens every weight is exact; else d times the row's power of two is
    rounded to 2^-24 / 2 where the largest scale is 256 (Q4_0: 4096) and more: a value's error is at most 2^-32 (2^-36) of the row's largest
    scale times 128 (8).  x reads single weights back."""
    from block_quantized_token_gb300 import runtime
    rng = np.random.default_rng(12)
    rows, cols = 64, 128
    nb = cols // 32
    d = 2.0 ** rng.uniform(-14, 15.9, (rows, nb)) * rng.choice([-1, 1], (rows, nb))
    d[:, 0] = 2.0 ** rng.uniform(8, 15.9, rows)
    d[0], d[1], d[2] = [256.0, 2.0 ** -14 * (1 + 2.0 ** -10), 2.0 ** -20, 2.0 ** -24], [65504.0, 2.0 ** -14, 1.0, 2.0 ** -24], 2.0 ** -24
    raw = synth.quantize(np.ones((rows, cols), np.float32), w_type).reshape(rows, nb, -1).copy()
    raw[..., :2] = np.ascontiguousarray(d.astype(np.float16)).view(np.uint8).reshape(rows, nb, 2)
    raw[..., 2:] = rng.integers(0, 256, raw[..., 2:].shape)
    raw = raw.reshape(-1)
    w = oracle.dequant(raw, w_type, rows, cols)
    m = runtime.Matrix(w_type, rows, cols, torch.from_numpy(raw).cuda())
    largest = np.abs(d.astype(np.float16).astype(float)).max(1) * (128 if w_type == "q8_0" else 8)
    least = largest >= (256 * 128 if w_type == "q8_0" else 4096 * 8)
    for c0 in range(0, cols, n):
        k = min(n, cols - c0)
        x = torch.zeros((n, cols), device="cuda")
        x[torch.arange(k), torch.arange(c0, c0 + k)] = 1.0
        out = torch.empty((n, rows), device="cuda")
        m.mul(x, out)
        got, want = host(out)[:k], w[:, c0:c0 + k].T
        off = np.abs(got - want) - 2.0 ** -24 * np.abs(want)  # (fp32 holds every weight: the rest is for sums)
        if n <= 16:
            assert (off <= 0).all()
        else:
            assert (off <= (least * largest * 2.0 ** (-32 if w_type == "q8_0" else -36))).all()
    assert m.error()[1] == 0


@pytest.mark.parametrize("w_type", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [3, 16, 40, 100, 300])
def test_the_low_bits_of_weights_count_in_wide_products(n, dtype, w_type):
    """Columns by turns of 32: scales d and d + 1 unit of fp16, codes q; x is +1 and -1 by turns (of a size by token).  With w = d q,
    2^10 <= |d| / unit < 2^11, y is half the columns' sum of q unit: at least 2^-11 of it a column, while every partial sum stays
    below 64 w.  What the sums lose: at most 8 (fp32: 12) additions a step, cut off at 2^-23 of 64 w:
        |y - exact| <= 12 n_steps 2^-23 64 w + half a step of y
    (few tokens add blocks of 32 in fewer additions).  At 14336 columns that is 0.021 w + ..., and y = 7168 q unit >= 3.5 w.  The high
    halves alone step by 2^-11 w and more, as much as a column's share of y: without the low ones y would be another number."""
    from block_quantized_token_gb300 import runtime
    rows, cols = 40, 14336
    rng = np.random.default_rng(11)
    nb = cols // 32
    base = (1024 + rng.integers(0, 1022, rows)) * 2.0 ** -18
    d = np.repeat(base[:, None], nb, 1)
    d[:, 1::2] += 2.0 ** -18
    q = rng.integers(65, 127, (rows, 1)) if w_type == "q8_0" else rng.integers(5, 8, (rows, 1))
    head = np.ascontiguousarray(d.astype(np.float16)).view(np.uint8).reshape(rows, nb, 2)
    if w_type == "q8_0":
        body = np.broadcast_to(q[:, :, None], (rows, nb, 32)).astype(np.int8).view(np.uint8)
    else:
        body = np.broadcast_to(((q + 8) * 17)[:, :, None], (rows, nb, 16)).astype(np.uint8)
    raw = np.ascontiguousarray(np.concatenate([head, body], 2)).reshape(-1)
    w = oracle.dequant(raw, w_type, rows, cols)
    m = runtime.Matrix(w_type, rows, cols, torch.from_numpy(raw).cuda())
    sign = np.where(np.arange(cols) // 32 % 2, -1.0, 1.0)
    size = 2.0 ** rng.integers(-3, 4, (n, 1))
    x = torch.tensor(sign * size).to(DT[dtype]).cuda()
    out = torch.empty((n, rows), dtype=DT[dtype], device="cuda")
    m.mul(x, out)
    y = host(x) @ w.T
    top = 64 * np.abs(w).max(1) * size
    tol = 12 * (cols // 64) * 2.0 ** -23 * top + HALF[dtype] * np.abs(y)
    assert (np.abs(host(out) - y) <= tol).all(), float((np.abs(host(out) - y) / tol).max())
    assert (tol < 0.02 * np.abs(y)).all()  # (the tolerance tells the two apart)
    assert m.error()[1] == 0


@pytest.mark.parametrize("n", [5, 16, 17, 100, 300])
@pytest.mark.parametrize("cols", [4096, 14336])
def test_fp32_rows_in_norm(cols, n):
    """The error in norm, where an output's own tolerance is wide.  Random terms: partial sums of k of K terms are sqrt(k / K) of
    the whole sum's size, so additions that cut off lose at most 2^-23 of 2 / 3 of it each on average.  24 in the tensor cores (by then
    the partial sum is of two steps: sqrt(2 / n_steps)), the others to nearest and in turn, by chance: n_steps of 2^-24 each
    at most; halves of x 2^-22, of terms by chance; W exactly:
        |y - exact| <= (24 sqrt(2 / n_steps) 2^-23 sqrt(n_steps) + n_steps 2^-24 + 2^-21) |exact| < (n_steps 2^-24 + 2^-17.5) |exact|
    W's low halves (2^-12 of a weight by chance, 2.4e-4) or x's would show."""
    c = Case("q8_0", 200, cols)
    x = c.rows_of(n, "f32")
    y = host(x) @ c.w.T
    steps = cols // 64
    bound = steps * 2.0 ** -24 + 2.0 ** -17.5
    assert bound < 1e-4 / 4
    err = np.linalg.norm(host(c.run(x, "f32")) - y) / np.linalg.norm(y)
    assert err <= bound, (err, bound)
    c.fine()


@pytest.mark.parametrize("dtype,adapter_type", [("f32", "f16"), ("f16", "bf16"), ("bf16", "bf16")])
def test_the_largest_ranks_and_the_last_slot(dtype, adapter_type):
    """Ranks of 129 to 256 beside small ones, in the last of 4096 slots too."""
    c = Case("q4_0", 100, 288, ranks=[256, 200, 3], adapter_type=adapter_type, slots=4096, max_rank=256)
    c.put(4095, 129)
    for n in (2, 16, 17, 64, 65, 130, 300):
        for pick in ([0], [-1, 0, 1, 2, 4095], [2, 4095]):
            ids = c.rng.choice(pick, n)
            x = c.rows_of(n, dtype)
            c.check(x, c.run(x, dtype, ids), dtype, ids)
    c.fine()
