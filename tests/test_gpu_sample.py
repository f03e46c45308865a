"""er_sample on the GPU against the float64 oracle (oracle/requests.py).

Tokens are equal where u's place is further than 2^-38 of the kept sum from every kept token's border (the masses' whole
numbers of 2^-44 are within 5 of their value, and at most 2^18 are added: 2^-42 2^9 as they come, by chance); no input of these
tests lies nearer.  Log-probabilities: z within 2^-22 of its size, the sum's logarithm within 2^-22 of its
size and 2^-23: |l - exact| <= 2^-22 (|z| + |l - z|) + 2^-22.
"""

from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import requests as orq

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def dev(x, dtype=torch.float32):
    return None if x is None else torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def run(logits, u, logprobs=True, **kw):
    from block_quantized_token_gb300 import runtime
    n = logits.shape[0]
    tokens = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((n,), math.nan, device="cuda") if logprobs else None
    k = kw.pop("top_k", None)
    runtime.sample(logits, dev(u), tokens, top_k=dev(k, torch.int32), logprobs=lp, **{a: dev(b) for a, b in kw.items()})
    return tokens, lp


def check(logits, u, **kw):
    tokens, lp = run(logits, u, **kw)
    again, lp2 = run(logits, u, **kw)
    assert torch.equal(tokens, again) and torch.equal(lp, lp2)
    x, t, l = logits.detach().cpu().double().numpy(), tokens.cpu().numpy(), lp.cpu().double().numpy()
    for i in range(len(x)):
        row = {a: float(np.float32(b[i])) if a != "top_k" else int(b[i]) for a, b in kw.items() if b is not None}
        want, logp, distance = orq.sample(x[i], float(np.float32(u[i])), **row)
        assert distance > 2.0 ** -38, (i, distance)
        assert t[i] == want, (i, int(t[i]), want, row, u[i], distance)
        if math.isinf(logp):
            assert l[i] == logp
        else:
            temp = row.get("temperature", 1.0)
            z = 0.0 if not temp > 0 or x[i][want] == np.nanmax(x[i]) else abs((x[i][want] - np.nanmax(x[i])) / temp)
            assert abs(l[i] - logp) <= 2.0 ** -22 * (z + abs(abs(logp) - z)) + 2.0 ** -22, (i, l[i], logp)
    return t


def bulk(rng, n, v, spread=2.0, likely=20, high=8.0):
    x = rng.standard_normal((n, v)) * spread
    for r in x:
        r[rng.choice(v, min(v, likely), replace=False)] += high
    return x


FILTERS = {
    "temperature": dict(temperature=[0.7, 1.0, 1.5, 0.1, 4.0]),
    "top_k": dict(top_k=[1, 2, 40, 200, 0, 5, 3000, 100000]),
    "top_p": dict(top_p=[0.9, 0.5, 0.99, 0.999, 0.05, 1.0, 0.7]),
    "min_p": dict(min_p=[0.05, 0.5, 0.001, 1.0, 0.0, 0.2]),
    "all": dict(temperature=[0.7, 1.0, 1.3, 0.0], top_k=[50, 0, 1000, 7, 2500], top_p=[0.9, 1.0, 0.95], min_p=[0.0, 0.05]),
}


# vocabularies at every change of the cluster's size, and of a thread's elements
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [1, 2, 31, 513, 8192, 8193, 16385, 32000, 50257, 128256])
@pytest.mark.parametrize("filters", sorted(FILTERS))
def test_filters(filters, vocab, dtype):
    rng = np.random.default_rng([vocab, sorted(FILTERS).index(filters), sorted(DT).index(dtype)])
    n = 12 if vocab < 20000 else 6
    for spread, high in ((2.0, 8.0), (3.0, 0.0), (0.02, 0.0)):
        x = torch.tensor(bulk(rng, n, vocab, spread, high=high)).to(DT[dtype]).cuda()
        kw = {a: [b[int(rng.integers(len(b)))] for _ in range(n)] for a, b in FILTERS[filters].items()}
        check(x, rng.random(n, np.float32) * 0.999 + 0.0005, **kw)


@pytest.mark.parametrize("u", [0.0, 1e-30, 0.99999994, 1.0, 2.0, -1.0, math.nan])
def test_random_numbers_at_the_ends(u):
    rng = np.random.default_rng(1)
    x = torch.tensor(bulk(rng, 4, 3000)).float().cuda()
    kw = dict(top_k=[0, 30, 0, 2600], top_p=[1.0, 1.0, 0.9, 1.0])
    t, lp = run(x, [u] * 4, **kw)
    for i in range(4):
        want, logp, _ = orq.sample(x[i].cpu().double().numpy(), u, top_k=kw["top_k"][i], top_p=float(np.float32(kw["top_p"][i])))
        # at 1 - 2^-24 the last element of a wide row has less than that share
        assert int(t[i]) == want or u == 0.99999994, (i, int(t[i]), want)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [100, 20000, 128256])
def test_masked_rows(vocab, dtype):
    """Grammars: -infinity, the type's lowest value and NaN in masked places; one token left, none left, all masked alike."""
    rng = np.random.default_rng(vocab)
    low = float(torch.finfo(DT[dtype]).min)
    rows = []
    for mask in (-math.inf, low, math.nan):
        for left in (0, 1, 5):
            r = np.full(vocab, mask)
            r[rng.choice(vocab, left, replace=False)] = rng.standard_normal(left)
            rows.append(r)
    rows.append(np.where(rng.random(vocab) < 0.5, -math.inf, low))  # the lowest value is all there is
    x = torch.tensor(np.array(rows)).to(DT[dtype]).cuda()
    n = len(rows)
    u = rng.random(n, np.float32) * 0.98 + 0.01
    for kw in ({}, dict(top_k=[3] * n), dict(top_p=[0.8] * n), dict(min_p=[0.3] * n), dict(temperature=[0.0] * n),
               dict(top_k=[2100] * n, top_p=[0.7] * n), dict(temperature=[1e-3] * n), dict(temperature=[50.0] * n, top_p=[0.9] * n)):
        t = check(x, u, **kw)
        assert t[0] == t[6] == -1  # (-infinity and NaN everywhere; the lowest value everywhere is a row like any other)
        assert t[3] >= 0


@pytest.mark.parametrize("vocab", [10, 5000, 128256])
def test_equal_logits(vocab):
    """Ties go by index: all alike, a few values, as far as top-k and top-p reach into a value."""
    rng = np.random.default_rng(vocab)
    rows = [np.zeros(vocab), np.full(vocab, -3.5), rng.integers(0, 3, vocab).astype(float), rng.integers(-2, 2, vocab) / 64.0]
    x = torch.tensor(np.array(rows)).bfloat16().cuda()
    for k, p in ((0, 1.0), (vocab // 2 + 1, 1.0), (3, 1.0), (0, 0.5), (0, 0.33), (vocab - 1, 0.7), (2100, 0.9)):
        check(x, rng.random(4, np.float32) * 0.98 + 0.01, top_k=[k] * 4, top_p=[p] * 4)


def test_ranges_that_are_split_again():
    """More than 2048 elements of a few values next to each other, far from the others."""
    rng = np.random.default_rng(4)
    v = 100000
    x = np.full((3, v), -40.0)
    x[:, ::2] = -6.0 - rng.integers(0, 5, (3, v // 2)) / 128.0
    x[:, 77] = 0.0
    x = torch.tensor(x).float().cuda()
    for t in (1.0, 8.0):
        for k, p in ((9000, 1.0), (2500, 1.0), (0, 0.3), (0, 0.77), (45000, 0.5)):
            check(x, [0.1, 0.5, 0.9], temperature=[t] * 3, top_k=[k] * 3, top_p=[p] * 3)


def test_infinite_logits():
    x = torch.tensor([[0.0, math.inf, 5.0, math.inf], [math.inf, -math.inf, math.nan, 1.0], [1e38, -1e38, 3e38, 3e38]], device="cuda")
    for kw in ({}, dict(top_k=[2] * 3), dict(top_p=[0.4] * 3), dict(temperature=[2.0] * 3), dict(temperature=[math.inf] * 3)):
        check(x, [0.6, 0.3, 0.7], **kw)


@pytest.mark.parametrize("temperature", [1e-30, 1e-6, 1e6, 1e30, math.inf, 0.0, -1.0, math.nan])
def test_temperatures_of_every_size(temperature):
    rng = np.random.default_rng(3)
    x = torch.tensor(rng.standard_normal((3, 9000)) * 3).float().cuda()
    check(x, [0.3, 0.6, 0.8], temperature=[temperature] * 3)
    check(x, [0.3, 0.6, 0.8], temperature=[temperature] * 3, top_k=[20, 0, 2500], top_p=[0.9, 0.5, 1.0])


@pytest.mark.parametrize("temperature", [2.0 ** -120, 1e-37, 1e-40, 1e-45])
@pytest.mark.parametrize("vocab", [300, 9000])
def test_the_least_temperatures(vocab, temperature):
    """So small that only the largest logit has a mass: what is as large shares it."""
    x = torch.tensor(np.random.default_rng(4).standard_normal((5, vocab)) * 3).float().cuda()
    x[:, [17, 160, 291]] = 20.0
    u = [0.1, 0.4, 0.9, 0.6, 0.2]
    for kw in ({}, dict(top_k=[0, 2, 3, 40, 2]), dict(top_p=[0.9, 0.5, 1.0, 0.99, 0.6]), dict(min_p=[0.5, 1.0, 0.0, 0.1, 1e-3])):
        check(x, u, temperature=[temperature] * 5, **kw)
    assert check(x, u, temperature=[temperature] * 5).tolist() == [17, 160, 291, 160, 17]


def test_parameters_out_of_range_leave_nothing_out():
    rng = np.random.default_rng(8)
    x = torch.tensor(rng.standard_normal((4, 700))).float().cuda()
    u = [0.2, 0.4, 0.6, 0.8]
    want = check(x, u)
    assert (check(x, u, top_k=[-5, 0, 700, 2 ** 31 - 1], top_p=[1.5, math.nan, math.inf, 1.0], min_p=[-1.0, math.nan, 0.0, -0.0]) == want).all()
    assert (check(x, u, top_p=[0.0, -1.0, 1e-30, -math.inf]) == x.argmax(1).cpu().numpy()).all()
    assert (check(x, u, min_p=[1.0, 7.0, math.inf, 1.0]) == x.argmax(1).cpu().numpy()).all()


def test_the_largest_vocabulary():
    rng = np.random.default_rng(9)
    x = torch.tensor(bulk(rng, 3, 262144)).float().cuda()
    for kw in ({}, dict(top_k=[50] * 3), dict(top_p=[0.95] * 3), dict(top_k=[4000] * 3, top_p=[0.99] * 3)):
        check(x, [0.25, 0.5, 0.75], **kw)


def test_many_rows():
    rng = np.random.default_rng(10)
    n = 2000
    x = torch.tensor(rng.standard_normal((n, 300)) * 2).half().cuda()
    check(x, rng.random(n, np.float32) * 0.98 + 0.01, temperature=rng.uniform(0.5, 2, n), top_k=rng.integers(0, 300, n),
          top_p=rng.uniform(0.3, 1.1, n), min_p=rng.uniform(0, 0.2, n))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_odd_addresses(dtype):
    rng = np.random.default_rng(11)
    for v, off, pad in ((1000, 1, 0), (40000, 3, 5), (50257, 0, 1), (40000, 8, 8)):
        flat = torch.full((4 * (v + pad) + 16,), 50.0, dtype=DT[dtype], device="cuda")
        x = flat[off:off + 4 * (v + pad)].view(4, v + pad)[:, :v]
        x.copy_(torch.tensor(bulk(rng, 4, v)))
        check(x, [0.1, 0.4, 0.7, 0.95], top_k=[0, 20, 0, 3000], top_p=[1.0, 1.0, 0.9, 1.0])


def test_rows_past_2_31_elements():
    rng = np.random.default_rng(12)
    n, v = 16800, 128256
    x = torch.full((n, v), -30.0, dtype=torch.bfloat16, device="cuda")
    at = [0, 16743, 16744, n - 1]
    x[at] = torch.tensor(bulk(rng, 4, v)).bfloat16().cuda()
    t, _ = run(x, [0.37] * n, top_k=[40] * n)
    for i in at:
        want, _, _ = orq.sample(x[i].cpu().double().numpy(), float(np.float32(0.37)), top_k=40)
        assert int(t[i]) == want


def test_no_rows_no_logprobs_and_longer_arrays():
    rng = np.random.default_rng(13)
    x = torch.tensor(rng.standard_normal((5, 100))).float().cuda()
    from block_quantized_token_gb300 import runtime
    tokens = torch.full((9,), -7, dtype=torch.int32, device="cuda")
    runtime.sample(x[:0], dev([0.5] * 9), tokens)
    assert (tokens == -7).all()
    runtime.sample(x, dev([0.5] * 9), tokens, top_k=dev([9] * 9, torch.int32))
    assert (tokens[5:] == -7).all()
    t, _ = run(x, [0.5] * 5, logprobs=False, top_k=[9] * 5)
    assert torch.equal(t, tokens[:5])


def test_two_streams_and_a_captured_call():
    from block_quantized_token_gb300 import runtime
    rng = np.random.default_rng(14)
    xs = [torch.tensor(bulk(rng, n, 32000)).float().cuda() for n in (3, 40)]
    us = [dev(rng.random(len(x), np.float32)) for x in xs]
    ks = [torch.full((len(x),), 50, dtype=torch.int32, device="cuda") for x in xs]
    want, outs = [], []
    for x, u, k in zip(xs, us, ks):
        want.append(torch.empty(len(x), dtype=torch.int32, device="cuda"))
        runtime.sample(x, u, want[-1], top_k=k)
        outs.append(torch.empty_like(want[-1]))
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, x, u, k, o in zip(streams, xs, us, ks, outs):
            with torch.cuda.stream(s):
                runtime.sample(x, u, o, top_k=k)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # a captured call sees new numbers, parameters and logits
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        runtime.sample(xs[0], us[0], outs[0], top_k=ks[0])
    for step in range(4):
        xs[0].copy_(torch.tensor(bulk(rng, 3, 32000)))
        us[0].copy_(dev(rng.random(3, np.float32)))
        ks[0].fill_([5, 0, 2500, 100][step])
        g.replay()
        runtime.sample(xs[0], us[0], want[0], top_k=ks[0])
        assert torch.equal(outs[0], want[0])


def test_runtime_refuses_wrong_tensors():
    from block_quantized_token_gb300 import er, runtime
    x, u, t = torch.zeros((3, 50), device="cuda"), torch.zeros(3, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (lambda: runtime.sample(x[0], u, t), lambda: runtime.sample(x.double(), u, t), lambda: runtime.sample(x.cpu(), u, t),
                lambda: runtime.sample(x.t(), u, t), lambda: runtime.sample(x, u[:2], t), lambda: runtime.sample(x, u, t.long()),
                lambda: runtime.sample(x, u, t, top_k=u), lambda: runtime.sample(x, u, t, temperature=t),
                lambda: runtime.sample(x, u, t, logprobs=u.double()), lambda: runtime.sample(x, u.cpu(), t)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(er.ErError) as e:
        runtime.sample(torch.zeros((1, 262145), device="cuda"), u, t)
    assert e.value.status == er.ER_EUNSUPPORTED


def test_greedy_is_the_decode_step_s_argmax():
    """At temperature 0 the token is the one er_decode_step's argmax takes from the same logits."""
    import synth
    from block_quantized_token_gb300 import runtime
    wl = synth.workload("tiny")
    s = wl.shape
    model = runtime.DecodeModel(s, synth.gen.model_weights(s), max_batch=1)
    state = runtime.DecodeState(model, 1, wl.capacity)
    for l in range(s.n_layers):
        state.write_rows(0, l, *synth.kv_prefill(wl, 0, l))
    logits, argmax = torch.empty((1, s.vocab), device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    state.step(torch.tensor(wl.tokens0(), device="cuda"), torch.tensor(wl.positions0(), device="cuda"), logits, argmax)
    t, lp = run(logits, [0.5], temperature=[0.0])
    assert torch.equal(t, argmax) and float(lp) == 0.0
    check(logits, [0.7], temperature=[0.8], top_k=[40], top_p=[0.95])
    state.close()
    model.close()


def test_top_k_of_either_integer_type():
    """int64 is what torch makes of Python's numbers: taken as it is, numbers past 31 bits among them."""
    from block_quantized_token_gb300 import runtime
    rng = np.random.default_rng(15)
    ks = [50, 0, -3, 2 ** 40, -2 ** 40, 7, 2500, 2 ** 32 + 5, -2 ** 63, 2 ** 63 - 1, 1, 2 ** 31, 2 ** 32]
    n = len(ks)
    x, u = torch.tensor(bulk(rng, n, 9000)).float().cuda(), rng.random(n, np.float32) * 0.98 + 0.01
    want = check(x, u, top_k=[min(max(k, -1), 2 ** 31 - 1) for k in ks])
    tokens, lp = torch.full((n + 2,), -7, dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda")
    k = torch.tensor(ks + [3], device="cuda")
    assert k.dtype is torch.int64
    runtime.sample(x, dev(u), tokens, top_k=k, logprobs=lp)
    assert (tokens[:n].cpu().numpy() == want).all() and (tokens[n:] == -7).all()
    for bad in (lambda: runtime.sample(x, dev(u), tokens, top_k=k.short()), lambda: runtime.sample(x, dev(u), tokens, top_k=k[: n - 1]),
                lambda: runtime.sample(x, dev(u), tokens, top_k=k.cpu())):
        with pytest.raises(ValueError):
            bad()
    # captured, with numbers that change
    g, du = torch.cuda.CUDAGraph(), dev(u)
    with torch.cuda.graph(g):
        runtime.sample(x, du, tokens, top_k=k)
    for number in (1, 2 ** 33, 2100):
        k.fill_(number)
        g.replay()
        assert torch.equal(tokens[:n], run(x, u, top_k=[min(number, 2 ** 31 - 1)] * n)[0])


def test_top_k_that_is_all_that_reaches_the_groups_bound():
    """As many elements reach the bound that groups of elements give as top-k asks for, and more than the sort takes: the others,
    whose masses are no smaller than anyone's, are still left out."""
    v = 65536
    x = torch.zeros((4, v), device="cuda")
    at = np.concatenate([r * 8704 + 4 * np.arange(257) for r in range(8)])  # 8 CTAs' parts, the first element of a thread's four
    at = at[at < v]
    x[:, torch.tensor(at, device="cuda")] = 1.0
    u = [0.05, 0.35, 0.65, 0.95]
    for k in (len(at), len(at) - 1, len(at) + 1, 2049):
        check(x, u, top_k=[k] * 4)
        check(x, u, top_k=[k] * 4, min_p=[0.3, 0.5, 0.0, 1.0])
        check(x, u, top_k=[k] * 4, top_p=[1.0, 0.9, 0.99, 0.5])


def test_two_host_threads_with_other_vocabularies():
    """The kernel's shared memory is a setting of the device's: one thread's call does not lower it under another's."""
    import threading

    from block_quantized_token_gb300 import runtime
    rng = np.random.default_rng(17)
    xs = [torch.tensor(bulk(rng, 2, v)).float().cuda() for v in (300, 262144)]
    u, failed, begin = dev([0.3, 0.8]), [], threading.Barrier(2)
    want = [run(x, [0.3, 0.8], top_k=[40, 0])[0] for x in xs]
    k = dev([40, 0], torch.int32)

    def work(x, w):
        t = torch.empty(2, dtype=torch.int32, device="cuda")
        begin.wait()
        try:
            for _ in range(3000):
                runtime.sample(x, u, t, top_k=k)
            assert torch.equal(t, w)
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(xs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("temperature", [9e29, 1.1e30, 3e37, 1e38, 3.4e38, math.inf])
@pytest.mark.parametrize("vocab", [4, 700, 30000])
def test_differences_past_the_largest_number(vocab, temperature):
    """Finite logits further apart than float32's largest number, at temperatures where it counts."""
    rng = np.random.default_rng(vocab)
    x = rng.uniform(-3.4e38, 3.4e38, (4, vocab))
    x[0, :4], x[1, :4], x[2, :4] = [3e38, -3e38, 0.0, 1e38], [-3.4e38, 3.4e38, -1e38, 3.4e38], [3.4e38, -3.4e38, -3.3e38, -math.inf]
    x = torch.tensor(x).float().cuda()
    for u in ([0.9983, 0.3141, 0.9871, 0.4713], [0.1057, 0.8969, 0.6131, 0.0117]):
        for kw in ({}, dict(top_k=[3] * 4), dict(top_p=[0.99, 0.9, 0.5, 0.7]), dict(min_p=[1e-4, 0.5, 1e-9, 0.2]),
                   dict(top_k=[3, 2500, 20, 300], top_p=[0.999] * 4)):
            check(x, u, temperature=[temperature] * 4, **kw)


def test_min_p_on_masses_that_are_next_to_each_other():
    """Logits so close that their masses, whole numbers within 5 of the exact ones, do not all fall with them, with min_p's mass
    among them: which of these are kept is open, but what is kept is one beginning of the order, and a token is always drawn from it."""
    rng = np.random.default_rng(16)
    v, n = 300, 64
    for _ in range(30):
        p = np.float32(rng.uniform(2e-5, 9e-5))
        top = np.float32(-math.log(float(p)))  # logits next to 0 then have masses next to p
        at = float(top) + math.log(float(p))
        row = at + (np.arange(v) - v / 2) * 0.08 / (float(p) * 2.0 ** 44)  # 0.08 units of mass apart
        row = row[rng.permutation(v)].astype(np.float32)
        row[0] = top
        x = torch.tensor(np.broadcast_to(row, (n, v)).copy()).cuda()
        u = 1.0 - np.linspace(1e-5, 0.9 * v * float(p) / 2, n)
        tokens, lp = run(x, u, min_p=[float(p)] * n, top_k=[v - 1] * n)
        t, l = tokens.cpu().numpy(), lp.cpu().double().numpy()
        assert (t >= 0).all()
        z = row[t].astype(np.float64) - float(top)
        count = (np.exp(z - l) - 1.0) / float(p)  # elements kept beside the largest, within what the log-probability is exact to
        tol = 3e-6 / float(p)
        assert np.ptp(count) < 2 * tol and -tol < count.min() and count.max() < v
        rank = np.argsort(np.argsort(-row.astype(np.float64), kind="stable"))
        assert (rank[t] <= count + tol).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [5, 3000, 60000])
def test_negative_zeros_tie_with_zeros(vocab, dtype):
    """-0 and 0 are equal logits: the lower index comes first, among the largest as among top-k's and top-p's last."""
    rng = np.random.default_rng(vocab)
    x = np.zeros((5, vocab))
    x[1] = rng.integers(-1, 1, vocab) / 64.0
    x[2] = rng.integers(0, 2, vocab) / 64.0
    x[3] = np.where(rng.random(vocab) < 0.5, -math.inf, 0.0)
    x[4] = rng.integers(-2, 3, vocab)
    x[(x == 0) & (rng.random(x.shape) < 0.5)] = -0.0
    x[0, 0] = -0.0
    x = torch.tensor(x).to(DT[dtype]).cuda()
    assert bool(torch.signbit(x[0, 0]))
    for kw in ({}, dict(temperature=[0.0] * 5), dict(top_k=[1] * 5), dict(top_k=[vocab // 3 + 1] * 5), dict(top_p=[0.37] * 5),
               dict(top_k=[vocab // 2 + 1] * 5, top_p=[0.73] * 5), dict(top_k=[2100] * 5, min_p=[0.99] * 5)):
        check(x, [0.1357, 0.3511, 0.5713, 0.7331, 0.9177], **kw)
