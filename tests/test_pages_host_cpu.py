"""The paged cache's host side over a stand-in for the CUDA runtime (tests/fake_cuda.py)."""

from __future__ import annotations

import functools

import pytest

import fake_cuda

torch = pytest.importorskip("torch")


def test_error_words_are_cleared_when_the_call_returns(tmp_path):
    """A clear that is still on its way could wipe out the flag, or the arrivals, of a call on another stream."""
    fake_cuda.run(tmp_path, """
h = er.er_pages_create(cfg, pool_ptr)
assert word("fake_pending").value == 0
flags = ctypes.c_int.from_address(ctypes.c_void_p.in_dll(fake, "fake_last_alloc").value)
for code in (0, 1, 2, 4, 7):
    flags.value = code
    assert er.er_pages_error(h) == ((er.ER_EDEVICE if code else er.ER_OK), code)
    assert flags.value == 0 and word("fake_pending").value == 0, code
er.er_pages_destroy(h)
""")


def test_decode_states_error_word_is_cleared_when_the_call_returns(tmp_path):
    fake_cuda.run(tmp_path, """
x = er.er_config(dim=64, n_layers=1, n_heads=1, n_kv_heads=1, head_dim=64, ffn_dim=64, vocab=64, rope_base=1e4, rms_eps=1e-5,
                 w_type=er.ER_Q8_0, tied=1, max_batch=1)
buf = (ctypes.c_uint8 * (1 << 20))()
p = ctypes.addressof(buf)
layers = (er.er_layer_weights * 1)()
for name, _ in er.er_layer_weights._fields_:
    setattr(layers[0], name, p)
w = er.er_weights(tok_embd=p, output_norm=p, output=None, layers=ctypes.cast(layers, ctypes.POINTER(er.er_layer_weights)))
m = er.er_model_create(x, w, 0)
kv = er.er_kv_create(m, 1, 64)
word("fake_pending").value = 0
er.er_get_device_error(kv)
assert word("fake_pending").value == 0
""")


def test_memory_of_another_device_is_refused(tmp_path):
    fake_cuda.run(tmp_path, """
for own, other in ((0, 1), (1, 0)):
    word("fake_device").value, word("fake_pointer_device").value = own, other
    assert refused(er.er_rope_table, 64, 10000.0, 4, at) == er.ER_EINVAL
    assert refused(er.er_pages_create, cfg, pool_ptr) == er.ER_EINVAL
    assert word("fake_launches").value == own
    word("fake_pointer_device").value = own
    assert refused(er.er_rope_table, 64, 10000.0, 4, at) == er.ER_OK
    h = er.er_pages_create(cfg, pool_ptr)
    word("fake_device").value = other
    assert refused(er.er_pages_read, h, 0, 4, at, er.ER_F32, pool_ptr, None) == er.ER_EINVAL
    er.er_pages_destroy(h)
""")

def test_release_refuses_more_entries_than_it_can_number(tmp_path):
    """The kernel's running number of an entry must not pass an int, nor the first of the block's width after the last."""
    fake_cuda.run(tmp_path, """
h = er.er_pages_create(cfg, pool_ptr)
for n, stride in ((1024, 1 << 21), (2, 2**30), (1, 2**31 - 1), (1, 2**31 - 1023)):
    assert refused(er.er_pages_release, h, n, at, at, at, stride, at, at) == er.ER_EINVAL, (n, stride)
assert word("fake_launches").value == 0
for n, stride in ((1023, 1 << 21), (1, 2**31 - 1024), (1024, 1)):
    assert refused(er.er_pages_release, h, n, at, at, at, stride, at, at) == er.ER_OK, (n, stride)
er.er_pages_destroy(h)
""")

def test_a_single_token_is_no_prompt(tmp_path):
    """A token's 64 query heads on one K/V head are one launch of the kernel that spreads the cached rows over the SMs."""
    fake_cuda.run(tmp_path, """
one = er.er_pages_config(1, 10, 32, 1, 64, er.ER_Q4_0)
h = er.er_pages_create(one, pool_ptr)
def launches(seqs, tokens):
    before = word("fake_launches").value
    er.er_pages_attention(h, 0, er.er_pages_attention_args(seqs, tokens, 64, er.ER_BF16, 10, 0, pool_ptr, pool_ptr, None, 4096,
                                                           4096, at, at, at, 0.0))
    return word("fake_launches").value - before
assert launches(1, 1) == 1 and launches(3, 3) == 1 and launches(1, 2) == 2 and launches(3, 4) == 2
er.er_pages_destroy(h)
""")

class Current:
    """Stands for torch.cuda.device: which device a call found current."""

    def __init__(self, start):
        self.now = start

    def __call__(self, device):
        return _Held(self, device)


class _Held:
    def __init__(self, current, device):
        self.current, self.device = current, device

    def __enter__(self):
        self.before, self.current.now = self.current.now, self.device

    def __exit__(self, *_):
        self.current.now = self.before


def _runtime(monkeypatch, current, home=None):
    from block_quantized_token_gb300 import build
    build.build()
    from block_quantized_token_gb300 import er, runtime
    seen = []

    def call(name, *a):
        if name != "er_rope_table" and current.now != home:  # as the library refuses it
            raise er.ErError(name, er.ER_EINVAL)
        if a[0] is None:
            raise er.ErError(name, er.ER_EUNSUPPORTED)
        seen.append((name, current.now))

    for name in ("er_rope_table", "er_pages_plan", "er_pages_release", "er_pages_append", "er_pages_read", "er_pages_attention",
                 "er_pages_error"):
        monkeypatch.setattr(er, name, functools.partial(call, name))
    monkeypatch.setattr(torch.cuda, "device", current)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current.now, raising=False)
    return runtime, seen


def test_rope_table_runs_on_the_device_of_its_memory(monkeypatch):
    current = Current(3)
    runtime, seen = _runtime(monkeypatch, current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: type("S", (), dict(cuda_stream=0)))
    runtime.rope_table(64, 10000.0, 4, device="cpu")
    assert seen == [("er_rope_table", torch.device("cpu"))] and current.now == 3


def test_paged_calls_run_on_the_cache_s_device(monkeypatch):
    current = Current(3)
    runtime, seen = _runtime(monkeypatch, current, home=-1)
    from block_quantized_token_gb300 import er
    c = object.__new__(runtime.PagedCache)
    c.n_kv_heads, c.head_dim, c.cfg, c.handle = 2, 64, er.er_pages_config(1, 4, 16, 2, 64, er.ER_Q4_0), 1
    c.device, c._index = torch.device("cpu"), -1  # (a CPU tensor's index)
    try:
        i, x, t = torch.zeros(8, dtype=torch.int32), torch.zeros(4, 2, 64), torch.zeros(1, 2, dtype=torch.int32)
        one = i[:1]
        c.plan(one, one, t, i, one, one, one, i, i, i, i, stream=0)
        c.release(one, one, t, i, one, stream=0)
        c.append(0, None, x, x, None, i, stream=0)
        c.read(0, i[:4], x, x, stream=0)
        c.attention(0, x, x, i, one, t, stream=0)
        c.error()
        assert [d for _, d in seen] == [-1] * 6 and current.now == 3
        # any other refusal stays one, wherever it happens
        c.handle = None
        for now in (3, -1):
            current.now = now
            for f in (c.error, lambda: c.read(0, i[:4], x, x, stream=0)):
                with pytest.raises(er.ErError) as e:
                    f()
                assert e.value.status == er.ER_EUNSUPPORTED and current.now == now
    finally:
        c.handle = None
