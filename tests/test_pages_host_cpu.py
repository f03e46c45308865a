"""The paged cache's host side over a stand-in for the CUDA runtime (tests/fake_cuda.py)."""

from __future__ import annotations

import fake_cuda


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
