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
