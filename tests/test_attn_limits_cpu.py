"""Without a GPU: refusals of what the attention side's structures carry beyond
pointers of tensors."""
import ctypes as C

import pytest

import moe_speculative_verify_gb300 as m

FAKE = 1 << 40                    # never dereferenced: the call is refused first
INVALID = 1


@pytest.fixture(scope="module")
def lib():
    m.build()
    return m.load()


def test_rope_error_word_is_aligned(lib):
    c = m.KVCache(FAKE, FAKE, None, None, 8 * 64 * 128, 64 * 128, 128, m.KV_BF16, 10, 64, 8, 128)
    s = m.Seqs(FAKE, FAKE, FAKE, 2, 4, 1)
    r = m.Rope(FAKE, 128, 0, 1.0, FAKE + 2)
    call = lambda t: lib.moe_rope_append(C.byref(r), C.byref(c), C.byref(s), FAKE, 8192, FAKE, 1024, FAKE, 1024, FAKE, t, 64,
                                         FAKE, 8192, None)
    assert call(2) == INVALID and call(0) == 0
    assert m.Rope(FAKE, 128, 0, 1.0).err is None
