"""Bounds of the shared-prefix decode that its kernels' 32-bit positions cannot step through: refused before CUDA is touched.

A count of splits is (length + chunk - 1) / chunk in 32 bits.  One split's chunk is its bound rounded up to 64, so with a bound
past 2^30 a length below it can pass 2^31 on the way (100 + (2^31 - 64) - 1 is negative: no split, and the row comes out
as if it had no keys), and a bound above 2^31 - 64 has no chunk at all."""
import ctypes

import pytest

from paged_kv_cache_298_gb300 import binding

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below fails validation first
SHAPE, WORKSPACE = 2, 4


def call(prefix, suffix):
    """One sequence whose block table covers 2^31 positions; without a workspace, what passes the other checks stops there."""
    return binding.load().decode_attn_paged_shared(FAKE, 1024, 128, FAKE, FAKE, 64, 1024, FAKE, 1 << 21, FAKE, FAKE, FAKE, FAKE, 1, 1,
                                                   64, prefix, suffix, 1, 8, 2, 128, 0.1, 1, 1, None, 0, FAKE, 1024, 128, None)


@pytest.mark.parametrize("big", [2 ** 30 - 63, 2 ** 30, 2 ** 31 - 64, 2 ** 31 - 1])
def test_bounds_past_the_limit(big):
    assert call(100, big) == SHAPE and call(big, 100) == SHAPE and call(big, big) == SHAPE


def test_bounds_up_to_the_limit():
    top = 2 ** 30 - 64
    assert call(top, 100) == WORKSPACE and call(100, top) == WORKSPACE and call(top, top) == WORKSPACE
    chunk = binding.chunk_tokens(top, 1)
    assert chunk == top and top + 31 + chunk - 1 < 2 ** 31   # (the suffix's first tile starts up to 31 positions early)
