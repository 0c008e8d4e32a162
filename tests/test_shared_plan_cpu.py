"""The shared-prefix decode's planner on the host: its time, and the counts that it may give."""
import ctypes
import time

import pytest

from paged_kv_cache_298_gb300 import binding


def plan(prefix, suffix, sms=152):
    a, b = ctypes.c_int(0), ctypes.c_int(0)
    assert binding.load().dap_shared_plan(sms, 1, 64, 64, 8, 128, prefix, suffix, 0, ctypes.byref(a), ctypes.byref(b)) == 0
    return a.value, b.value


@pytest.mark.parametrize("prefix", [32768, 10 ** 6, 10 ** 8, 2 ** 30, 2 ** 31 - 1])
def test_time_does_not_grow_with_the_prefix(prefix):
    """A caller that leaves the counts to the planner pays for it on every call.  It has at most as many prefix counts to
    consider as the device has SMs, whatever the prefix: some microseconds, where a walk over every tile of 2^30 keys takes 50
    milliseconds.  The fastest of several, so that a busy machine does not matter."""
    best = 1e9
    for _ in range(7):
        t = time.perf_counter()
        plan(prefix, 1000)
        best = min(best, time.perf_counter() - t)
    assert best < 1e-3


def test_counts_split_the_prefix_evenly():
    """Every count that is chosen is one that some whole number of tiles a split gives: none of its splits is empty."""
    for sms in (1, 16, 152):
        for prefix in list(range(1, 3000, 37)) + [10 ** 6, 2 ** 30]:
            for suffix in (0, 700):
                n, _ = plan(prefix, suffix, sms)
                tiles = -(-prefix // 64)
                per = -(-tiles // n)
                assert 1 <= n <= tiles and -(-tiles // per) == n and n * 8 <= max(8, sms)
