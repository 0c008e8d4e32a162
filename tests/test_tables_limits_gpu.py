"""Page tables at the ends of their ranges: lengths and row numbers near 2^31, and more new rows than that."""
import pytest
import torch

from paged_kv_cache_298_gb300 import binding
from test_tables_gpu import Pool

pytestmark = pytest.mark.gpu

MOST = (1 << 31) - 1


@pytest.fixture(autouse=True)
def _clean():
    binding.get_device_errors(clear=True)
    yield


@pytest.mark.parametrize("first,others", [(1000, 0), (3000, 0), (1000, 80), (12000, 80), (40000, 0)])
def test_positions_near_the_largest(first, others):
    """A sequence that ends at position 2^31 - 2 behind others with many new rows, whose numbers its own begin after: in one CTA,
    in a cluster and on the whole device."""
    ps = 1 << 20
    lens = [0] + [7] * others + [MOST - 51, MOST - 1, MOST]
    new = [first] + [7 + i % 3 for i in range(others)] + [MOST, MOST, MOST - ps - 5]
    p = Pool(lens, ps, 2048, 5, seed=1)
    for extra in (0, 3):
        p.step(new, extra=extra)
        p.step(lens)
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("B", [3, 100])
@pytest.mark.parametrize("rows", [0, 7, 20000])
def test_more_new_rows_than_31_bits(B, rows):
    """Nothing is changed where the new rows pass 2^31 - 1; up to there they are counted."""
    ps = 1 << 30
    lens = [0] * B
    for new, good in [([1 << 30, 1 << 30, 0], False), ([1 << 30] * 3, False), ([1 << 30, (1 << 30) - 1, 1], False),
                      ([1 << 30, (1 << 30) - 1, 0], True), ([1 << 30, 0, (1 << 30) - 2], True)]:
        new = new + [0] * (B - 3)
        p = Pool(lens, ps, 1, B, seed=2)
        indptr, slots = p.resize(new, rows)
        flags = binding.get_device_errors()
        if not good:
            assert flags == binding.DEVERR_SEQLEN
            assert indptr.tolist() == [0] * (B + 1) and bool((slots == -1).all())
            p.same()
            continue
        assert flags == (binding.DEVERR_SLOT if rows else 0)
        assert indptr.tolist() == [sum(new[:b]) for b in range(B + 1)]
        top = p.free[p.count - 2:p.count]
        assert p.gpu[2].item() == p.count - 2
        at = [b for b in range(B) if new[b]]
        want = [-7] * B
        for b, page in zip(at, top):
            want[b] = page
        assert p.gpu[0].view(-1).tolist() == want and p.gpu[1].tolist() == p.free
        assert slots.tolist() == [top[0] * ps + r for r in range(rows)]
