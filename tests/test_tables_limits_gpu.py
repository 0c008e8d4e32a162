"""Page tables and commits at the ends of their ranges: lengths and row numbers near 2^31, more new rows than that, and rows whose
bits are no numbers."""
import random

import pytest
import torch

from paged_kv_cache_298_gb300 import binding
from test_tables_gpu import Pool, committed, ints

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


@pytest.mark.parametrize("ps", [1, 16])
def test_rows_move_whatever_their_bits(ps):
    """NaN of every kind, infinities and negative zeros in rows that move, in K and in V."""
    r = random.Random(ps)
    base, paths = [5, 40], [list(range(1, 100)), [3, 4, 9, 30, 31, 32, 77]]
    rows = list(range(2 * -(-160 // ps)))
    r.shuffle(rows)
    rows = [rows[::2], rows[1::2]]
    k, v = (torch.randint(-(1 << 15), 1 << 15, (2 * len(rows[0]), ps, 2, 64), device="cuda").to(torch.int16) for _ in "kv")
    for b, path in enumerate(paths):                          # (each pattern in a row that moves)
        for i, bits in enumerate((0x7FC0, 0x7FBF, 0x7F81, 0x7FFF, 0x7F80, -0x80, -1, -0x7F, -0x8000)):
            at = base[b] + path[i % len(path)]
            k[rows[b][at // ps], at % ps, i % 2], v[rows[b][at // ps], at % ps, 1 - i % 2] = bits, bits
    want = [x.clone() for x in (k, v)]
    for x in want:
        for b, path in enumerate(paths):
            x.copy_(committed(x, rows[b], ps, base[b], path))
    assert not any(torch.equal(x, y) for x, y in zip((k, v), want))
    wide = max(map(len, paths))
    binding.kv_commit_paged(k.view(torch.bfloat16), v.view(torch.bfloat16), ints(rows), ints(base),
                            ints([x + [0] * (wide - len(x)) for x in paths]), ints([len(x) for x in paths]))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    assert binding.get_device_errors() == 0
