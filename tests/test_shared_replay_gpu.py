"""Shared-prefix decode: captured calls replayed with other lengths and prefixes, against plain attention on those; and the same
bits from call to call.  Case and its tolerance are test_shared_gpu's."""
import threading

import pytest
import torch

from paged_kv_cache_298_gb300 import binding
from test_shared_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    binding.get_device_errors(clear=True)
    yield


def test_two_groups_replayed_with_a_shorter_prefix():
    """Two captured steps on one workspace; the second has two groups, D = 256, and is replayed with a prefix of 180 instead of
    200 and lengths down to it.  Positions 192 .. 199 lie in each sequence's own page, which holds a copy of the first one's
    rows here, so that what a sequence reads behind the shorter prefix is defined and the result is compared with plain
    attention over the lengths and prefixes of the replay."""
    a = Case([30], [400], [17] * 30, 8, 2, 128, 16, seed=1)
    b = Case([7, 5], [200, 333], [50] * 12, 16, 2, 256, 16, seed=2)
    page = b.table[:7, 12].long()
    for x in (b.k, b.v):
        assert bool(x[page[1:], :8].isnan().all())
        x[page[1:], :8] = x[page[0], :8].clone()
    kw = dict(max_prefix_len=450, max_suffix_len=70)
    ws = torch.empty(max(binding.workspace_bytes_shared(c.plan, **kw) for c in (a, b)), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    side = torch.cuda.Stream()
    for c in (a, b):
        c.table = torch.cat([c.table, torch.full((c.B, 8), -1, dtype=torch.int32, device="cuda")], dim=1).contiguous()
        out = torch.zeros_like(c.q)
        c.run(workspace=ws, out=out, **kw)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c.run(workspace=ws, out=out, **kw)
        outs.append(out)
        graphs.append(g)
    for step, (prefix, lens) in enumerate(((180, [180, 181, 190, 195, 250, 200, 0]), (200, [200, 201, 250, 0, 219, 249, 240]),
                                           (0, [1, 0, 64, 191, 30, 16, 70]))):
        a.lens -= 3 * (a.lens > 0).to(torch.int32)
        a.lens[4 + step] = 0
        b.prefix[0] = prefix
        b.lens[:7] = torch.tensor(lens, dtype=torch.int32)
        if prefix == 0:   # (70 keys at most behind the prefix)
            b.lens[:7] = b.lens[:7].clamp(max=70)
        refs = [c.plain() for c in (a, b)]
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(5):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for c, o, r, what in zip((a, b), outs, refs, "ab"):
            c.check(o, r, f"{what}, step {step}")
        assert binding.get_device_errors() == 0


SHAPES = [
    # sizes, prefixes, lengths behind the prefix, Hq, Hkv, D, page size
    ([2], [128], [5, 70], 8, 2, 64, 16),
    ([16], [2048], [25 * i for i in range(16)], 32, 8, 128, 16),
    ([128], [1500], [8 * i for i in range(128)], 32, 8, 128, 16),
    ([64], [3000], [1, 600] * 32, 64, 8, 128, 64),
    ([20, 9, 12], [1001, 700, 900], [12 * i for i in range(41)], 16, 4, 256, 12),
    ([70, 60], [900, 333], [40] * 130, 8, 2, 256, 32),
]


@pytest.mark.parametrize("sizes,prefixes,suffix,Hq,Hkv,D,ps", SHAPES, ids=[f"B{sum(s[0])}_P{s[1][0]}_D{s[5]}_ps{s[6]}" for s in SHAPES])
def test_the_same_bits_every_time(sizes, prefixes, suffix, Hq, Hkv, D, ps):
    """No result depends on which CTA or warp comes first: repeated calls, alone, in a row and beside other work on another
    stream, give the same bits (the first of them is checked against plain attention)."""
    c = Case(sizes, prefixes, suffix, Hq, Hkv, D, ps, seed=8)
    first = c.run()
    c.check(first, c.plain())
    other = torch.randn((2048, 2048), device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(60):
        if i % 3 == 1:
            with torch.cuda.stream(side):
                other @ other
        out = c.run()
        if i % 3 == 2:
            torch.cuda.synchronize()
        assert torch.equal(out, first), f"call {i}"
    assert binding.get_device_errors() == 0


def test_two_threads_at_once():
    """Two host threads with a stream each, the lock of the interpreter being released inside a call: one plan for both, whose
    bounds (and so its kept split counts) differ from call to call."""
    c = Case([20], [300], [7 * j for j in range(20)], 8, 2, 128, 16, seed=9)
    bounds = [dict(max_prefix_len=300 + 4 * i, max_suffix_len=133 + 70 * i) for i in range(2)]
    c.table = torch.cat([c.table, torch.full((20, 8), -1, dtype=torch.int32, device="cuda")], dim=1).contiguous()
    want = [c.run(**b) for b in bounds]
    torch.cuda.synchronize()
    results, errors = [[], []], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for n in range(100):
                results[i].append((n % 2, c.run(stream=stream, **bounds[n % 2])))
            stream.synchronize()
        except Exception as e:   # noqa: BLE001 (shown by the assert below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for r in results:
        assert len(r) == 100 and all(torch.equal(o, want[k]) for k, o in r)
    assert binding.get_device_errors() == 0
