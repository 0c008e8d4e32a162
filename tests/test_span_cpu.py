"""Host side of windowed and tree attention, page tables and commits, without a GPU: plans, split counts, and refusals that
come back with the documented status before CUDA is touched."""
import ctypes

import pytest
import torch

from paged_kv_cache_298_gb300 import binding

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p((1 << 20) + 2)
NULL, SHAPE, UNSUPPORTED, WORKSPACE, ALIGN = 1, 2, 3, 4, 5


def span(tree, **kw):
    a = dict(q=FAKE, qst=32 * 128, qsh=128, k=FAKE, v=FAKE, P=64, ps=16, table=FAKE, maxp=64, lens=FAKE, parents=FAKE,
             qi=FAKE, tb=FAKE, ti=FAKE, tiles=2, tpt=4, total=8, window=100, sinks=4, most=500, B=2, Hq=32, Hkv=8, D=128,
             scale=0.1, S=2, ws=None, wsb=0, out=FAKE, ost=32 * 128, osh=128)
    a.update(kw)
    f = binding.load().decode_attn_paged_tree if tree else binding.load().decode_attn_paged_window
    return f(a["q"], a["qst"], a["qsh"], a["k"], a["v"], a["P"], a["ps"], a["table"], a["maxp"], a["lens"],
             *([a["parents"]] if tree else []), a["qi"], a["tb"], a["ti"], a["tiles"], a["tpt"], a["total"], a["window"],
             a["sinks"], a["most"], a["B"], a["Hq"], a["Hkv"], a["D"], a["scale"], a["S"], a["ws"], a["wsb"], a["out"],
             a["ost"], a["osh"], None)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), SHAPE), (dict(B=0), SHAPE), (dict(total=-1), SHAPE), (dict(total=0), SHAPE), (dict(tiles=0), SHAPE),
    (dict(tiles=9), SHAPE), (dict(tiles=-1), SHAPE), (dict(Hq=31), SHAPE), (dict(Hkv=0), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(window=-1), SHAPE), (dict(sinks=-1), SHAPE), (dict(most=-1), SHAPE), (dict(most=64 * 16 + 1), SHAPE),
    (dict(most=1 << 30, ps=1 << 30), SHAPE), (dict(S=-2), SHAPE), (dict(S=70000), SHAPE), (dict(P=0), SHAPE),
    (dict(ps=0), SHAPE), (dict(maxp=0), SHAPE), (dict(tpt=0), SHAPE), (dict(tpt=3), SHAPE), (dict(tpt=8), SHAPE),
    (dict(tpt=-4), SHAPE), (dict(qst=-8), SHAPE), (dict(qst=0), SHAPE), (dict(osh=0), SHAPE),
    (dict(qi=None, tb=None, ti=None), SHAPE), (dict(qi=None, tb=None, ti=None, total=2), SHAPE),
    (dict(S=-1), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(Hq=24), UNSUPPORTED), (dict(Hq=128), UNSUPPORTED),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL),
    (dict(qi=None), NULL), (dict(tb=None), NULL), (dict(ti=None), NULL), (dict(out=None), NULL),
    (dict(q=ODD), ALIGN), (dict(k=ODD), ALIGN), (dict(v=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(table=ODD), ALIGN),
    (dict(lens=ODD), ALIGN), (dict(qi=ODD), ALIGN), (dict(tb=ODD), ALIGN), (dict(ti=ODD), ALIGN), (dict(qsh=132), ALIGN),
    (dict(ost=4100), ALIGN),
    (dict(), WORKSPACE), (dict(ws=FAKE, wsb=1000), WORKSPACE), (dict(ws=ODD, wsb=1 << 30), WORKSPACE),
])
def test_bad_arguments(tree, kw, status):
    assert span(tree, **kw) == status


def test_arguments_of_one_of_the_two():
    assert span(False, window=0) == SHAPE
    assert span(True, window=0) == WORKSPACE        # (past every check of shapes)
    assert span(True, parents=None) == NULL and span(True, parents=ODD) == ALIGN
    for tree in (False, True):
        assert span(tree, total=0, tiles=0) == 0    # nothing to do


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=0), SHAPE), (dict(P=0), SHAPE), (dict(ps=0), SHAPE), (dict(maxp=0), SHAPE),
    (dict(most=-1), SHAPE), (dict(most=257), SHAPE), (dict(D=12), UNSUPPORTED), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(table=None), NULL), (dict(pos=None), NULL), (dict(path=None), NULL), (dict(n=None), NULL), (dict(k=ODD), ALIGN),
    (dict(v=ODD), ALIGN), (dict(table=ODD), ALIGN), (dict(pos=ODD), ALIGN), (dict(path=ODD), ALIGN), (dict(n=ODD), ALIGN),
    (dict(B=0), 0), (dict(most=0), 0),
])
def test_bad_arguments_of_a_commit(kw, status):
    a = dict(k=FAKE, v=FAKE, P=4, ps=16, table=FAKE, maxp=4, pos=FAKE, path=FAKE, n=FAKE, most=5, B=2, Hkv=2, D=64)
    a.update(kw)
    assert binding.load().kv_commit_paged(a["k"], a["v"], a["P"], a["ps"], a["table"], a["maxp"], a["pos"], a["path"],
                                          a["n"], a["most"], a["B"], a["Hkv"], a["D"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), SHAPE), (dict(maxp=0), SHAPE), (dict(ps=0), SHAPE), (dict(P=0), SHAPE), (dict(rows=-1), SHAPE),
    (dict(bytes=2), SHAPE), (dict(bytes=0), SHAPE), (dict(B=8193), UNSUPPORTED), (dict(B=1 << 13, maxp=(1 << 17) + 1), UNSUPPORTED),
    (dict(bytes=4, P=1 << 20, ps=1 << 11), UNSUPPORTED), (dict(old=None), NULL), (dict(new=None), NULL), (dict(table=None), NULL),
    (dict(free=None), NULL), (dict(count=None), NULL), (dict(indptr=None), NULL), (dict(slots=None), NULL), (dict(old=ODD), ALIGN),
    (dict(new=ODD), ALIGN), (dict(table=ODD), ALIGN), (dict(free=ODD), ALIGN), (dict(count=ODD), ALIGN), (dict(indptr=ODD), ALIGN),
    (dict(slots=ODD), ALIGN), (dict(slots=ctypes.c_void_p((1 << 20) + 4)), ALIGN),
])
def test_bad_arguments_of_a_resize(kw, status):
    a = dict(old=FAKE, new=FAKE, table=FAKE, maxp=8, ps=16, free=FAKE, P=100, count=FAKE, indptr=FAKE, slots=FAKE, bytes=8,
             rows=10, B=2)
    a.update(kw)
    assert binding.load().kv_resize_paged(a["old"], a["new"], a["table"], a["maxp"], a["ps"], a["free"], a["P"], a["count"],
                                          a["indptr"], a["slots"], a["bytes"], a["rows"], a["B"], None) == status


def test_plans():
    p = binding.SpanPlan([1] * 5, 32, 8, 128, "cpu")
    assert p.map is None and (p.B, p.total_q, p.num_tiles, p.tokens_per_tile) == (5, 5, 5, 2)
    p = binding.SpanPlan([1, 0, 3], 32, 8, 128, "cpu")
    assert p.tokens_per_tile == 4 and p.num_tiles == 2
    assert p.map.tolist() == [0, 1, 1, 4] + [0, 2] + [0, 0]
    p = binding.SpanPlan(torch.tensor([2, 2]), 32, 8, 32, "cpu")
    assert p.tokens_per_tile == 2
    assert binding.SpanPlan([], 32, 8, 128, "cpu").total_q == 0
    for bad in (dict(Hq=12, Hkv=4), dict(Hq=16, Hkv=1), dict(Hq=7, Hkv=2)):
        with pytest.raises(ValueError):
            binding.SpanPlan([1], bad["Hq"], bad["Hkv"], 128, "cpu")
    with pytest.raises(ValueError):
        binding.SpanPlan([3, -1], 8, 8, 128, "cpu")


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_tiles_hold_whole_tokens(D, G):
    for n in (0, 1, 2, 8, 9, 16, 17, 100, 5000):
        t = binding.load().dap_span_tokens_per_tile(148, 100, 8 * G, 8, D, n)
        assert t * G in ((8, 16) if D == 32 else (8, 16, 128, 256))
        assert n <= 8 // G or t > 8 // G
    assert binding.load().dap_span_tokens_per_tile(148, 100, 8 * G, 8, D, -1) == 0


def test_split_counts():
    lib = binding.load()

    def splits(tiles=16, tpt=2, most=32768, window=0, sinks=0, tree=0, total=0, S=0, sms=148):
        return lib.dap_span_splits(sms, tiles, 16, 16, 32, 8, 128, tpt, most, window, sinks, tree, total, S)
    assert splits(S=1) == 1 and splits(S=5) == 5
    # what a window leaves is cut, not the length: 128 + 62 + 2 keys, sinks in a tile of their own
    assert splits(window=128, S=100) == 3 and splits(window=128, sinks=4, S=100) == 4
    assert splits(window=1 << 30, S=100) == splits(S=100)
    assert splits(window=128, tree=1, S=100) == 7    # (and up to 256 nodes)
    assert splits(most=0) == 1 and splits(tiles=0) >= 1
    for bad in (dict(tiles=-1), dict(most=-1), dict(window=-1), dict(sinks=-1), dict(S=-1), dict(tpt=0), dict(total=-1)):
        assert splits(**bad) == 0
    plan = binding.SpanPlan([1] * 4, 32, 8, 128, "cpu")
    assert plan.splits(1000, 100, 4, num_splits=1) == 1
    with pytest.raises(ValueError):
        plan.splits(1000, -1, 4)
    n = binding.workspace_bytes_span(plan, max_kv_len=1000, window=100, num_splits=3)
    assert n == binding.workspace_bytes_multi(4, 32, 128, plan.splits(1000, 100, 0, num_splits=3))


def test_the_binding_refuses_before_the_library_sees_a_pointer():
    x = torch.zeros((2, 32, 128), dtype=torch.bfloat16)
    cache = torch.zeros((4, 16, 8, 128), dtype=torch.bfloat16)
    table, lens = torch.zeros((2, 4), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    plan = binding.SpanPlan([1, 1], 32, 8, 128, "cpu")
    with pytest.raises(ValueError):
        binding.decode_attn_paged_window(x, cache, cache, table, lens, plan, window=0, max_kv_len=64)
    with pytest.raises(ValueError):
        binding.decode_attn_paged_tree(x, cache, cache, table, lens, None, plan, max_kv_len=64)
    with pytest.raises(ValueError):
        binding.decode_attn_paged_tree(x, cache, cache, table, lens, lens, binding.SpanPlan([257], 32, 8, 128, "cpu"), max_kv_len=64)
    with pytest.raises(binding.DapError):
        binding.decode_attn_paged_window(x, cache, cache, table, lens, plan, window=5, max_kv_len=64)
    with pytest.raises(binding.DapError):
        binding.kv_commit_paged(cache, cache, table, lens, table, lens)
    with pytest.raises(binding.DapError):
        binding.kv_resize_paged(lens, lens, table, lens, lens[:1], page_size=16)


def test_a_commit_refuses_caches_that_overlap():
    row = 2 * 64 * 2
    for apart, status in ((0, SHAPE), (row, SHAPE), (4 * 16 * row - 16, SHAPE)):
        for k, v in ((0, apart), (apart, 0)):
            assert binding.load().kv_commit_paged(ctypes.c_void_p((1 << 20) + k), ctypes.c_void_p((1 << 20) + v), 4, 16, FAKE, 4,
                                                  FAKE, FAKE, FAKE, 5, 2, 2, 64, None) == status
