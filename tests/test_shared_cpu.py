"""Host side of the shared-prefix decode, without a GPU: the work map, the planner, the workspace, and
refusals that come back with the documented status before CUDA is touched."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_298_gb300 import binding

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p((1 << 20) + 2)
NULL, SHAPE, UNSUPPORTED, WORKSPACE, ALIGN = 1, 2, 3, 4, 5


def call(**kw):
    a = dict(q=FAKE, qsb=32 * 128, qsh=128, k=FAKE, v=FAKE, P=64, ps=16, table=FAKE, maxp=64, lens=FAKE, plens=FAKE,
             sg=FAKE, tl=FAKE, groups=1, tiles=1, spt=64, maxpre=500, maxsuf=100, B=4, Hq=32, Hkv=8, D=128,
             scale=0.1, pre=2, suf=1, ws=None, wsb=0, out=FAKE, osb=32 * 128, osh=128)
    a.update(kw)
    return binding.load().decode_attn_paged_shared(
        a["q"], a["qsb"], a["qsh"], a["k"], a["v"], a["P"], a["ps"], a["table"], a["maxp"], a["lens"], a["plens"],
        a["sg"], a["tl"], a["groups"], a["tiles"], a["spt"], a["maxpre"], a["maxsuf"], a["B"], a["Hq"], a["Hkv"],
        a["D"], a["scale"], a["pre"], a["suf"], a["ws"], a["wsb"], a["out"], a["osb"], a["osh"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), SHAPE), (dict(Hq=31), SHAPE), (dict(Hkv=0), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(scale=float("inf")), SHAPE), (dict(pre=-1), SHAPE), (dict(suf=-1), SHAPE), (dict(pre=70000), SHAPE),
    (dict(suf=70000), SHAPE), (dict(maxpre=-1), SHAPE), (dict(maxsuf=-1), SHAPE), (dict(maxpre=64 * 16 + 1), SHAPE),
    (dict(maxsuf=64 * 16 + 1), SHAPE), (dict(P=0), SHAPE), (dict(ps=0), SHAPE), (dict(maxp=0), SHAPE), (dict(groups=0), SHAPE),
    (dict(tiles=0), SHAPE), (dict(tiles=5), SHAPE), (dict(spt=32), SHAPE), (dict(spt=0), SHAPE), (dict(qsb=-8), SHAPE),
    (dict(qsb=0), SHAPE), (dict(osh=0), SHAPE),
    (dict(D=32, qsb=1024, qsh=32), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(Hq=24), UNSUPPORTED),
    (dict(Hq=128, spt=16), UNSUPPORTED),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL),
    (dict(plens=None), NULL), (dict(sg=None), NULL), (dict(tl=None), NULL),
    (dict(out=None), NULL),
    (dict(q=ODD), ALIGN), (dict(k=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(table=ODD), ALIGN), (dict(plens=ODD), ALIGN),
    (dict(sg=ODD), ALIGN), (dict(tl=ODD), ALIGN), (dict(tl=ctypes.c_void_p((1 << 20) + 4)), ALIGN), (dict(qsh=132), ALIGN),
    (dict(osb=4100), ALIGN),
    (dict(), WORKSPACE), (dict(ws=FAKE, wsb=1000), WORKSPACE), (dict(ws=ODD, wsb=1 << 30), WORKSPACE),
])
def test_bad_arguments(kw, status):
    assert call(**kw) == status


def test_an_empty_batch_is_nothing_to_do():
    assert call(B=0) == 0


def test_map_covers_every_sequence_once():
    for sizes in ([1], [64], [65], [3, 0, 200, 1], [0, 5], [128, 128]):
        plan = binding.SharedPlan(sizes, 32, 8, 128, "cpu")
        assert plan.seqs_per_tile == 64 and plan.B == sum(sizes)
        assert plan.seq_group.tolist() == [g for g, n in enumerate(sizes) for _ in range(n)]
        starts = [0] + list(np.cumsum(sizes))
        seen = []
        for g, q0, a, n in plan.tiles.tolist():
            assert q0 == starts[g] and 1 <= n <= 64 and (a - q0) % 64 == 0 and a + n <= starts[g + 1]
            seen += list(range(a, a + n))
        assert seen == list(range(sum(sizes)))


def test_plan_refuses():
    for sizes, Hq, Hkv, D in (([], 32, 8, 128), ([-1, 2], 32, 8, 128), ([2], 24, 8, 128), ([2], 32, 8, 32), ([2], 33, 8, 128)):
        with pytest.raises(ValueError):
            binding.SharedPlan(sizes, Hq, Hkv, D, "cpu")
    assert binding.load().dap_shared_seqs_per_tile(64, 8, 256) == 16
    assert binding.load().dap_shared_seqs_per_tile(8, 8, 64) == 256
    # the map without room for its tiles
    n = torch.tensor([100], dtype=torch.int32)
    out = [torch.zeros(200, dtype=torch.int32) for _ in range(2)]
    f = binding.load().dap_shared_map
    assert f(n.data_ptr(), 1, 64, out[0].data_ptr(), out[1].data_ptr(), 1) == -1
    assert f(n.data_ptr(), 1, 64, out[0].data_ptr(), out[1].data_ptr(), 2) == 2
    assert f(n.data_ptr(), 1, 0, out[0].data_ptr(), out[1].data_ptr(), 200) == -1
    assert f(n.data_ptr(), 1, 64, None, out[1].data_ptr(), 2) == -1 and f(None, 1, 64, out[0].data_ptr(), out[1].data_ptr(), 2) == -1


def plan(tiles, B, Hq, Hkv, D, pre, suf, total=0, sms=152, want=(0, 0)):
    a, b = ctypes.c_int(want[0]), ctypes.c_int(want[1])
    r = binding.load().dap_shared_plan(sms, tiles, B, Hq, Hkv, D, pre, suf, total, ctypes.byref(a), ctypes.byref(b))
    return (a.value, b.value) if r == 0 else None


def test_plan_covers_both_parts():
    for tiles, B, Hq, Hkv, D in ((1, 1, 8, 1, 128), (1, 16, 32, 8, 128), (2, 128, 32, 8, 128), (8, 64, 64, 8, 256), (40, 2000, 32, 8, 64)):
        for P in (0, 1, 63, 64, 65, 1000, 8192, 32768, 10 ** 6):
            for L in (0, 1, 64, 500, 30000):
                for total in (0, B * L // 2):
                    S, T = plan(tiles, B, Hq, Hkv, D, P, L, total)
                    assert (S == 0) == (P == 0) and (T == 0) == (L == 0)
                    assert P == 0 or (S <= -(-P // 64) and S * binding.chunk_tokens(P, S) >= P)
                    assert L == 0 or (T <= -(-L // 64) and T * binding.chunk_tokens(L, T) >= L)
    # explicit counts are kept, lowered where they cannot be filled
    assert plan(2, 128, 32, 8, 128, 8192, 1024, want=(5, 3)) == (5, 3)
    assert plan(2, 128, 32, 8, 128, 130, 10, want=(50, 3)) == (3, 1)
    # a prefix alone fills the device; beside a large suffix it leaves SMs to it
    alone, _ = plan(2, 128, 32, 8, 128, 8192, 0)
    beside, _ = plan(2, 128, 32, 8, 128, 8192, 1024, 64000)
    assert 7 <= alone <= 9 and beside < alone
    for bad in ((-1, 4, 8, 2, 64, 10, 10), (1, -4, 8, 2, 64, 10, 10), (1, 4, 9, 2, 64, 10, 10), (1, 4, 8, 2, 64, -1, 10), (1, 4, 8, 2, 64, 10, -1)):
        assert plan(*bad) is None
    assert plan(1, 4, 8, 2, 64, 10, 10, want=(-1, 0)) is None
    assert plan(1, 4, 8, 2, 64, 10, 10, sms=0) == (1, 1)


def test_bounds_up_to_32_bits():
    p = binding.SharedPlan([2], 8, 2, 64, "cpu")
    for n in (2 ** 31 - 1, 2 ** 31 - 64, 2 ** 30 + 1):
        assert min(p.splits(64, n, prefix_splits=1, suffix_splits=1)) == 1
    with pytest.raises(ValueError):
        p.splits(-1, 64)


def test_workspace():
    w = binding.load().dap_workspace_bytes_shared
    assert w(4, 32, 128, 0, 0) == 0
    assert w(4, 32, 128, 2, 1) >= 4 * 3 * 32 * 130 * 4
    assert w(0, 32, 128, 2, 1) == 0 and w(4, 32, 128, -1, 1) == 0
