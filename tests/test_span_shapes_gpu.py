"""Windowed and tree attention in each kernel shape that the rules pick for large batches: 256 query rows a tile in two streams,
128 rows with two CTAs an SM, tiles ranked by length, and the warp-level kernel's 32-key tiles, at every head dim they have and
with page runs and row gather.  Operators and bounds are span_reference's."""
import pytest
import torch

from paged_kv_cache_298_gb300 import binding
from span_reference import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    binding.get_device_errors(clear=True)
    yield


def call(b, plan, w, sinks, **kw):
    if b.trees is None:
        return binding.decode_attn_paged_window(b.q, b.k, b.v, b.table, b.seq_lens, plan, window=w or b.max_len, sinks=sinks,
                                                max_kv_len=b.max_len, **kw)
    return binding.decode_attn_paged_tree(b.q, b.k, b.v, b.table, b.seq_lens, b.parents, plan, window=w, sinks=sinks,
                                          max_kv_len=b.max_len, **kw)


def check(b, plan, w, sinks, splits, what=()):
    """Calls of these split counts against the operator in 64 bits, found once."""
    ref, bound = b.reference(w, sinks)
    for S in splits:
        got = call(b, plan, w, sinks, num_splits=S)
        assert got.shape == ref.shape and not torch.isnan(got).any(), (*what, w, sinks, S)
        over = ((got.double() - ref).abs() / bound).max().item()
        assert over <= 1.0, (*what, w, sinks, S, over)


def plan_of(b, cols):
    """A plan whose tiles have `cols` query columns."""
    plan = binding.SpanPlan(b.counts, b.Hq, b.Hkv, b.D, "cuda", tokens_per_tile=cols * b.Hkv // b.Hq)
    assert plan.map is not None or cols == 8
    return plan


def hide(b, w, sinks):
    """NaN and infinities where no token sees, no entry for pages without a place that is seen."""
    for q in range(b.B):
        see = b.seen(q, w, sinks).any(0) if b.counts[q] else torch.zeros(b.lens[q], dtype=torch.bool, device="cuda")
        page, slot = b.places(q, b.lens[q])
        b.k[page[~see], slot[~see]] = float("inf")
        b.v[page[~see], slot[~see]] = float("nan")
        for e in range(-(-b.lens[q] // b.ps)):
            if not see[e * b.ps:(e + 1) * b.ps].any():
                b.table[q, e] = -1


def wide_counts(G):
    """Tiles of one token, of one stream's rows and one less or more, of all rows, and a second tile."""
    half = 128 // G
    return [1, half - 1, half, half + 1, 2 * half - 1, 2 * half, min(256, 2 * half + 5), 0]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ps", [12, 16, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("kind", [None, "chain", "mixed", "roots"])
def test_two_streams(D, ps, G, kind):
    counts = wide_counts(G)
    b = Batch([0, 3, 64, 130, 517, 63, 300, 40], counts, 2 * G, 2, D, ps, seed=G, kind=kind)
    plan = plan_of(b, 256)
    for w, sinks in [(0, 0), (1, 0), (70, 65), (100, 5), (300, 0)]:
        check(b, plan, w, sinks, (0, 1, 3))
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ps", [5, 16, 128])
@pytest.mark.parametrize("kind", [None, "mixed"])
def test_two_streams_over_what_no_token_sees(D, ps, kind):
    for G, sinks in ((1, 0), (4, 4), (8, 70)):
        b = Batch([700, 391, 66, 1500], [256 // G, 128 // G + 1, 128 // G, 1], 2 * G, 2, D, ps, seed=1, kind=kind)
        plan = plan_of(b, 256)
        want = call(b, plan, 100, sinks)
        b.check(want, 100, sinks)
        hide(b, 100, sinks)
        check(b, plan, 100, sinks, (0, 1, 3), what=(G,))
        for _ in range(3):
            assert torch.equal(call(b, plan, 100, sinks), want)
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("ps", [12, 16])
def test_two_streams_padding_bad_pages_and_lengths(ps):
    n = 40                                                    # 160 rows: the second stream in part
    for kind in (None, "mixed"):
        b = Batch([200, 0, 90, 0], [n] * 4, 8, 2, 128, ps, seed=6, kind=kind)
        plan = plan_of(b, 256)
        want = call(b, plan, 50, 3).clone()
        b.check(want, 50, 3)
        b.seq_lens[1] = b.seq_lens[3] = 0
        table, b.table = b.table, b.table.clone()
        b.table[1] = b.table[3] = -1
        for S in (0, 1, 3):
            got = call(b, plan, 50, 3, num_splits=S)
            assert (got[n:2 * n] == 0).all() and (got[3 * n:] == 0).all()
            if S == 0:
                assert torch.equal(got[:n], want[:n]) and torch.equal(got[2 * n:3 * n], want[2 * n:3 * n])
        assert binding.get_device_errors() == 0
        b.table = table
        b.seq_lens[:] = torch.tensor(b.lens, dtype=torch.int32)
        last = (b.lens[2] - 1) // ps
        page, b.table[2, last] = int(b.table[2, last]), b.pool + 7
        got = call(b, plan, 50, 3)
        assert binding.get_device_errors() & binding.DEVERR_PAGE
        assert torch.equal(got[:2 * n], want[:2 * n]) and torch.equal(got[3 * n:], want[3 * n:])
        b.table[2, last] = page
        b.seq_lens[0] = -3
        got = call(b, plan, 50, 3)
        assert binding.get_device_errors() & binding.DEVERR_SEQLEN
        assert (got[:n] == 0).all() and torch.equal(got[n:], want[n:])
        b.seq_lens[0] = b.lens[0]
        assert torch.equal(call(b, plan, 50, 3), want) and binding.get_device_errors() == 0


def test_two_streams_replayed():
    b = Batch([500, 300, 71], [33, 64, 50], 8, 2, 128, 16, seed=8, kind="mixed")
    c = Batch([420, 499, 0], [33, 64, 50], 8, 2, 128, 16, seed=9, kind="chain")
    plan = plan_of(b, 256)
    pool, width = max(b.pool, c.pool), max(b.table.shape[1], c.table.shape[1])
    k, v = (torch.zeros((pool, 16, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    table = torch.zeros((3, width), dtype=torch.int32, device="cuda")
    q, lens, parents = torch.empty_like(b.q), torch.empty_like(b.seq_lens), torch.empty_like(b.parents)
    bound = max(b.max_len, c.max_len)
    ws = torch.empty(binding.workspace_bytes_span(plan, max_kv_len=bound, tree=True, num_splits=3), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]

    def load(x):
        table[:, :x.table.shape[1]] = x.table
        k[:x.pool], v[:x.pool] = x.k, x.v
        q.copy_(x.q)
        lens.copy_(x.seq_lens)
        parents.copy_(x.parents)

    def calls():
        for out, S in zip(outs, (1, 3)):
            binding.decode_attn_paged_tree(q, k, v, table, lens, parents, plan, max_kv_len=bound, num_splits=S, workspace=ws, out=out)
    load(b)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for x in (b, c, b):
        load(x)
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        graph.replay()
        for o in outs:
            x.check(o)
    assert binding.get_device_errors() == 0


def at_least(b, cols, ctas, S=1):
    """A plan of `cols` columns whose CTAs pass `ctas`."""
    plan = plan_of(b, cols)
    assert plan.num_tiles * b.Hkv * S > ctas
    return plan


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ps", [12, 16, 64])
@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("kind", [None, "mixed"])
def test_128_rows_with_two_ctas_an_sm(D, ps, G, kind):
    sms, Hkv = binding.device_sm_count(), 8
    counts = [(17 * i) % (128 // G) + 1 + (128 // G if i % 5 == 0 else 0) for i in range(24)]
    b = Batch([(37 * i) % 400 for i in range(24)], counts, G * Hkv, Hkv, D, ps, seed=G, kind=kind)
    plan = at_least(b, 128, sms)
    for w, sinks in [(0, 0), (1, 1), (70, 65), (130, 0)]:
        check(b, plan, w, sinks, (0, 1, 2))
    hide(b, 100, 4)
    check(b, plan, 100, 4, (1, 2))
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("D,cols", [(64, 128), (128, 128), (256, 128), (64, 256), (128, 256)])
@pytest.mark.parametrize("ps", [12, 16])
def test_tiles_ranked_by_length(D, cols, ps):
    """More CTAs than run at once, of unequal lengths and without a window: 2, 100 and 128 work tiles are ranked, 129 not."""
    sms = binding.device_sm_count()
    for tiles, Hkv, S in ((2, 8, 40), (100, 8, 1), (128, 8, 1), (129, 8, 1), (50, 8, 3)):
        if tiles == 2:
            ctx = [2600, 2900]
        else:
            ctx = [0 if i % 9 == 0 else 20 + (i * 131) % 700 for i in range(tiles)]
        n = [1 + (7 * i) % (cols // 4) for i in range(tiles)]
        b = Batch(ctx, n, 4 * Hkv, Hkv, D, ps, seed=tiles, kind="mixed")
        plan = plan_of(b, cols)
        S = plan.splits(b.max_len, tree=True, num_splits=S)
        assert plan.num_tiles == tiles and tiles * Hkv * S > 2 * sms
        b.check(call(b, plan, 0, 0, num_splits=S), what=(tiles, S))
        if tiles == 100:                                      # (an entry that names nothing is ranked last, and flagged)
            want = call(b, plan, 0, 0, num_splits=1)
            plan.map[b.B + 1 + 3] = -1
            out = torch.full_like(want, 9.0)
            call(b, plan, 0, 0, num_splits=1, out=out)
            at = sum(n[:3])
            assert (out[at:at + n[3]] == 9.0).all()
            assert torch.equal(out[:at], want[:at]) and torch.equal(out[at + n[3]:], want[at + n[3]:])
            assert binding.get_device_errors() & binding.DEVERR_QMAP
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("ps", [12, 16, 64])
@pytest.mark.parametrize("G,cols", [(1, 8), (4, 8), (8, 8), (1, 16), (4, 16), (8, 16)])
def test_32_key_tiles(D, ps, G, cols):
    sms, Hkv, B = binding.device_sm_count(), 8, 48
    for kind in (None, "mixed"):
        counts = [1 + i % (cols // G) for i in range(B)]
        b = Batch([(41 * i) % 500 for i in range(B)], counts, G * Hkv, Hkv, D, ps, seed=G, kind=kind)
        plan = at_least(b, cols, 2 * sms)
        for w, sinks in [(0, 0), (1, 0), (33, 31), (70, 65), (128, 4)]:
            check(b, plan, w, sinks, (0, 1, 3), what=(kind,))
        hide(b, 100, 4)
        check(b, plan, 100, 4, (1, 3), what=(kind,))
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_32_key_tiles_without_a_map(D):
    sms, Hkv, B = binding.device_sm_count(), 8, 64
    b = Batch([(97 * i) % 1500 for i in range(B)], [1] * B, 4 * Hkv, Hkv, D, 16, seed=3)
    plan = binding.SpanPlan(b.counts, b.Hq, Hkv, D, "cuda")
    assert plan.map is None and B * Hkv > 2 * sms
    for w, sinks in [(1024, 4), (200, 0)]:
        b.check(call(b, plan, w, sinks), w, sinks)
    b.seq_lens[5:9] = 0                                       # padding
    b.table[5:9] = -1
    got = call(b, plan, 1024, 4)
    assert (got[5:9] == 0).all() and binding.get_device_errors() == 0
