"""Windowed and tree attention on the GPU against the operators in 64 bits (span_reference.py has the bounds)."""
import random

import pytest
import torch

from paged_kv_cache_298_gb300 import binding
from span_reference import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    binding.get_device_errors(clear=True)
    yield


def plan_of(b):
    return binding.SpanPlan(b.counts, b.Hq, b.Hkv, b.D, "cuda")


def window(b, w, sinks, **kw):
    kw.setdefault("plan", plan_of(b))
    return binding.decode_attn_paged_window(b.q, b.k, b.v, b.table, b.seq_lens, kw.pop("plan"), window=w, sinks=sinks,
                                            max_kv_len=kw.pop("max_kv_len", b.max_len), **kw)


def tree(b, w=0, sinks=0, **kw):
    kw.setdefault("plan", plan_of(b))
    return binding.decode_attn_paged_tree(b.q, b.k, b.v, b.table, b.seq_lens, b.parents, kw.pop("plan"), window=w,
                                          sinks=sinks, max_kv_len=kw.pop("max_kv_len", b.max_len), **kw)


HEADS = [(1, 1), (2, 1), (8, 2), (8, 1), (12, 3)]


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("ps", [1, 5, 8, 12, 16, 64, 100, 128])
def test_window_one_token(D, ps):
    for i, (Hq, Hkv) in enumerate(HEADS):
        b = Batch([0, 1, 15, 16, 63, 64, 65, 127, 200, 511, 900], [1] * 11, Hq, Hkv, D, ps, seed=ps + i)
        for w, sinks in [(1, 0), (1, 1), (2, 0), (16, 4), (63, 0), (64, 64), (65, 65), (128, 0), (100, 200), (300, 3),
                         (5000, 7)]:
            for S in (0, 1, 3):
                b.check(window(b, w, sinks, num_splits=S), w, sinks, what=(Hq, Hkv, w, sinks, S))
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("ps", [5, 16, 64])
def test_window_many_tokens(D, ps):
    for i, (Hq, Hkv) in enumerate(HEADS):
        for n in (2, 3, 17, 70):
            b = Batch([0, 1, 64, 130, 517], [n, 1, n, n - 1, 0], Hq, Hkv, D, ps, seed=n + i)
            for w, sinks in [(1, 0), (2, 1), (16, 4), (64, 64), (70, 0), (129, 66), (4000, 0)]:
                for S in (0, 1, 2):
                    b.check(window(b, w, sinks, num_splits=S), w, sinks, what=(Hq, Hkv, n, w, sinks, S))
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("ps", [5, 16, 64])
@pytest.mark.parametrize("kind", ["chain", "star", "roots", "mixed"])
def test_tree(D, ps, kind):
    for i, (Hq, Hkv) in enumerate(HEADS):
        for n in (1, 2, 7, 33):
            b = Batch([0, 1, 40, 64, 333], [n, 1, n, max(0, n - 1), 0], Hq, Hkv, D, ps, seed=n + i, kind=kind)
            for w, sinks in [(0, 0), (1, 0), (3, 2), (64, 1), (70, 65)]:
                for S in (0, 1, 2):
                    b.check(tree(b, w, sinks, num_splits=S), w, sinks, what=(Hq, Hkv, n, w, sinks, S))
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("kind", ["chain", "mixed", "roots"])
@pytest.mark.parametrize("Hq,Hkv,D,ps", [(8, 2, 128, 16), (4, 4, 64, 12), (8, 1, 256, 64), (2, 2, 128, 64), (8, 4, 32, 16)])
def test_large_trees(kind, Hq, Hkv, D, ps):
    """Up to 256 nodes, several tiles a tree, contexts that end inside and at the ends of tiles."""
    b = Batch([64, 1000, 63, 0, 129], [256, 255, 130, 256, 64], Hq, Hkv, D, ps, seed=3, kind=kind)
    for w, sinks in [(0, 0), (100, 5), (300, 0)]:
        for S in (0, 1, 4):
            b.check(tree(b, w, sinks, num_splits=S), w, sinks, what=(w, sinks, S))
    assert binding.get_device_errors() == 0


def test_random_batches():
    r = random.Random(7)
    for i in range(60):
        Hkv, G, D, ps = r.choice([1, 2, 3, 8]), r.choice([1, 2, 4, 8]), r.choice([32, 64, 128, 256]), r.choice(
            [1, 5, 8, 12, 16, 24, 32, 64, 100, 128])
        B = r.randint(1, 9)
        tree_case = r.random() < 0.5
        most = r.choice([1, 2, 5, 16, 40, 90, 200])
        ctx = [r.choice([0, r.randint(0, 70), r.randint(0, 900)]) for _ in range(B)]
        counts = [r.choice([0, 1, most, r.randint(0, most)]) for _ in range(B)]
        b = Batch(ctx, counts, G * Hkv, Hkv, D, ps, seed=i, kind="mixed" if tree_case else None, qmag=r.choice([0.1, 1, 4]))
        w = r.choice([0, 0, r.randint(1, 1000)]) if tree_case else r.randint(1, 1000)
        sinks = r.choice([0, 4, r.randint(0, 200)]) if w else 0
        S = r.choice([0, 0, 1, 2, 7])
        got = tree(b, w, sinks, num_splits=S, total_kv=sum(b.lens)) if tree_case else window(b, w, sinks, num_splits=S)
        b.check(got, w, sinks, what=(i, ctx, counts, G, Hkv, D, ps, w, sinks, S))
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("ps", [12, 16])
def test_a_long_context(n, ps):
    """Only what a window reaches is read, at places far behind the first page."""
    b = Batch([70001, 33333], [n, n], 8, 2, 128, ps, seed=5)
    for w, sinks in [(1000, 4), (8192, 0)]:
        for S in (0, 1, 5):
            b.check(window(b, w, sinks, num_splits=S), w, sinks, what=(w, sinks, S))
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("ps", [5, 16, 128])
@pytest.mark.parametrize("n", [1, 5, 60])
@pytest.mark.parametrize("sinks", [0, 4, 70])
def test_what_no_token_sees_may_be_gone(ps, n, sinks):
    """Pages between the sinks and the window have no entry any more, and rows that no token sees hold NaN or infinities."""
    for kind in (None, "mixed"):
        b = Batch([700, 391, 66], [n, n, n], 8, 2, 128, ps, seed=1, kind=kind)
        w = 100
        call = window if kind is None else tree
        want = call(b, w, sinks)
        b.check(want, w, sinks)
        for q, c in enumerate(b.ctx):
            see = b.seen(q, w, sinks).any(0)
            page, slot = b.places(q, b.lens[q])
            hidden = ~see
            b.k[page[hidden], slot[hidden]] = float("inf")
            b.v[page[hidden], slot[hidden]] = float("nan")
            for e in range(-(-b.lens[q] // ps)):
                if not see[e * ps:(e + 1) * ps].any():
                    b.table[q, e] = -1
        for S in (0, 1, 2):
            b.check(call(b, w, sinks, num_splits=S), w, sinks, what=(kind, S))
        assert torch.equal(call(b, w, sinks), want)
    assert binding.get_device_errors() == 0


def test_equals_the_causal_call_without_a_window():
    """A window that reaches everything, and a chain, are the causal multi-token decode (within both calls' bounds)."""
    for n in (3, 50):
        b = Batch([300, 17], [n, n], 8, 2, 128, 16, seed=2, kind="chain")
        other = binding.decode_attn_paged_multi(b.q, b.k, b.v, b.table, b.seq_lens,
                                                binding.MultiPlan(b.counts, 8, 2, "cuda", D=128), max_kv_len=b.max_len)
        b.check(other)
        b.check(tree(b))
        b.check(window(b, 10 ** 9, 0))


def test_strided_views_and_given_buffers():
    for n, D in [(1, 128), (5, 64), (40, 128), (40, 256)]:
        b = Batch([100, 300], [n, n], 8, 2, D, 16, seed=4, kind="mixed")
        wide = torch.full((b.total, 16, 2 * D), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 4:12, :D] = b.q
        q = b.q
        out = torch.full((b.total + 2, 12, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        b.q = wide[:, 4:12, :D]
        for S in (1, 3):
            view = out[1:-1, 2:10, :D]
            assert tree(b, out=view, num_splits=S) is not None
            got = view.clone()
            b.q = q
            b.check(got)
            b.q = wide[:, 4:12, :D]
            view.fill_(7.0)
            assert (out == 7.0).all()   # nothing beside the view was written


@pytest.mark.parametrize("n,D", [(1, 64), (3, 128), (40, 128), (40, 256), (60, 64)])
def test_heads_further_apart_than_tokens(n, D):
    b = Batch([100, 300], [n, n], 8, 2, D, 16, seed=4, kind="mixed")
    want = tree(b)
    b.check(want)
    b.q = b.q.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty((8, b.total, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    assert torch.equal(tree(b, out=out), want)


@pytest.mark.parametrize("n", [1, 3, 40])
def test_padding_of_a_batch(n):
    """Sequences of length 0 give zero rows and no error, whatever their tables and q hold."""
    for kind in (None, "mixed"):
        b = Batch([200, 0, 90, 0], [n] * 4, 8, 2, 128, 16, seed=6, kind=kind)
        call = window if kind is None else tree
        want = call(b, 50, 3).clone()
        b.seq_lens[1] = b.seq_lens[3] = 0
        b.table[1] = b.table[3] = -1
        b.q[n:2 * n] = float("nan")
        for S in (0, 1, 3):
            got = call(b, 50, 3, num_splits=S)
            assert (got[n:2 * n] == 0).all() and (got[3 * n:] == 0).all()
            if S == 0:
                assert torch.equal(got[:n], want[:n]) and torch.equal(got[2 * n:3 * n], want[2 * n:3 * n])
    assert binding.get_device_errors() == 0


def test_errors_are_flagged_and_kept_in_bounds():
    for n in (1, 40):
        b = Batch([200, 90], [n, n], 8, 2, 128, 16, seed=6, kind="chain")
        want = tree(b)
        b.table[0, 3] = b.pool + 5           # a page outside the pool
        tree(b)
        assert binding.get_device_errors() & binding.DEVERR_PAGE
        b.table[0, 3] = b.rows[0][3]
        b.seq_lens[1] = b.max_len + 50       # a length past its bound
        got = tree(b)
        assert binding.get_device_errors() & binding.DEVERR_SEQLEN
        assert torch.equal(got[:n], want[:n])
        b.seq_lens[1] = b.lens[1]
        b.seq_lens[0] = -3
        got = tree(b)
        assert binding.get_device_errors() & binding.DEVERR_SEQLEN
        assert (got[:n] == 0).all() and torch.equal(got[n:], want[n:])
        b.seq_lens[0] = b.lens[0]
        assert torch.equal(tree(b), want) and binding.get_device_errors() == 0
    # parents that are no earlier node count as children of the context
    b = Batch([50, 60], [40, 3], 8, 2, 128, 16, seed=6, kind="roots")
    b.check(tree(b))
    b.parents[5], b.parents[7], b.parents[40] = 5, 1000, -2
    b.check(tree(b))
    assert binding.get_device_errors() & binding.DEVERR_TREE
    # more new tokens than places: the tokens in front of the cache give zero rows
    b = Batch([0], [40], 8, 2, 128, 16, seed=6)
    b.seq_lens[0] = 30
    got = window(b, 100, 0)
    assert binding.get_device_errors() & binding.DEVERR_SEQLEN
    assert (got[:10] == 0).all() and torch.isfinite(got).all() and (got[10:] != 0).any()


def test_a_map_that_names_nothing_is_flagged():
    for n in (3, 40):
        b = Batch([200, 90], [n, n], 8, 2, 128, 16, seed=6, kind="chain")
        plan = plan_of(b)
        want = tree(b, plan=plan)
        tiles = plan.map[b.B + 1:b.B + 1 + plan.num_tiles]
        kept = tiles.clone()
        for bad in (-1, b.B, 1 << 30):
            tiles[0] = bad
            out = torch.full_like(want, 9.0)
            tree(b, plan=plan, out=out)   # (with several splits the rows that no entry names are undefined)
            assert binding.get_device_errors() & binding.DEVERR_QMAP
            assert torch.equal(out[n:], want[n:])
            out.fill_(9.0)
            tree(b, plan=plan, out=out, num_splits=1)
            assert binding.get_device_errors() & binding.DEVERR_QMAP
            assert (out[0] == 9.0).all()
            tiles.copy_(kept)
        assert torch.equal(tree(b, plan=plan), want) and binding.get_device_errors() == 0


def test_nothing_to_do():
    b = Batch([5, 0], [0, 0], 8, 2, 128, 16)
    b.parents = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert tree(b).shape == (0, 8, 128) and window(b, 3, 0).shape == (0, 8, 128)
    assert binding.get_device_errors() == 0


def test_captured_and_replayed_with_other_lengths_and_trees():
    for n in (1, 6, 40):
        b = Batch([500, 300], [n, n], 8, 2, 128, 16, seed=8, kind="mixed")
        c = Batch([420, 499], [n, n], 8, 2, 128, 16, seed=9, kind="mixed")
        plan, bound = plan_of(b), 640
        st = torch.cuda.Stream()
        width = max(b.table.shape[1], c.table.shape[1])
        pool = max(b.pool, c.pool)
        table = torch.zeros((2, 60), dtype=torch.int32, device="cuda")
        k, v = (torch.zeros((pool, 16, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q, lens, parents = torch.empty_like(b.q), torch.empty_like(b.seq_lens), torch.empty_like(b.parents)

        def load(x):
            table[:, :x.table.shape[1]] = x.table
            k[:x.pool], v[:x.pool] = x.k, x.v
            q.copy_(x.q)
            lens.copy_(x.seq_lens)
            parents.copy_(x.parents)
        load(b)
        ws = torch.empty(max(1, binding.workspace_bytes_span(plan, max_kv_len=bound, tree=True)), dtype=torch.uint8, device="cuda")
        outs = [torch.empty_like(q) for _ in range(2)]

        def calls():
            binding.decode_attn_paged_tree(q, k, v, table, lens, parents, plan, max_kv_len=bound, workspace=ws, out=outs[0])
            binding.decode_attn_paged_window(q, k, v, table, lens, plan, window=77, sinks=3, max_kv_len=bound, out=outs[1])
        with torch.cuda.stream(st):
            calls()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls()
        for x in (b, c, b):
            load(x)
            for o in outs:
                o.fill_(5.0)
            graph.replay()
            x.check(outs[0], what=n)
            x.trees, keep = None, x.trees
            x.check(outs[1], 77, 3, what=n)
            x.trees = keep
    assert binding.get_device_errors() == 0


def test_the_same_bits_on_any_pages_and_every_time():
    for n, S in [(1, 3), (6, 2), (40, 3), (64, 1)]:
        a = Batch([500, 300], [n, n], 8, 2, 128, 16, seed=8, kind="mixed")
        want = tree(a, 100, 5, num_splits=S)
        order = torch.randperm(a.pool, device="cuda")
        k, v = torch.empty_like(a.k), torch.empty_like(a.v)
        k[order], v[order] = a.k, a.v
        a.k, a.v = k, v
        a.table = torch.where(a.table >= 0, order[a.table.long().clamp(min=0)].int(), a.table)
        for _ in range(5):
            assert torch.equal(tree(a, 100, 5, num_splits=S), want)


def test_two_streams_at_once():
    a = Batch([900, 700], [40, 40], 8, 2, 128, 16, seed=8, kind="mixed")
    b = Batch([400, 800], [1, 1], 32, 8, 128, 16, seed=9)
    want_a, want_b = tree(a, num_splits=3), window(b, 300, 4, num_splits=4)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    plan_a, plan_b = plan_of(a), plan_of(b)
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        got.append((tree(a, num_splits=3, stream=s, plan=plan_a), window(b, 300, 4, num_splits=4, stream=t, plan=plan_b)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, want_a) and torch.equal(y, want_b)
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("ps", [12, 16])
def test_caches_of_more_than_32_bits(ps):
    """Pages at both ends of a cache of more than 2^32 numbers give the bits of a small one, and its rows move alike."""
    pages = (1 << 32) // (ps * 2 * 128) + 200
    big = [torch.empty((pages, ps, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    for n in (1, 3, 40):
        b = Batch([300, 71], [n, n], 8, 2, 128, ps, seed=n, kind="mixed")
        to = torch.arange(b.pool, device="cuda")
        to[1:] = pages - to[1:]                       # (one page at the cache's beginning)
        for x, y in zip(big, (b.k, b.v)):
            x[to] = y
        table = torch.where(b.table >= 0, to[b.table.long().clamp(min=0)].int(), b.table)
        for S in (1, 3):
            want = [tree(b, num_splits=S), window(b, 100, 5, num_splits=S)]
            small = b.k, b.v, b.table
            b.k, b.v, b.table = *big, table
            assert torch.equal(tree(b, num_splits=S), want[0]) and torch.equal(window(b, 100, 5, num_splits=S), want[1])
            b.k, b.v, b.table = small
        path = torch.arange(n // 2, n, dtype=torch.int32, device="cuda").repeat(2, 1)
        count = torch.full((2,), n - n // 2, dtype=torch.int32, device="cuda")
        base = b.seq_lens - n
        binding.kv_commit_paged(b.k, b.v, b.table, base, path, count)
        binding.kv_commit_paged(*big, table, base, path, count)
        for x, y in zip(big, (b.k, b.v)):
            assert torch.equal(x[to].view(torch.int16), y.view(torch.int16))
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("D,n", [(128, 128), (64, 2)])
def test_partial_sums_of_more_than_32_bits(D, n):
    """512 x 128 or 65536 x 2 new tokens of 32 heads in 16 or more splits: the partial sums pass 2^32 numbers."""
    seqs = 512 if n == 128 else 65536
    b = Batch([1000 if n == 128 else 1023], [n], 32, 4, D, 16, seed=1)
    q = torch.randn((seqs * n, 32, D), device="cuda").to(torch.bfloat16)
    plan = binding.SpanPlan([n] * seqs, 32, 4, D, "cuda")
    S = plan.splits(b.max_len, 1100, 0, num_splits=64)
    assert q.numel() * S > 1 << 32
    out = binding.decode_attn_paged_window(q, b.k, b.v, b.table.expand(seqs, -1).contiguous(), b.seq_lens.expand(seqs).contiguous(),
                                           plan, window=1100, max_kv_len=b.max_len, num_splits=S)
    for at in (0, seqs // 2, seqs - 1):
        b.q = q[at * n:at * n + n]
        b.check(out[at * n:at * n + n], 1100, 0, what=at)
    assert binding.get_device_errors() == 0
