"""Windowed and tree attention, resizes and commits as programs make them: from two threads on one plan, captured on streams of
their own and replayed with other contents, with views of larger tensors in the shapes for large batches."""
import random
import threading

import pytest
import torch

from paged_kv_cache_298_gb300 import binding
from span_reference import Batch, parents_of
from test_span_shapes_gpu import call, plan_of
from test_tables_gpu import Pool, committed, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    binding.get_device_errors(clear=True)
    yield


def test_two_threads_on_one_plan():
    """Each thread with a stream of its own, calls of several shapes with bounds that differ from call to call."""
    b = [Batch([500, 300], [40, 40], 8, 2, 128, 16, seed=i, kind="mixed") for i in (1, 2)]
    plan, wide = binding.SpanPlan([40, 40], 8, 2, 128, "cuda"), plan_of(b[0], 256)
    forms = [(p, w, s, S) for p in (plan, wide) for w, s in ((0, 0), (100, 4), (31, 0)) for S in (0, 1, 3)]
    want = [[call(x, p, w, s, num_splits=S) for p, w, s, S in forms] for x in b]
    pools = [Pool([0] * 70, 16, 40, 70 * 40, seed=i) for i in (1, 2)]
    torch.cuda.synchronize()
    failed = []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                r = random.Random(i)
                for _ in range(20):
                    got = [call(b[i], p, w, s, num_splits=S) for p, w, s, S in forms]
                    pools[i].step([r.randint(0, 600) for _ in range(70)], extra=r.choice([0, 20000]))
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(x, y) for x, y in zip(got, want[i])):
                        failed.append(i)
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("ps", [5, 16])
def test_commits_replayed_on_a_stream(ps):
    r = random.Random(ps)
    B, nodes, Hkv, D = 12, 70, 2, 64
    pages = -(-(100 + nodes) // ps)
    table = torch.randperm(B * pages).int().view(B, pages)
    k, v = (torch.randn((B * pages, ps, Hkv, D), device="cuda").to(torch.bfloat16) for _ in "kv")
    base, path, count = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B,), (B, 40), (B,)))
    gt, st = table.cuda(), torch.cuda.Stream()
    torch.cuda.synchronize()
    binding.kv_commit_paged(k, v, gt, base, path, count, stream=st)     # (no path: nothing moves)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        binding.kv_commit_paged(k, v, gt, base, path, count)
        binding.kv_commit_paged(k, v, gt, base, path, count)            # (the second reads what the first has written)
    for _ in range(4):
        paths = [sorted(r.sample(range(nodes), r.randint(0, 40))) for _ in range(B)]
        at = [r.randint(0, 100) for _ in range(B)]
        base.copy_(ints(at))
        path.copy_(ints([x + [0] * (40 - len(x)) for x in paths]))
        count.copy_(ints([len(x) for x in paths]))
        want = [k.clone(), v.clone()]
        for _ in range(2):
            for i, x in enumerate(want):
                for b in range(B):
                    x = committed(x, table[b].tolist(), ps, at[b], paths[b])
                want[i] = x
        graph.replay()
        assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("D,cols", [(64, 256), (128, 256), (64, 128), (128, 128), (256, 128), (128, 16)])
def test_views_of_larger_tensors(D, cols):
    """q inside a fused projection, or heads first; outputs with room between rows, which stays as it is."""
    Hkv, G, B = 8, 4, 24
    n = [1 + (5 * i) % (cols // G) for i in range(B)]
    b = Batch([(53 * i) % 300 for i in range(B)], n, G * Hkv, Hkv, D, 16, seed=cols, kind="mixed")
    plan, q = plan_of(b, cols), b.q
    for S in (1, 2):
        want = call(b, plan, 100, 4, num_splits=S)
        b.check(want, 100, 4)
        fused = torch.full((b.total, (G + 2) * Hkv * D), float("nan"), dtype=torch.bfloat16, device="cuda")
        views = [fused[:, :G * Hkv * D].view(b.total, G * Hkv, D), torch.empty((G * Hkv, b.total, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1)]
        for view in views:
            view.copy_(q)
            b.q = view
            out = torch.full((b.total + 2, G * Hkv + 3, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
            inner = out[1:-1, 2:-1, :D]
            call(b, plan, 100, 4, num_splits=S, out=inner)
            assert torch.equal(inner, want)
            inner.fill_(7.0)
            assert bool((out == 7.0).all())
            b.q = q
    assert binding.get_device_errors() == 0


def test_one_workspace_for_two_graphs():
    """Graphs that share a workspace and are replayed in turn."""
    a, c = Batch([500, 90], [64, 33], 8, 2, 128, 16, seed=1, kind="mixed"), Batch([300] * 3, [1, 2, 3], 16, 2, 64, 12, seed=2)
    plans = plan_of(a, 256), binding.SpanPlan(c.counts, 16, 2, 64, "cuda")
    size = max(binding.workspace_bytes_span(p, max_kv_len=x.max_len, window=200, sinks=3, tree=t, num_splits=4)
               for p, x, t in zip(plans, (a, c), (True, False)))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty_like(x.q) for x in (a, c)], []
    for x, p, o in zip((a, c), plans, outs):
        call(x, p, 200, 3, num_splits=4, workspace=ws, out=o)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(x, p, 200, 3, num_splits=4, workspace=ws, out=o)
        graphs.append(g)
    for o in outs:
        o.fill_(float("nan"))
    for _ in range(20):
        for g in graphs:
            g.replay()
    a.check(outs[0], 200, 3)
    c.check(outs[1], 200, 3)
    assert binding.get_device_errors() == 0


def test_parents_that_change_behind_a_plan():
    """One plan, trees of every kind in turn, and a batch whose trees hold fewer nodes than their places (the rest hang from the
    context)."""
    n = [30, 64, 7]
    b = Batch([100, 411, 0], n, 8, 2, 128, 16, seed=3, kind="mixed")
    plan, r = plan_of(b, 256), random.Random(1)
    for kind in ("chain", "star", "roots", "mixed", "chain"):
        b.trees = [parents_of(m, kind, r) for m in n]
        b.parents.copy_(ints([p for t in b.trees for p in t]))
        for w, s in ((0, 0), (20, 3)):
            b.check(call(b, plan, w, s), w, s, what=(kind, w))
    assert binding.get_device_errors() == 0
