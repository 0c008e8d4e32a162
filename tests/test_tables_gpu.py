"""Page tables resized on the GPU and accepted drafts moved into place, against plain Python on the same integers and rows."""
import random

import pytest
import torch

from paged_kv_cache_298_gb300 import binding
from span_reference import Batch, parents_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    binding.get_device_errors(clear=True)
    yield


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    """Tables, stack and lengths on the GPU, and the same in Python."""

    def __init__(self, lens, ps, max_pages, spare, seed=0):
        r = random.Random(seed)
        need = [-(-n // ps) for n in lens]
        self.ps, self.max_pages, self.lens = ps, max_pages, list(lens)
        self.num_pages = sum(need) + spare
        order = list(range(self.num_pages))
        r.shuffle(order)
        self.table, at = [], 0
        for n in need:
            self.table.append(order[at:at + n] + [-7] * (max_pages - n))
            at += n
        self.free = order[at:] + [-9] * at
        self.count = spare
        self.gpu = (ints(self.table).view(len(lens), max_pages), ints(self.free), ints([self.count]))

    def python(self, new):
        pages = lambda n: -(-n // self.ps)  # noqa: E731
        for row, a, b in zip(self.table, self.lens, new):
            for i in range(pages(b), pages(a)):
                self.free[self.count] = row[i]
                self.count += 1
        taken = sum(max(0, pages(b) - pages(a)) for a, b in zip(self.lens, new))
        assert self.count >= taken
        self.count -= taken
        at, slots, indptr = self.count, [], [0]
        for row, a, b in zip(self.table, self.lens, new):
            for i in range(pages(a), pages(b)):
                row[i] = self.free[at]
                at += 1
            slots += [row[t // self.ps] * self.ps + t % self.ps for t in range(a, b)]
            indptr.append(len(slots))
        self.lens = list(new)
        return indptr, slots

    def same(self):
        table, free, count = self.gpu
        assert count.item() == self.count
        assert table.tolist() == self.table
        assert free.tolist() == self.free

    def resize(self, new, rows, **kw):
        table, free, count = self.gpu
        return binding.kv_resize_paged(kw.pop("old", ints(self.lens)), ints(new), table, free, count, page_size=self.ps,
                                       total_rows=rows, **kw)

    def step(self, new, extra=0, **kw):
        rows = sum(max(0, b - a) for a, b in zip(self.lens, new))
        indptr, slots = self.resize(new, rows + extra, **kw)
        want_indptr, want = self.python(new)
        assert indptr.tolist() == want_indptr
        assert slots.tolist() == want + [-1] * extra
        self.same()


@pytest.mark.parametrize("ps", [1, 5, 16, 64])
@pytest.mark.parametrize("B", [1, 2, 31, 33, 65, 511, 512, 513, 1500])
def test_steps_of_all_kinds(ps, B):
    r = random.Random(B * 100 + ps)
    most = max(3, min(400, 20000 // B))
    p = Pool([r.choice([0, r.randint(0, most)]) for _ in range(B)], ps, -(-most // ps) + 1, B * (-(-most // ps) + 1), seed=B)
    kinds = [lambda n: n, lambda n: 0, lambda n: min(most, n + 1), lambda n: min(most, n + r.randint(0, 20)),
             lambda n: max(0, n - r.randint(0, 20)), lambda n: r.randint(0, most)]
    for kind in kinds[1:] + [None, None, None]:
        new = [(kind or r.choice(kinds))(n) for n in p.lens]
        p.step(new, extra=r.choice([0, 1, 77]), slot_dtype=r.choice([torch.int32, torch.int64]))
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("rows", [2048, 2049, 16384, 16385, 50000])
@pytest.mark.parametrize("wide", [False, True])
def test_long_slot_maps(rows, wide):
    """Either side of the sizes from which a cluster, and then the whole device, works on the rows."""
    r = random.Random(rows)
    cuts = sorted(r.randint(0, rows) for _ in range(36))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
    start = [r.choice([0, 0, r.randint(1, 50)]) for _ in lens]
    new = [a + n for a, n in zip(start, lens)]
    p = Pool(start, 16, max(new) // 16 + 2, rows // 16 + 200, seed=1)
    p.step(new, extra=100, slot_dtype=torch.int64 if wide else torch.int32)
    p.step([0] * len(lens))
    assert binding.get_device_errors() == 0


def test_the_longest_slot_map():
    rows = (1 << 31) - 1                        # (8.6 GB of int32 slots; only the first sequences' rows are there)
    p = Pool([5, 30], 16, 8, 12)
    new = [100, 20]
    out = torch.empty(rows, dtype=torch.int32, device="cuda")
    got, slots = binding.kv_resize_paged(ints(p.lens), ints(new), *p.gpu, page_size=16, total_rows=rows, slots=out)
    indptr, want = p.python(new)
    assert got.tolist() == indptr and slots[:len(want)].tolist() == want
    assert all(bool((x == -1).all()) for x in slots[len(want):].split(1 << 29))
    p.same()


@pytest.mark.parametrize("B", [65, 300, 8192])
def test_many_sequences_of_a_few_rows(B):
    r = random.Random(B)
    p = Pool([r.randint(0, 40) for _ in range(B)], 12, 5, B * 4, B)
    for rows in (0, B * 3, 17000 + B * 3):      # (in one cluster, and on the whole device)
        new = [min(60, max(0, n + r.choice([-13, -1, 0, 1, 3, 3]))) for n in p.lens]
        old = ints(p.lens)
        got, slots = binding.kv_resize_paged(old, ints(new), *p.gpu, page_size=12, total_rows=rows)
        indptr, want = p.python(new)
        assert got.tolist() == indptr and slots.tolist() == (want + [-1] * rows)[:rows]
        p.same()
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("ps", [1, 2, 5, 64])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("off", [0, 1, 2, 3])
def test_a_long_slot_map_that_begins_and_ends_anywhere(ps, dtype, off):
    r = random.Random(ps + off)
    lens = [r.choice([0, 0, 1, 2, 3, r.randint(0, 900)]) for _ in range(70)]
    new = [max(0, n + r.choice([0, 0, -5, 1, 1, 2, 3, 700, 900])) for n in lens]
    wide = max(new) // ps + 2
    p = Pool(lens, ps, wide, 70 * wide, seed=2)
    for extra in (0, 1, 2, 3):
        rows = 17000 + extra
        out = torch.full((rows + off + 1,), 5, dtype=dtype, device="cuda")
        indptr, slots = p.resize(new, rows, slots=out[off:off + rows])
        want_indptr, want = p.python(new)
        assert indptr.tolist() == want_indptr and slots.tolist() == (want + [-1] * rows)[:rows]
        assert out[:off].tolist() == [5] * off and out[-1].item() == 5
        p.same()
        new = [max(0, n + r.choice([0, 0, -300, 1, 1, 2, 3, 300])) for n in p.lens]
        new = [min(n, p.max_pages * ps) for n in new]
        if sum(max(0, n - m) for n, m in zip(new, p.lens)) > sum(m for m in p.lens) // 2:
            new = [n // 2 for n in p.lens]
    binding.get_device_errors(clear=True)             # (a map shorter than the rows is flagged)


def test_backwards_restores_everything():
    r = random.Random(3)
    p = Pool([r.randint(0, 300) for _ in range(100)], 16, 20, 400, seed=3)
    lens, free = list(p.lens), list(p.free)
    for _ in range(3):
        new = [max(0, n + r.randint(-100, 20)) for n in lens]
        p.step(new)
        p.step(lens)
        assert p.count == 400 and p.free[:400] == free[:400]


@pytest.mark.parametrize("B", [3, 200])
def test_a_pool_that_cannot_give_the_pages_changes_nothing(B):
    for spare in (0, 1, B - 1):
        p = Pool([16] * B, 16, 4, spare, seed=2)
        indptr, slots = p.resize([17] * B, B)
        assert binding.get_device_errors() & binding.DEVERR_POOL
        assert indptr.tolist() == [0] * (B + 1) and slots.tolist() == [-1] * B
        p.same()
    p = Pool([16] * B, 16, 4, B, seed=2)   # just enough
    p.step([17] * B)
    p = Pool([16] * B + [48], 16, 4, B - 3, seed=2)   # enough with what the call itself returns
    p.step([17] * B + [0])
    assert binding.get_device_errors() == 0


def test_a_stack_out_of_range_changes_nothing():
    for count in (-1, 10 ** 6, 2 ** 31 - 1):
        p = Pool([40, 40], 16, 4, 5, seed=2)
        p.gpu[2].fill_(count)
        before = [x.clone() for x in p.gpu]
        indptr, slots = p.resize([10, 41], 1)
        assert binding.get_device_errors() & binding.DEVERR_POOL
        assert indptr.tolist() == [0, 0, 0] and slots.tolist() == [-1]
        assert all(torch.equal(a, b) for a, b in zip(before, p.gpu))
    p = Pool([40, 40], 16, 4, 5, seed=2)
    p.gpu[2].fill_(p.num_pages)            # more would come back than the pool has
    p.resize([10, 40], 0)
    assert binding.get_device_errors() & binding.DEVERR_POOL and p.gpu[2].item() == p.num_pages


def test_lengths_out_of_range_leave_their_sequence():
    for bad_old, bad_new in [(-1, 5), (5, -1), (65, 5), (5, 65), (2 ** 31 - 1, 0), (0, 2 ** 31 - 1), (-2 ** 31, 3)]:
        p = Pool([5, 20, 30], 16, 4, 6, seed=2)
        indptr, slots = p.resize([9, bad_new, 40], 14, old=ints([5, bad_old, 30]))
        assert binding.get_device_errors() & binding.DEVERR_SEQLEN
        want_indptr, want = p.python([9, 20, 40])
        assert indptr.tolist() == want_indptr and slots.tolist() == want
        p.same()


def test_more_rows_than_the_slot_map_holds():
    for rows, B in [(3, 2), (9000, 70)]:
        each = rows // B + 50
        p = Pool([0] * B, 16, each // 16 + 1, B * (each // 16 + 1), seed=2)
        indptr, slots = p.resize([each] * B, rows)
        assert binding.get_device_errors() & binding.DEVERR_SLOT
        want_indptr, want = p.python([each] * B)
        assert indptr.tolist() == want_indptr and slots.tolist() == want[:rows]
        p.same()


@pytest.mark.parametrize("B", [3, 200])
def test_a_call_that_wants_no_slot_map(B):
    p = Pool([5] * B, 16, 8, 7 * B, seed=2)
    indptr, slots = p.resize([100] * B, 0)
    want_indptr, _ = p.python([100] * B)
    assert indptr.tolist() == want_indptr and slots.numel() == 0
    p.same()
    assert binding.get_device_errors() == 0


def test_pages_outside_the_pool_have_no_slot():
    for rows in (30, 9000):
        p = Pool([0, 10], 16, rows // 16 + 2, rows // 16 + 3, seed=2)
        p.gpu[1][p.count - 1] = p.num_pages + 4   # the top of the stack is taken
        _, slots = p.resize([rows, 10], rows)
        assert binding.get_device_errors() & binding.DEVERR_PAGE
        _, want = p.python([rows, 10])
        got = slots.tolist()
        at = [i for i, (a, b) in enumerate(zip(got, want)) if a != b]
        assert len(at) == (rows - 1) % 16 + 1 and all(got[i] == -1 for i in at)   # the last page's rows


def test_given_outputs_an_empty_batch_and_other_streams():
    p = Pool([5, 16], 16, 4, 6, seed=2)
    indptr, slots = torch.full((4,), 9, dtype=torch.int32, device="cuda"), torch.full((6,), 9, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = p.resize([7, 18], 4, indptr=indptr[:3], slots=slots[:4], stream=s)
    torch.cuda.synchronize()
    assert out[0].data_ptr() == indptr.data_ptr() and out[1].data_ptr() == slots.data_ptr()
    want_indptr, want = p.python([7, 18])
    assert indptr.tolist() == want_indptr + [9] and slots.tolist() == want + [9, 9]
    p.same()
    none = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    free, count = ints([1, 2, 3]), ints([2])
    indptr, slots = binding.kv_resize_paged(ints([]), ints([]), none, free, count, page_size=16, total_rows=3)
    assert indptr.tolist() == [0] and slots.tolist() == [-1] * 3 and count.item() == 2 and free.tolist() == [1, 2, 3]
    assert binding.get_device_errors() == 0


def test_captured_steps():
    p = Pool([30, 0, 47], 16, 8, 12, seed=4)
    old, new = ints([30, 0, 47]), ints([31, 17, 40])
    table, free, count = p.gpu
    indptr, slots = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(40, dtype=torch.int64, device="cuda")

    def call():
        binding.kv_resize_paged(old, new, table, free, count, page_size=16, total_rows=40, indptr=indptr, slots=slots)
        old.copy_(new)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        call()
    torch.cuda.synchronize()
    p.python([31, 17, 40])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([32, 0, 48], [0, 33, 49], [40, 33, 0]):
        new.copy_(ints(lens))
        g.replay()
        want_indptr, want = p.python(lens)
        assert indptr.tolist() == want_indptr and slots.tolist() == want + [-1] * (40 - len(want))
        p.same()
    assert binding.get_device_errors() == 0


# ---- accepted drafts -----------------------------------------------------------------------------

def committed(k, rows, ps, base, path):
    out = k.clone()
    for j, n in enumerate(path):
        s, d = base + n, base + j
        out[rows[d // ps], d % ps] = k[rows[s // ps], s % ps]
    return out


@pytest.mark.parametrize("ps", [1, 5, 16, 64])
@pytest.mark.parametrize("Hkv,D", [(1, 8), (2, 32), (3, 64), (8, 128), (4, 256), (5, 72)])
def test_commit(ps, Hkv, D):
    r = random.Random(ps + Hkv)
    nodes = [0, 1, 5, 40, 100, 256]
    base = [r.randint(0, 100) for _ in nodes]
    paths = [sorted(r.sample(range(n), r.randint(0, n))) for n in nodes]
    paths[4] = list(range(100))          # everything accepted: nothing moves
    paths[5] = list(range(1, 256))       # every row moves by one
    need = [-(-(b + n) // ps) for b, n in zip(base, nodes)]
    order = list(range(sum(need) + 2))
    r.shuffle(order)
    rows, at = [], 0
    for n in need:
        rows.append(order[at:at + n])
        at += n
    width = max(need) + 1
    table = ints([x + [-1] * (width - len(x)) for x in rows])
    k, v = (torch.randn((len(order), ps, Hkv, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    k.view(torch.int16)[order[-1]] = 0x7FC0 - 1   # (bits move, whatever they mean)
    wk, wv = k, v
    for b, path in enumerate(paths):
        wk, wv = committed(wk, rows[b], ps, base[b], path), committed(wv, rows[b], ps, base[b], path)
    wide = max(1, max(map(len, paths)))
    path = ints([x + [3] * (wide - len(x)) for x in paths])
    out = binding.kv_commit_paged(k, v, table, ints(base), path, ints([len(x) for x in paths]))
    assert out[0].data_ptr() == k.data_ptr()
    assert torch.equal(k.view(torch.int16), wk.view(torch.int16)) and torch.equal(v.view(torch.int16), wv.view(torch.int16))
    assert binding.get_device_errors() == 0


def test_commit_refuses_on_the_device_what_is_no_path():
    def run(path, n, base=20, entry=None, flag=0):
        b = Batch([20, 30], [40, 40], 2, 2, 64, 16, seed=1)
        if entry is not None:
            b.table[0, entry] = b.pool
        k, v = b.k.clone(), b.v.clone()
        path = (path + [39] * 35)[:35]
        binding.kv_commit_paged(b.k, b.v, b.table, ints([base, 30]), ints([path, list(range(1, 36))]), ints([n, 3]))
        assert binding.get_device_errors() == flag
        other = committed(k, b.rows[1], 16, 30, [1, 2, 3])
        return b, k, other
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    for path, n, base, flag in [([3, 3], 2, 20, binding.DEVERR_QMAP), ([5, 4], 2, 20, binding.DEVERR_QMAP),
                                ([-1, 4], 2, 20, binding.DEVERR_QMAP), ([0], -1, 20, binding.DEVERR_QMAP),
                                ([0], 36, 20, binding.DEVERR_QMAP), (list(range(1, 33)) + [5], 33, 20, binding.DEVERR_QMAP),
                                ([1], 1, -5, binding.DEVERR_SEQLEN), ([1, 2 ** 31 - 1], 2, 20, binding.DEVERR_SEQLEN),
                                ([2], 1, 2 ** 31 - 2, binding.DEVERR_SEQLEN)]:
        b, k, other = run(path, n, base=base, flag=flag)
        assert same(b.k, other), (path, n, base)
    # a page outside the pool: its rows stay, the others move
    b, k, other = run([1, 20, 30], 3, entry=3, flag=binding.DEVERR_PAGE)   # place 50 is in entry 3
    want = committed(other, b.rows[0], 16, 20, [1, 20])
    assert same(b.k, want)
    b, k, other = run([5], 0)
    assert same(b.k, other)


# ---- a whole step ---------------------------------------------------------------------------------

@pytest.mark.parametrize("w,sinks", [(0, 0), (40, 4)])
@pytest.mark.parametrize("D,ps,n", [(128, 16, 12), (64, 12, 40), (256, 64, 5)])
def test_steps_of_speculative_decoding(w, sinks, D, ps, n):
    """Lengths grow by the drafts, the drafts' rows are written through the slot map, the trees are attended, the accepted
    paths are moved into place and the lengths shrink to them: three steps in a row give what plain attention over the
    accepted tokens gives."""
    r = random.Random(n)
    Hq, Hkv = 8, 2
    lens = [37, 0, 150]
    p = Pool(lens, ps, 40, 60, seed=5)
    table, free, count = p.gpu
    k, v = (torch.full((p.num_pages, ps, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lines = [[torch.randn((m, Hkv, D), device="cuda").to(torch.bfloat16) for _ in range(2)] for m in lens]
    for b, m in enumerate(lens):
        for t in range(m):
            k[p.table[b][t // ps], t % ps], v[p.table[b][t // ps], t % ps] = lines[b][0][t], lines[b][1][t]
    plan = binding.SpanPlan([n] * 3, Hq, Hkv, D, "cuda")
    for step in range(3):
        trees = [parents_of(n, "mixed", r) for _ in lens]
        rows = [torch.randn((3 * n, Hkv, D), device="cuda").to(torch.bfloat16) for _ in range(2)]
        q = torch.randn((3 * n, Hq, D), device="cuda").to(torch.bfloat16)
        drafted = [m + n for m in lens]
        _, slots = binding.kv_resize_paged(ints(lens), ints(drafted), table, free, count, page_size=ps, total_rows=3 * n,
                                           slot_dtype=torch.int32)
        # the slot map is a block table of one-slot pages
        one = (p.num_pages * ps, 1, Hkv, D)
        binding.kv_append_paged(rows[0], rows[1], k.view(one), v.view(one), slots.view(-1, 1), torch.zeros_like(slots))
        out = binding.decode_attn_paged_tree(q, k, v, table, ints(drafted), ints([x for t in trees for x in t]), plan,
                                             max_kv_len=max(drafted), window=w, sinks=sinks)
        paths = []
        for b, t in enumerate(trees):
            node = r.randrange(n)
            path = []
            while node >= 0:
                path.append(node)
                node = t[node]
            paths.append(path[::-1])
            new = [torch.cat([lines[b][x], rows[x][b * n:(b + 1) * n][paths[b]]]) for x in range(2)]
            # the last node of the path sees its line, and nothing else
            c = Batch([0], [1], Hq, Hkv, D, 16)
            m = len(new[0])
            c.ctx, c.counts, c.lens, c.rows, c.ps, c.total = [m - 1], [1], [m], [[0]], m, 1
            c.k, c.v, c.q = new[0][None], new[1][None], q[b * n + paths[b][-1]][None]
            c.check(out[b * n + paths[b][-1]][None], w, sinks, what=(step, b))
            lines[b] = new
        wide = max(map(len, paths))
        binding.kv_commit_paged(k, v, table, ints(lens), ints([x + [0] * (wide - len(x)) for x in paths]),
                                ints([len(x) for x in paths]))
        kept = [m + len(x) for m, x in zip(lens, paths)]
        binding.kv_resize_paged(ints(drafted), ints(kept), table, free, count, page_size=ps)
        lens = kept
        held = table.tolist()
        for b, m in enumerate(lens):
            at = torch.arange(m)
            page = torch.tensor(held[b])[at // ps].cuda()
            assert torch.equal(k[page, (at % ps).cuda()], lines[b][0]) and torch.equal(v[page, (at % ps).cuda()], lines[b][1])
    assert count.item() == p.num_pages - sum(-(-m // ps) for m in lens)
    assert binding.get_device_errors() == 0
