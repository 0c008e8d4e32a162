"""Shared-prefix decode on the GPU against plain attention in 64 bits, sequence by sequence.

Tolerance (with A = sum_t w_t |v_t|, the weights' sum of absolute values): the weights are rounded to bf16
for the product with V (at most 2^-8 of each: 2^-8 A), the suffix's normaliser sums the rounded weights
(2^-8 |out| <= 2^-8 A), and the output is rounded to bf16 (2^-8 |out|).  Scores are binary32 sums of D
products (relative error of a weight at most D 2^-24 sum |q k| scale, below 2^-12 at these sizes), the
exponential and the merges are within 2^-20.  Rows that nothing may read (unused pages, positions past a
sequence's end) hold NaN, so reading one shows."""
import math

import pytest
import torch

from paged_kv_cache_298_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    binding.get_device_errors(clear=True)
    yield


class Case:
    """Groups of sequences over one pool; whole pages of a prefix are shared, the page that it ends in is each sequence's
    own (only the first sequence's copy of the prefix's rows in it is valid: the others hold NaN there)."""

    def __init__(self, sizes, prefixes, suffix, Hq, Hkv, D, ps, seed=0, qmag=1.0):
        g = torch.Generator().manual_seed(1000 + seed)
        B = sum(sizes)
        group = [i for i, n in enumerate(sizes) for _ in range(n)]
        lens = [0 if s < 0 else prefixes[i] + s for i, s in zip(group, suffix)]
        whole = [p // ps for p in prefixes]
        own = [max(-(-max(n, prefixes[i]) // ps) - whole[i], 0) for n, i in zip(lens, group)]
        pool = sum(whole) + sum(own) + 2
        order = torch.randperm(pool, generator=g).tolist()
        width = max([1] + [whole[i] + n for i, n in zip(group, own)])
        table = torch.full((B, width), -1, dtype=torch.int32)
        at, shared = 0, []
        for w in whole:
            shared.append(order[at:at + w])
            at += w
        k = torch.full((pool, ps, Hkv, D), float("nan"))
        v = torch.full((pool, ps, Hkv, D), float("nan"))
        b = 0
        for i, n in enumerate(sizes):
            for page in shared[i]:
                k[page], v[page] = torch.randn((ps, Hkv, D), generator=g), torch.randn((ps, Hkv, D), generator=g)
            for j in range(n):
                mine = shared[i] + order[at:at + own[b]]
                at += own[b]
                table[b, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
                first = whole[i] * ps if j == 0 else prefixes[i]
                for t in range(first, max(lens[b], prefixes[i] if j == 0 else 0)):
                    k[mine[t // ps], t % ps] = torch.randn((Hkv, D), generator=g)
                    v[mine[t // ps], t % ps] = torch.randn((Hkv, D), generator=g)
                b += 1
        self.sizes, self.group, self.Hq, self.Hkv, self.D, self.ps, self.B = sizes, group, Hq, Hkv, D, ps, B
        self.q = (torch.randn((B, Hq, D), generator=g) * qmag).to(torch.bfloat16).cuda()
        self.k, self.v = k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda()
        self.table = table.cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.prefix = torch.tensor(prefixes, dtype=torch.int32, device="cuda")
        self.max_prefix, self.max_suffix = max(prefixes), max(0, max(suffix, default=0))
        self.plan = binding.SharedPlan(sizes, Hq, Hkv, D, "cuda")
        self.scale = 1.0 / math.sqrt(D)

    def run(self, **kw):
        a = dict(max_prefix_len=self.max_prefix, max_suffix_len=self.max_suffix, scale=self.scale)
        a.update(kw)
        return binding.decode_attn_paged_shared(self.q, self.k, self.v, self.table, self.lens, self.prefix, self.plan, **a)

    def plain(self):
        """(out, A) in 64 bits."""
        out = torch.zeros((self.B, self.Hq, self.D), dtype=torch.float64, device="cuda")
        A = torch.zeros_like(out)
        starts = [sum(self.sizes[:i]) for i in range(len(self.sizes))]
        for b, n in enumerate(self.lens.tolist()):
            P = int(self.prefix[self.group[b]])
            if n == 0 or n < P:
                continue
            t = torch.arange(n, device="cuda")
            row = torch.where(t < P, starts[self.group[b]], b)
            page = self.table[row, t // self.ps].long()
            G = self.Hq // self.Hkv
            k, v = (x[page, t % self.ps].double().repeat_interleave(G, dim=1) for x in (self.k, self.v))
            w = torch.softmax(torch.einsum("hd,thd->ht", self.q[b].double(), k) * self.scale, dim=1)
            out[b] = torch.einsum("ht,thd->hd", w, v)
            A[b] = torch.einsum("ht,thd->hd", w, v.abs())
        return out, A

    def check(self, out, ref, what="", rows=slice(None)):
        want, A = (r[rows] for r in ref)
        got = out.double()[rows]
        assert bool(torch.isfinite(got).all()), f"{what}: not finite"
        excess = (got - want).abs() - (2.0 ** -8 * (2 * A + want.abs()) + 2.0 ** -12 * A)
        assert float(excess.max()) <= 0, f"{what}: off by {float(excess.max()):.3g} more than the bound at {int(excess.argmax())}"


CASES = [
    # sizes, prefixes, lengths behind the prefix (-1: empty row), Hq, Hkv, D, page size
    ([1], [1], [1], 1, 1, 64, 16),
    ([2], [64], [5, 70], 8, 2, 64, 16),
    ([2], [128], [0, 0], 8, 2, 128, 16),                       # nothing behind the prefix
    ([3], [0], [1, 64, 130], 8, 8, 128, 16),                   # no prefix
    ([3], [65], [1, -1, 63], 16, 2, 128, 16),                  # prefix ends inside a page and a tile; an empty row
    ([4], [200], [-1, -1, -1, -1], 8, 2, 64, 8),               # only empty rows
    ([16], [777], [3 * i for i in range(16)], 32, 8, 128, 16),
    ([33], [300], [i % 5 for i in range(33)], 4, 1, 128, 64),  # 132 rows: both streams, the second with 4 rows
    ([70], [513], [7] * 70, 8, 2, 128, 32),                    # 280 rows: two tiles
    ([40], [1000], [11] * 40, 8, 1, 64, 128),                  # G = 8, 320 rows
    ([66], [333], [3] * 66, 8, 2, 128, 8),                     # 264 rows: the second tile of the pair has 8
    ([200], [450], [2] * 200, 8, 2, 128, 64),                  # 800 rows: four tiles
    ([130, 70, 3], [450, 100, 64], [2] * 203, 16, 4, 128, 16), # tiles 3 + 2 + 1: pairs across groups stay apart
    ([90, 64], [129, 200], [1] * 154, 4, 1, 256, 32),          # D = 256: three tiles and two
    ([130], [190], [2] * 130, 1, 1, 64, 16),                   # G = 1
    ([20], [640], [i for i in range(20)], 16, 2, 256, 16),     # D = 256: 160 rows, two tiles of 128
    ([5], [129], [31, 0, 1, 64, 100], 4, 2, 256, 32),
    ([2, 1, 0, 40], [100, 37, 50, 321], [4] * 43, 16, 4, 128, 16),   # groups, one of one sequence, an empty one
    ([3, 4], [0, 90], [50, 1, 2, 3, 4, 5, 200], 8, 4, 64, 8),        # a group without a prefix beside one with
    ([6], [100], [1, 2, 3, 40, 50, 60], 8, 2, 128, 12),        # row gather
    ([6], [77], [0, 1, 2, 90, 5, 6], 8, 2, 64, 5),
    ([5], [130], [9, 10, 70, 0, 33], 8, 1, 256, 12),
    ([3], [50], [3, 4, 5], 6, 3, 128, 1),
    ([4], [250], [3, 64, 65, 129], 12, 3, 128, 100),
    ([9], [2000], [1] * 9, 64, 8, 128, 64),
    ([3], [192], [64, 128, 63], 4, 4, 128, 24),
]


@pytest.mark.parametrize("sizes,prefixes,suffix,Hq,Hkv,D,ps", CASES,
                         ids=[f"g{'_'.join(map(str, c[0]))}_P{c[1][0]}_G{c[3] // c[4]}_D{c[5]}_ps{c[6]}" for c in CASES])
def test_against_plain_attention(sizes, prefixes, suffix, Hq, Hkv, D, ps):
    c = Case(sizes, prefixes, suffix, Hq, Hkv, D, ps)
    ref = c.plain()
    for pre, suf in ((0, 0), (1, 1), (3, 2), (1000, 1000)):
        c.check(c.run(prefix_splits=pre, suffix_splits=suf), ref, f"splits {pre}, {suf}")
        assert binding.get_device_errors() == 0
    c.check(c.run(max_prefix_len=min(c.table.shape[1] * ps, c.max_prefix + 500),
                  max_suffix_len=min(c.table.shape[1] * ps, c.max_suffix + 300), total_suffix=sum(max(s, 0) for s in suffix)),
            ref, "loose bounds")
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_merging_of_many_partials(G, D):
    """One suffix split, which may merge its rows itself, and any number of prefix partials: none, fewer than the warps, one
    trip and two of them, more than a CTA takes itself."""
    c = Case([5], [64 * 50 - 7], [0, -1, 1, 40, 90], 2 * G, 2, D, 16, seed=40 + G)
    ref = c.plain()
    for n in (1, 2, 3, 4, 7, 12, 13, 24, 25, 48, 50):
        c.check(c.run(prefix_splits=n, suffix_splits=1), ref, f"{n} prefix partials")
    c.prefix.zero_()
    c.max_prefix = 0
    c.lens = torch.tensor([0, 1, 64, 65, 90], dtype=torch.int32, device="cuda")
    c.table[:] = c.table[0]
    c.max_suffix = 90
    c.check(c.run(suffix_splits=1), c.plain(), "no prefix")
    assert binding.get_device_errors() == 0


def test_equals_ordinary_decode():
    """The same batch through decode_attn_paged (page-aligned prefix: the block tables are complete)."""
    c = Case([24], [512], [i * 9 for i in range(24)], 32, 8, 128, 16)
    n = int(c.lens.max())
    a = c.run()
    b = binding.decode_attn_paged(c.q, c.k, c.v, c.table.clamp(min=0), c.lens, max_kv_len=n, scale=c.scale)
    ref = c.plain()
    c.check(a, ref)
    c.check(b, ref)


@pytest.mark.parametrize("ps", [16, 12])
def test_any_placement_of_the_pages_gives_the_same_bits(ps):
    c = Case([20, 3], [330, 100], [i * 7 for i in range(23)], 8, 2, 128, ps)
    a = c.run(prefix_splits=3, suffix_splits=2)
    perm = torch.randperm(c.k.shape[0], generator=torch.Generator().manual_seed(5)).cuda()
    inv = torch.argsort(perm).to(torch.int32)
    c.k, c.v = c.k[perm].contiguous(), c.v[perm].contiguous()
    c.table = torch.where(c.table >= 0, inv[c.table.clamp(min=0).long()], c.table)
    assert torch.equal(a, c.run(prefix_splits=3, suffix_splits=2))
    assert torch.equal(a, c.run(prefix_splits=3, suffix_splits=2))


def test_strided_q_and_out():
    c = Case([10], [150], [i for i in range(10)], 8, 2, 128, 16)
    want = c.run()
    big = torch.full((10, 12, 160), 3.0, dtype=torch.bfloat16, device="cuda")
    big[:, 2:10, 16:144] = c.q
    c.q = big[:, 2:10, 16:144]
    out = torch.full((10, 3, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = c.run(out=out[:, 1])
    assert got.data_ptr() == out[:, 1].data_ptr()
    assert torch.equal(out[:, 1], want) and bool((out[:, 0] == 7).all()) and bool((out[:, 2] == 7).all())


@pytest.mark.parametrize("qmag", [1e3, 1e18])
def test_large_scores(qmag):
    """Scores so large that one key takes all the weight: that key's row of V comes out, whatever the order of the tiles
    (the running maximum moves by more than 2^8 many times)."""
    c = Case([40], [700], [30] * 40, 8, 2, 128, 16, qmag=qmag)
    ref = c.plain()
    top = ref[1].abs().double()
    out = c.run().double()
    assert bool(torch.isfinite(out).all())
    # a score is off by D 2^-24 sum |q k| scale: at qmag 1e3 that is 0.1 to 1, so rows with a close second are left out
    w_top = (ref[0].abs() - top).abs().max(-1).values < 1e-9
    assert int(w_top.sum()) > 100
    err = (out - ref[0]).abs() - 2.0 ** -8 * ref[0].abs()
    assert float(err[w_top].max()) <= 2.0 ** -8 * float(ref[1].max())


def test_negative_and_zero_scale():
    c = Case([9], [200], [i * 3 for i in range(9)], 8, 2, 64, 16)
    for scale in (-0.2, 0.0):
        c.scale = scale
        c.check(c.run(), c.plain(), f"scale {scale}")


def test_infinite_values_stay_in_their_row():
    """An infinite V of one sequence's suffix, and a NaN q of one sequence, reach that sequence's rows only."""
    c = Case([12], [300], [20] * 12, 8, 2, 128, 16)
    ref = c.run()
    t = int(c.lens[3]) - 1
    c.v[int(c.table[3, t // 16]), t % 16, 0, 5] = float("inf")
    c.q[7, 2] = float("nan")
    out = c.run()
    keep = torch.ones((12, 8, 128), dtype=torch.bool)
    keep[3, 0:4, 5] = False
    keep[7, 2] = False
    assert torch.equal(out[keep.cuda()], ref[keep.cuda()])
    assert bool(out[3, 0:4, 5].isinf().all())


def test_bad_lengths_groups_and_pages_are_flagged():
    c = Case([8, 4], [200, 100], [30] * 12, 8, 2, 128, 16)
    ref = c.plain()
    good = c.lens.clone()
    # a length inside the prefix gives a zero row; one past the bound is lowered to it; a negative one is empty
    c.lens[1], c.lens[2], c.lens[3] = 150, 300, -5
    out = c.run()
    assert binding.get_device_errors() & binding.DEVERR_SEQLEN
    assert bool((out[1] == 0).all()) and bool((out[3] == 0).all())
    c.check(out, ref, rows=[0, 2, 4, 5, 6, 7, 8, 9, 10, 11])
    c.lens = good.clone()
    # a prefix past its bound is lowered: every row of that group changes, none of the other
    c.prefix[0] = 201
    out = c.run()
    assert binding.get_device_errors() & binding.DEVERR_SEQLEN
    c.check(out, ref, rows=[8, 9, 10, 11])
    c.prefix[0] = 200
    # groups out of range
    sg = c.plan.seq_group.clone()
    c.plan.seq_group[4], c.plan.seq_group[5] = 2, -1
    out = c.run()
    assert binding.get_device_errors() & binding.DEVERR_QMAP
    assert bool((out[4:6] == 0).all())
    c.check(out, ref, rows=[0, 1, 2, 3, 6, 7, 8, 9, 10, 11])
    c.plan.seq_group.copy_(sg)
    tiles = c.plan.tiles.clone()
    for at, bad in (((1, 0), 5), ((1, 0), -1), ((1, 1), 12), ((0, 2), -1), ((1, 2), 11), ((0, 3), 65), ((0, 3), 0)):
        c.plan.tiles[at] = bad
        c.run()
        assert binding.get_device_errors() & binding.DEVERR_QMAP, (at, bad)
        c.plan.tiles.copy_(tiles)
    c.check(c.run(), ref)
    assert binding.get_device_errors() == 0
    # pages outside the pool: read as page 0, and flagged; the other sequences keep their results
    c.table[6, 13] = c.k.shape[0]
    c.k[0], c.v[0] = torch.nan_to_num(c.k[0]), torch.nan_to_num(c.v[0])
    out = c.run()
    assert binding.get_device_errors() & binding.DEVERR_PAGE
    c.check(out, ref, rows=[8, 9])
    c.table[0, 2] = -3
    c.run()
    assert binding.get_device_errors() & binding.DEVERR_PAGE


def test_offsets_past_32_bits():
    """Prefix and suffix pages beyond 2^31 elements of the pool."""
    Hkv, D, ps, pool = 8, 256, 64, 17000
    k = torch.empty((pool, ps, Hkv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = Case([5], [128], [10, 20, 64, 0, 1], 16, 8, D, ps)
    n = c.k.shape[0]
    k[-n:], v[-n:] = c.k, c.v
    ref = c.plain()
    c.k, c.v = k, v
    c.table = torch.where(c.table >= 0, c.table + (pool - n), c.table)
    c.check(c.run(), ref)
    k12, v12 = k.view(-1)[:(k.numel() // (12 * Hkv * D)) * 12 * Hkv * D].view(-1, 12, Hkv, D), v.view(-1)
    v12 = v12[:k12.numel()].view(k12.shape)
    c2 = Case([5], [130], [10, 20, 64, 0, 1], 16, 8, D, 12)
    n = c2.k.shape[0]
    k12[-n:], v12[-n:] = c2.k, c2.v
    ref = c2.plain()
    c2.k, c2.v = k12, v12
    c2.table = torch.where(c2.table >= 0, c2.table + (k12.shape[0] - n), c2.table)
    c2.check(c2.run(), ref)


def test_calls_in_a_row_share_a_workspace():
    """Calls queued without waiting, on one workspace: each gives what it gives alone."""
    cs = [Case([20], [300 + 64 * i], [5 * i + j for j in range(20)], 8, 2, 128, 16, seed=i) for i in range(3)]
    alone = [c.run() for c in cs]
    torch.cuda.synchronize()
    n = max(binding.workspace_bytes_shared(c.plan, max_prefix_len=c.max_prefix, max_suffix_len=c.max_suffix) for c in cs)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs = [cs[i % 3].run(workspace=ws) for i in range(60)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, alone[i % 3])


def test_append_then_decode_without_waiting():
    """Each step appends a token to every sequence and decodes at once: the decode sees it."""
    c = Case([16], [256], [0] * 16, 8, 2, 128, 16)
    steps = 40
    pages = torch.arange(16 * 3, dtype=torch.int32, device="cuda").view(16, 3) + c.k.shape[0]
    c.k = torch.cat([c.k, torch.full((48, 16, 2, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    c.v = torch.cat([c.v, torch.full((48, 16, 2, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    c.table = torch.cat([c.table[:, :16], pages], dim=1).contiguous()
    new = torch.randn((steps, 2, 16, 2, 128), device="cuda").to(torch.bfloat16)
    lens = [torch.full((16,), 256 + i, dtype=torch.int32, device="cuda") for i in range(steps + 1)]
    c.max_suffix = steps
    outs = []
    for i in range(steps):
        binding.kv_append_paged(new[i, 0], new[i, 1], c.k, c.v, c.table, lens[i])
        c.lens = lens[i + 1]
        outs.append(c.run())
    torch.cuda.synchronize()
    for i in (0, 1, 7, 15, 16, 31, steps - 1):
        c.lens = lens[i + 1]
        c.check(outs[i], c.plain(), f"step {i}")
    assert binding.get_device_errors() == 0


def test_lengths_that_grow_in_place():
    """One tensor of lengths, advanced on the device between calls that are queued without waiting: every kernel of a call
    sees the lengths of its step."""
    c = Case([16], [128], [90] * 16, 8, 2, 128, 16)
    full = c.lens.clone()
    c.lens.fill_(128)
    outs = []
    for _ in range(90):
        c.lens += 1
        outs.append(c.run(max_suffix_len=90))
    torch.cuda.synchronize()
    assert torch.equal(c.lens, full)
    for i in (0, 1, 2, 30, 31, 32, 63, 64, 88, 89):
        c.lens.fill_(128 + i + 1)
        c.check(outs[i], c.plain(), f"step {i}")
    assert binding.get_device_errors() == 0


def test_binding_refuses():
    c = Case([4], [40], [5] * 4, 8, 2, 64, 16)
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    bad = [dict(q=c.q.float()), dict(q=c.q[:3]), dict(q=c.q[..., ::2]), dict(k=c.k.float()), dict(v=c.v[:-1]),
           dict(table=c.table.long()), dict(table=c.table[:3]), dict(lens=c.lens.long()), dict(lens=c.lens[:3].contiguous()),
           dict(prefix=torch.zeros(2, dtype=torch.int32, device="cuda"))]
    empty = torch.empty((2 ** 31, 0, 2, 64), dtype=torch.bfloat16, device="cuda")
    bad.append(dict(k=empty, v=empty))   # more pages than 32 bits count
    for change in bad:
        kept = {n: getattr(c, n) for n in change}
        for n, t in change.items():
            setattr(c, n, t)
        with pytest.raises(ValueError):
            c.run()
        for n, t in kept.items():
            setattr(c, n, t)
    for kw in (dict(out=torch.empty((4, 8, 32), dtype=torch.bfloat16, device="cuda")), dict(out=c.q.float()),
               dict(workspace=torch.empty((1 << 16, 2), dtype=torch.uint8, device="cuda")[:, 0]), dict(max_prefix_len=-1),
               dict(prefix_splits=-1)):
        with pytest.raises(ValueError):
            c.run(**kw)
    for kw, status in ((dict(workspace=ws), 4), (dict(max_prefix_len=c.table.shape[1] * 16 + 1), 2),
                       (dict(max_suffix_len=c.table.shape[1] * 16 + 1), 2), (dict(scale=float("inf")), 2)):
        with pytest.raises(binding.DapError) as e:
            c.run(**kw)
        assert e.value.status == status
    for n in ("q", "table", "lens"):
        kept = getattr(c, n)
        setattr(c, n, kept.cpu())
        with pytest.raises(binding.DapError) as e:
            c.run()
        assert e.value.status is None
        setattr(c, n, kept)
    c.check(c.run(), c.plain())
    assert binding.get_device_errors() == 0


def test_graphs_that_share_a_workspace():
    """Two captured steps on one workspace, replayed with other lengths and prefixes than those captured, and on another
    stream; the bounds hold for all of them."""
    a = Case([30], [400], [17] * 30, 8, 2, 128, 16, seed=1)
    b = Case([7, 5], [200, 333], [50] * 12, 16, 2, 256, 16, seed=2)
    kw = dict(max_prefix_len=450, max_suffix_len=60)
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
    a.lens -= 3
    a.lens[4] = 0
    b.lens[:7] -= 60
    b.prefix[0] = 180
    b.lens[0:7] = torch.tensor([180, 181, 190, 195, 200, 180, 0], dtype=torch.int32)
    refs = [c.plain() if c is a else None for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(10):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    a.check(outs[0], refs[0])
    # b's sequences now read positions 180 .. 199 through their own tables, as the first sequence's they share the pages
    # of whole tiles: compare with the call outside a graph
    want = b.run(**kw)
    assert torch.equal(torch.nan_to_num(want), torch.nan_to_num(outs[1]))
    assert bool((outs[1][6] == 0).all())


def test_two_streams_with_a_workspace_each():
    cs = [Case([20], [300], [7 * j for j in range(20)], 8, 2, 128, 16, seed=4),
          Case([20], [500], [3 * j for j in range(20)], 8, 2, 64, 12, seed=5)]
    alone = [c.run() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    ws = [torch.empty(binding.workspace_bytes_shared(c.plan, max_prefix_len=c.max_prefix, max_suffix_len=c.max_suffix),
                      dtype=torch.uint8, device="cuda") for c in cs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for c, s, w in zip(cs, streams, ws):
            with torch.cuda.stream(s):
                outs.append(c.run(workspace=w))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, alone[i % 2])


def test_a_given_stream_keeps_what_the_call_allocates():
    """The call's own workspace is not handed to the current stream while the given stream still uses it."""
    c = Case([20], [300], [7 * j for j in range(20)], 8, 2, 128, 16, seed=6)
    want = c.run()
    n = binding.workspace_bytes_shared(c.plan, max_prefix_len=c.max_prefix, max_suffix_len=c.max_suffix)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            torch.cuda._sleep(5_000_000)   # (some milliseconds)
        got = c.run(stream=side)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.current_stream().synchronize()
        side.synchronize()
        assert torch.equal(got, want)
        del junk


def test_q_whose_heads_are_further_apart_than_its_sequences():
    c = Case([40], [150], [3] * 40, 16, 2, 128, 16, seed=7)
    want = c.run()
    c.q = c.q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    out = torch.empty((16, 40, 128), dtype=torch.bfloat16, device="cuda").permute(1, 0, 2)
    assert torch.equal(c.run(out=out), want)


def test_store_restore_and_decode():
    """The operators together: a prompt is quantised into the e4m3 cache, read back into a run of bf16 pages, and shared by a
    batch whose sequences append their own tokens behind it."""
    Hq, Hkv, D, ps, P, B = 16, 2, 128, 16, 200, 9
    g = torch.Generator().manual_seed(77)
    rows = [torch.randn((P, Hkv, D), generator=g).to(torch.bfloat16).cuda() for _ in "kv"]
    n = -(-P // ps)
    i32 = dict(dtype=torch.int32, device="cuda")
    codes = [torch.zeros((n, ps, Hkv, D), dtype=torch.uint8, device="cuda") for _ in "kv"]
    scale = [torch.zeros((n, Hkv, ps), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    run = (torch.randperm(n, generator=g).to(torch.int32).view(1, n).cuda(), torch.tensor([0, P], **i32), torch.zeros(1, **i32))
    binding.kv_append_paged_fp8_multi(*rows, *codes, *scale, *run)
    c = Case([B], [P], [1] * B, Hq, Hkv, D, ps)
    pool = c.k.shape[0]
    c.k = torch.cat([c.k, torch.full((n, ps, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")])
    c.v = torch.cat([c.v, torch.full((n, ps, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")])
    binding.kv_read_paged_fp8(*codes, *scale, *run, k_out=c.k[pool:].view(-1, Hkv, D)[:P], v_out=c.v[pool:].view(-1, Hkv, D)[:P])
    whole = P // ps
    c.table[:, :whole] = torch.arange(pool, pool + whole, **i32)
    c.table[0, whole] = pool + whole           # the first sequence's copy of the page that the prefix ends in
    new = [torch.randn((B, Hkv, D), generator=g).to(torch.bfloat16).cuda() for _ in "kv"]
    binding.kv_append_paged(*new, c.k, c.v, c.table, torch.full((B,), P, **i32))
    out = c.run()
    c.check(out, c.plain())
    # against the prompt as it was before its rounding to 8 bits: a value is off by 2^-4 of itself at most
    for t in range(P):
        c.k[pool + t // ps, t % ps], c.v[pool + t // ps, t % ps] = rows[0][t], rows[1][t]
    want, A = c.plain()
    assert float((out.double() - want).norm() / want.norm()) < 0.1
    assert binding.get_device_errors() == 0
