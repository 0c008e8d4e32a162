"""Every kernel that reads a block table, a slot map or rows, launched directly behind the resize or append that wrote them, with
no other kernel and no wait between: the resize lets the next kernel start at once, so that one is resident before the tables are
written.  The same calls one at a time, on tables made in Python, give the bits that have to come out."""
import random

import pytest
import torch

from paged_kv_cache_298_gb300 import binding
from test_tables_gpu import Pool, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    binding.get_device_errors(clear=True)
    yield


class Steps:
    """Steps of a batch whose pages all change from step to step, each with one call on the new table."""

    def __init__(self, ps, D, seed):
        r = random.Random(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ps, self.B, self.Hq, self.Hkv, self.D, self.most = ps, 20, 16, 4, D, 400
        B, Hkv, wide = self.B, self.Hkv, -(-self.most // ps) + 1
        self.pool = Pool([0] * B, ps, wide, B * wide, seed=seed)
        P = self.pool.num_pages
        bf = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.k, self.v, self.rows = bf(P, ps, Hkv, D), bf(P, ps, Hkv, D), [bf(B * self.most, Hkv, D) for _ in "kv"]
        self.codes = [torch.randint(0, 0x77, (P, ps, Hkv, D), generator=g, device="cuda", dtype=torch.uint8) for _ in "kv"]
        self.factors = [bf(P, Hkv, ps).abs() for _ in "kv"]
        self.latent = torch.zeros((P, ps, 256), dtype=torch.uint8, device="cuda"), bf(P * ps)
        self.latent_rows = bf(B * self.most, 256)
        self.zero, self.none = ints([0] * B), [0] * B
        self.q = {n: bf(B * n, self.Hq, D) for n in (1, 2, 40)}
        self.parents = {n: ints([-1 if i % 7 == 0 else i - 1 for i in range(n)] * B) for n in (1, 2, 40)}
        self.multi = {n: binding.MultiPlan([n] * B, self.Hq, Hkv, "cuda", D=D) for n in (2, 40)}
        self.span = {n: binding.SpanPlan([n] * B, self.Hq, Hkv, D, "cuda") for n in (1, 2, 40)}
        self.two = binding.SpanPlan([40] * B, self.Hq, Hkv, D, "cuda", tokens_per_tile=256 * Hkv // self.Hq)
        self.shared = binding.SharedPlan([B // 2, B - B // 2], self.Hq, Hkv, D, "cuda")
        self.prefix, self.path, self.five = ints([50, 64]), ints([[3, 9, 20, 21, 60]] * B), ints([5] * B)
        self.lens = [[r.randint(64, self.most) for _ in range(B)] for _ in self.calls()]
        self.gpu_lens = [ints(x) for x in self.lens]

    def calls(self):
        m = dict(max_kv_len=self.most)

        def attend(name, n, **kw):
            call = getattr(binding, "decode_attn_paged" + name)
            if name == "_multi":
                return lambda t, lens, ip, sl: call(self.q[n], self.k, self.v, t, lens, self.multi[n], **m, **kw)
            if name == "_window":
                return lambda t, lens, ip, sl: call(self.q[n], self.k, self.v, t, lens, self.span[n], **m, **kw)
            if name == "_tree":
                plan = kw.pop("plan", None)
                return lambda t, lens, ip, sl: call(self.q[n], self.k, self.v, t, lens, self.parents[n], plan or self.span[n],
                                                    **m, **kw)
            return lambda t, lens, ip, sl: call(self.q[1], self.k, self.v, t, lens, **m, **kw)

        def e4m3(S):
            return lambda t, lens, ip, sl: binding.decode_attn_paged_fp8kv(self.q[1], *self.codes, *self.factors, t, lens,
                                                                           num_splits=S, **m)

        def write_runs(t, lens, ip, sl):
            n = sl.numel()
            binding.kv_append_paged_fp8_multi(self.rows[0][:n], self.rows[1][:n], *self.codes, *self.factors, t, ip, self.zero)
            return binding.decode_attn_paged_fp8kv(self.q[1], *self.codes, *self.factors, t, lens, num_splits=2, **m)

        def read_runs(t, lens, ip, sl):
            return binding.kv_read_paged_fp8(*self.codes, *self.factors, t, ip, self.zero, total_tokens=sl.numel())

        def one_a_sequence(t, lens, ip, sl):
            binding.kv_append_paged(self.rows[0][:self.B], self.rows[1][:self.B], self.k, self.v, t, self.zero)
            binding.kv_append_paged_fp8(self.rows[0][:self.B], self.rows[1][:self.B], *self.codes, *self.factors, t, self.zero)
            return (binding.decode_attn_paged_fp8kv(self.q[1], *self.codes, *self.factors, t, lens, num_splits=1, **m),
                    binding.decode_attn_paged(self.q[1], self.k, self.v, t, lens, num_splits=1, **m))

        def through_slots(t, lens, ip, sl):
            n, one = sl.numel(), (self.k.shape[0] * self.ps, 1, self.Hkv, self.D)
            binding.kv_append_fp8(self.latent_rows[:n], *self.latent, sl)
            binding.kv_append_paged_fp8_multi(self.rows[1][:n], self.rows[0][:n], *self.codes, *self.factors, t, ip, self.zero)
            return binding.kv_read_paged_fp8(*self.codes, *self.factors, t, ip, self.zero, total_tokens=n), self.latent[0].clone()

        def commit(t, lens, ip, sl):
            binding.kv_commit_paged(self.k, self.v, t, self.zero, self.path, self.five)
            return binding.decode_attn_paged(self.q[1], self.k, self.v, t, lens, num_splits=1, **m)
        out = [attend("", 1, num_splits=S) for S in (0, 1, 3, binding.SPLITS_BALANCED)]
        out += [attend("_multi", n, num_splits=S) for n in (2, 40) for S in (1, 2)]
        out += [attend("_window", n, window=100, sinks=5, num_splits=S) for n in (1, 2, 40) for S in (0, 1, 3)]
        out += [attend("_tree", n, num_splits=S) for n in (2, 40) for S in (1, 3, 9)]
        if self.D <= 128:
            out += [attend("_tree", 40, plan=self.two, num_splits=S) for S in (1, 3)]
        out += [e4m3(1), e4m3(3), write_runs, read_runs, one_a_sequence, through_slots, commit, read_runs]
        out += [lambda t, lens, ip, sl, a=a, b=b: binding.decode_attn_paged_shared(
            self.q[1], self.k, self.v, t, lens, self.prefix, self.shared, max_prefix_len=64, max_suffix_len=self.most,
            prefix_splits=a, suffix_splits=b) for a, b in ((1, 1), (1, 4))]
        return out

    def state(self):
        return [self.k, self.v, *self.codes, *self.factors, self.latent[0], self.latent[1]]

    def keep(self):
        return [x.clone() for x in self.state() + list(self.pool.gpu)]

    def restore(self, kept):
        for x, y in zip(self.state() + list(self.pool.gpu), kept):
            x.copy_(y)

    def behind(self):
        """All steps without a wait: pages returned, others taken, and at once the call."""
        table, free, count = self.pool.gpu
        outs, old = [], self.zero
        for call, new, lens in zip(self.calls(), self.gpu_lens, self.lens):
            binding.kv_resize_paged(old, self.zero, table, free, count, page_size=self.ps)
            ip, sl = binding.kv_resize_paged(self.zero, new, table, free, count, page_size=self.ps, total_rows=sum(lens))
            outs.append(call(table, new, ip, sl))
            old = new
        binding.kv_resize_paged(old, self.zero, table, free, count, page_size=self.ps)
        return outs

    def alone(self):
        """The same, one call at a time on tables, boundaries and slots made in Python."""
        outs = []
        for call, new, lens in zip(self.calls(), self.gpu_lens, self.lens):
            self.pool.python(self.none)
            ip, sl = self.pool.python(lens)
            args = ints(self.pool.table).view(self.B, -1), new, ints(ip), torch.tensor(sl, device="cuda")
            torch.cuda.synchronize()
            outs.append(call(*args))
            torch.cuda.synchronize()
        self.pool.python(self.none)
        return outs


def same(a, b):
    flat = lambda x: [x] if isinstance(x, torch.Tensor) else [t for y in x for t in flat(y)]  # noqa: E731
    a, b = flat(a), flat(b)
    assert len(a) == len(b)
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), i


@pytest.mark.parametrize("D,ps", [(64, 12), (128, 16), (128, 64), (256, 5), (256, 128)])
def test_calls_behind_a_resize(D, ps):
    s = Steps(ps, D, seed=ps)
    before = s.keep()
    want = s.alone()
    after = [x.clone() for x in s.state()]
    assert not any(bool(torch.isnan(x).any()) for x in want[:10])
    s.restore(before)
    got = s.behind()
    torch.cuda.synchronize()
    same(got, want)
    same(s.state(), after)
    s.pool.same()
    # and captured: every edge between these kernels is the same early start
    s.restore(before)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.behind()
    for _ in range(3):
        s.restore(before)
        graph.replay()
        torch.cuda.synchronize()
        same(got, want)
        same(s.state(), after)
        s.pool.same()
    assert binding.get_device_errors() == 0


@pytest.mark.parametrize("ps", [12, 16])
def test_a_long_resize_in_front(ps):
    """A resize of many rows, two launches on the whole device, and the call behind it."""
    s = Steps(ps, 128, seed=1)
    table, free, count = s.pool.gpu
    rows = 200_000
    slots = torch.empty(rows, dtype=torch.int64, device="cuda")
    calls, want, got = s.calls()[:10], [], []
    before = s.keep()
    old = s.zero
    for call, new in zip(calls, s.gpu_lens):
        binding.kv_resize_paged(old, s.zero, table, free, count, page_size=s.ps)
        ip, sl = binding.kv_resize_paged(s.zero, new, table, free, count, page_size=s.ps, total_rows=rows, slots=slots)
        got.append(call(table, new, ip, sl))
        old = new
    torch.cuda.synchronize()
    s.restore(before)
    for call, new, lens in zip(calls, s.gpu_lens, s.lens):
        s.pool.python(s.none)
        s.pool.python(lens)
        t = ints(s.pool.table).view(s.B, -1)
        torch.cuda.synchronize()
        want.append(call(t, new, None, None))
        torch.cuda.synchronize()
    same(got, want)
    assert binding.get_device_errors() == 0
