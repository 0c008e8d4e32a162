"""Batches over a paged cache for the tests of windowed and tree attention, and the operators in 64 bits with the bound that a
kernel's output keeps.

The bound of an output, with A = sum_t w_t |v_t| (w: the softmax weights): a weight is rounded to bf16 for the product with V
(at most 2^-8 of it), and the normaliser sums the weights before or after that rounding, so that at most 2 * 2^-8 A comes
of it; a score is a binary32 sum of D products (each product and sum off by at most 2^-24 of the absolute sum so far: in all
at most (D + 2) 2^-24 scale sum |q k|, by which, to first order, a weight is off relatively, once in the numerator and once in
the normaliser); exponentials, merges and the sums of weights and values stay below 2^-16 A for up to 2^7 additions of 2^-24
each in a row of partial sums (a warp's or thread's lane sums its keys in steps of tiles); the output is rounded to bf16
(2^-8 |out|), where below the smallest normal number 2^-134 may be lost."""
import math
import random

import torch


def parents_of(n, kind, r):
    """Parents of a tree's n nodes: 'chain', 'star' (children of one root), 'roots' (children of the context) or 'mixed'."""
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1) if n else []
    if kind == "roots":
        return [-1] * n
    return [-1 if i == 0 or r.random() < 0.15 else r.randrange(max(0, i - 9), i) for i in range(n)]


class Batch:
    """Sequences with ctx[b] places in front of counts[b] new tokens, in pages at random places of a pool; K and V of
    places that exist are random, all other rows of the pool are NaN, and table entries that name no page are -1."""

    def __init__(self, ctx, counts, Hq, Hkv, D, ps, seed=0, kind=None, qmag=1.0):
        r = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        gc = torch.Generator(device="cuda").manual_seed(seed)
        self.ctx, self.counts, self.Hq, self.Hkv, self.D, self.ps = list(ctx), list(counts), Hq, Hkv, D, ps
        self.B, self.total = len(ctx), sum(counts)
        self.lens = [c + n for c, n in zip(ctx, counts)]
        need = [-(-n // ps) for n in self.lens]
        pool = sum(need) + 3
        order = torch.randperm(pool, generator=g).tolist()
        width = max(1, max(need)) + 1
        self.rows, at = [], 0
        table = torch.full((self.B, width), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            self.rows.append(order[at:at + n])
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.pool = pool
        self.table = table.cuda()
        self.k = torch.full((pool, ps, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v = torch.full_like(self.k, float("nan"))
        for b, n in enumerate(self.lens):
            page, slot = self.places(b, n)
            for x in (self.k, self.v):
                x[page, slot] = torch.randn((n, Hkv, D), generator=gc, device="cuda").to(torch.bfloat16)
        self.q = (torch.randn((self.total, Hq, D), generator=gc, device="cuda") * qmag).to(torch.bfloat16)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.max_len = max(1, max(self.lens))
        self.trees = None
        if kind is not None:
            self.trees = [parents_of(n, kind, r) for n in counts]
            self.parents = torch.tensor([p for t in self.trees for p in t], dtype=torch.int32, device="cuda")

    def places(self, b, n):
        t = torch.arange(n)
        page = torch.tensor(self.rows[b] or [0])[t // self.ps]
        return page.cuda(), (t % self.ps).cuda()

    def seen(self, b, window, sinks):
        """[new tokens, places]: which places each new token of sequence b sees."""
        c, n = self.ctx[b], self.counts[b]
        place = torch.arange(c + n)
        see = torch.ones((n, c + n), dtype=torch.bool)
        if self.trees is None:
            pos = place
            see &= place[None] <= (c + torch.arange(n))[:, None]
        else:
            depth, line = [], torch.zeros((n, n), dtype=torch.bool)
            for i, p in enumerate(self.trees[b]):
                depth.append(depth[p] + 1 if p >= 0 else 0)
                if p >= 0:
                    line[i] = line[p]
                line[i, i] = True
            pos = torch.cat([place[:c], c + torch.tensor(depth, dtype=torch.int64)])
            see[:, c:] = line
        if window:
            see &= (pos < sinks)[None] | (pos[None] > pos[c:, None] - window)
        return see.cuda()

    def reference(self, window=0, sinks=0, scale=None):
        """(output, bound of its error) in 64 bits."""
        scale = 1.0 / math.sqrt(self.D) if scale is None else scale
        G = self.Hq // self.Hkv
        out = torch.zeros((self.total, self.Hq, self.D), dtype=torch.float64, device="cuda")
        bound, at = torch.zeros_like(out), 0
        for b, n in enumerate(self.counts):
            if n == 0:
                continue
            page, slot = self.places(b, self.lens[b])
            k = self.k[page, slot].double().repeat_interleave(G, dim=1)   # [place, Hq, D]
            v = self.v[page, slot].double().repeat_interleave(G, dim=1)
            q = self.q[at:at + n].double()
            see = self.seen(b, window, sinks)
            any_seen = see.any(0)                                          # places that nobody sees may hold anything
            k, v = k.masked_fill(~any_seen[:, None, None], 0.0), v.masked_fill(~any_seen[:, None, None], 0.0)
            s = torch.einsum("ihd,thd->hit", q, k) * scale
            w = torch.softmax(s.masked_fill(~see, -math.inf), dim=-1)
            o, A = torch.einsum("hit,thd->ihd", w, v), torch.einsum("hit,thd->ihd", w, v.abs())
            e = (torch.einsum("ihd,thd->hit", q.abs(), k.abs()) * abs(scale)).masked_fill(~see, 0.0).amax(-1).T[..., None]
            out[at:at + n] = o
            bound[at:at + n] = 2.0 ** -8 * o.abs() + A * (2 * 2.0 ** -8 + 2 * (self.D + 2) * 2.0 ** -24 * e + 2.0 ** -16) + 2.0 ** -134
            at += n
        return out, bound

    def check(self, got, window=0, sinks=0, scale=None, what=""):
        ref, bound = self.reference(window, sinks, scale)
        assert got.shape == ref.shape and got.dtype == torch.bfloat16
        assert not torch.isnan(got).any(), what
        over = ((got.double() - ref).abs() / bound).max().item() if ref.numel() else 0.0
        assert over <= 1.0, (what, over)
