"""Cases of speculative and windowed decoding over the paged K/V cache, each in its plain form and through the library.

Four operators that a serving step with drafted tokens, or a model with a sliding window, makes in a row:

* ``resize``: pages taken and returned, block tables and slot maps of a batch whose lengths change, on the GPU;
* ``tree``: attention of the nodes of drafted token trees over the cache, with or without a window;
* ``window``: attention with a sliding window and a few first tokens that stay visible, for one or many new tokens;
* ``commit``: the accepted path of each tree moved to the places behind the context.

``own`` selects the library's calls; otherwise the plain form runs (float32 torch operations).
"""
import math
import random

import torch

own = False

DEV = "cuda"
NODES_MOST = 256  # nodes of one tree


# ---- cases ----------------------------------------------------------------------------------

def _resize(name, seqs, mode, lo, hi, step, ps, wide, mix):
    return dict(name=name, op="resize", seqs=seqs, mode=mode, lo=lo, hi=hi, step=step, ps=ps, wide=wide, mix=mix)


def _tree(name, seqs, nodes, ragged, Hq, Hkv, D, ps, lo, hi, window, sinks, mix):
    return dict(name=name, op="tree", seqs=seqs, nodes=nodes, ragged=ragged, Hq=Hq, Hkv=Hkv, D=D, ps=ps, lo=lo, hi=hi,
                window=window, sinks=sinks, mix=mix)


def _window(name, seqs, tokens, Hq, Hkv, D, ps, lo, hi, window, sinks, mix):
    return dict(name=name, op="window", seqs=seqs, tokens=tokens, Hq=Hq, Hkv=Hkv, D=D, ps=ps, lo=lo, hi=hi, window=window,
                sinks=sinks, mix=mix)


def _commit(name, seqs, nodes, path, Hkv, D, ps, lo, hi, mix):
    return dict(name=name, op="commit", seqs=seqs, nodes=nodes, path=path, Hkv=Hkv, D=D, ps=ps, lo=lo, hi=hi, mix=mix)


def listed():
    return [
        # a step of a few sequences with eight drafted tokens each: latency
        _resize("resize_draft", 16, "draft", 256, 4096, 8, 16, True, 1),
        # a step of a busy server: some requests end, some are admitted with their prompts, the others go on by one token
        _resize("resize_mixed", 301, "mixed", 100, 4096, 1, 12, False, 2),
        # prompts of a large batch admitted at once: the slot map is most of the work
        _resize("resize_admit", 256, "admit", 1000, 8192, 0, 16, True, 3),
        # two sequences, five drafted nodes each, a short context: launch latency
        _tree("tree_tiny", 2, 5, False, 8, 2, 64, 16, 40, 130, 0, 0, 4),
        # a small batch with drafts of 16 nodes: an ordinary verification step
        _tree("tree_b16", 16, 16, False, 32, 8, 128, 16, 2048, 2048, 0, 0, 5),
        # a large ragged batch with drafts of 64 nodes: K/V streamed once, and a large product
        _tree("tree_b64", 64, 64, False, 32, 8, 128, 64, 256, 4096, 0, 0, 6),
        # wide heads, pages of 12, drafts of unequal size (none and one node among them), a window with sinks
        _tree("tree_d256_page12", 9, 21, True, 16, 4, 256, 12, 1, 5000, 1000, 4, 7),
        # a decode step behind long contexts: only the window and the sinks are read
        _window("window_step", 64, 1, 32, 8, 128, 16, 1024, 32768, 1024, 4, 8),
        # a short window and few sequences: launch latency
        _window("window_short", 4, 1, 64, 8, 64, 16, 100, 5000, 128, 0, 9),
        # one chunk of each of several prompts, odd lengths: bound by its products
        _window("window_chunk", 4, 1021, 32, 8, 128, 16, 2000, 6000, 2048, 16, 10),
        # a few accepted tokens of a small batch: latency
        _commit("commit_step", 16, 16, 5, 8, 128, 16, 500, 2048, 11),
        # long accepted paths of a large batch
        _commit("commit_b256", 256, 64, 24, 8, 128, 64, 16, 300, 12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["resize", "tree", "tree", "window", "window", "commit"])
    ps = rng.choice([8, 16, 16, 24, 32, 64, 128, 1, 5, 12, 100])
    mix = rng.randrange(1 << 20)
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 4, 4, 8])
    D = rng.choice([64, 128, 128, 256])
    if op == "resize":
        mode = rng.choice(["draft", "mixed", "admit"])
        seqs = _log(rng, 1, 1000)
        hi = _log(rng, 4, min(8192, 1200000 // seqs))
        c = _resize("", seqs, mode, rng.randint(1, hi), hi, rng.randint(1, 64), ps, rng.random() < 0.5, mix)
    elif op == "commit":
        nodes = _log(rng, 1, NODES_MOST)
        c = _commit("", _log(rng, 1, 256), nodes, rng.randint(1, min(nodes, 32)), Hkv, D, ps, rng.randint(0, 40),
                    rng.randint(41, 300), mix)
    else:
        # a listed case's K/V and its products bound those of a drawn one
        def fits():
            keys = min(hi, window + sinks) + tokens if window else hi + tokens
            return (seqs * (hi + tokens) * Hkv * D <= 64 * 4200 * 8 * 128
                    and seqs * tokens * keys * Hkv * G * D <= 64 * 64 * 2300 * 32 * 128
                    and seqs * tokens * (keys + tokens) * Hkv * G <= 64 * 64 * 4200 * 32)
        seqs = _log(rng, 1, 200)
        tokens = _log(rng, 1, NODES_MOST) if op == "tree" else rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 2, 1500)])
        hi = _log(rng, 1, 32768)
        window = _log(rng, 4, 8192) if op == "window" or rng.random() < 0.3 else 0
        sinks = rng.choice([0, 4, rng.randint(1, 130)]) if window else 0
        while not fits():
            hi, tokens = max(1, hi * 3 // 4), max(1, tokens * 7 // 8)
            seqs = max(1, seqs * 7 // 8)
        lo = rng.randint(1, hi)
        if op == "tree":
            c = _tree("", seqs, tokens, rng.random() < 0.5, G * Hkv, Hkv, D, ps, lo, hi, window, sinks, mix)
        else:
            c = _window("", seqs, tokens, G * Hkv, Hkv, D, ps, lo, hi, window, sinks, mix)
    del c["name"]
    return c


def _lengths(case):
    """(lengths before, lengths after) of every sequence of a resize."""
    r = random.Random(case["mix"])
    old, new = [], []
    for _ in range(case["seqs"]):
        n = r.randint(case["lo"], case["hi"])
        kind = r.random() if case["mode"] == "mixed" else 0.5
        if case["mode"] == "admit" or kind < 0.03:
            a, b = 0, n
        elif kind > 0.97:
            a, b = n, 0
        else:
            a, b = n, n + case["step"]
        old.append(a)
        new.append(b)
    return old, new


def _contexts(case):
    """(keys in front of the new tokens, new tokens) of every sequence."""
    r = random.Random(case["mix"])
    ctx = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    if case["op"] == "window":
        return ctx, [case["tokens"]] * case["seqs"]
    if case["op"] == "tree" and case["ragged"]:
        return ctx, [r.choice([0, 1, r.randint(1, case["nodes"]), case["nodes"]]) for _ in ctx[:-1]] + [case["nodes"]]
    return ctx, [case["nodes"]] * case["seqs"]


def _parents(case, counts):
    """Parents of every tree's nodes, in front of their children; -1: the context.  Wide at the top, as drafts are."""
    r = random.Random(case["mix"] + 1)
    out = []
    for n in counts:
        out.append([-1 if i == 0 or r.random() < 1.0 / (1 + i) else r.randint(max(0, i // 2 - 2), i - 1) for i in range(n)])
    return out


def _paths(case):
    """Accepted nodes of every tree, in order."""
    r = random.Random(case["mix"] + 1)
    return [sorted(r.sample(range(case["nodes"]), r.randint(1, case["path"]))) for _ in range(case["seqs"])]


# ---- inputs ----------------------------------------------------------------------------------

def _rows(shape, g, spread=True):
    """bf16 rows as projections give them: a scale of its own for each head, some channels larger than others."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    if spread:
        x *= 1.0 + 3.0 * (torch.rand(shape[-1], generator=g, device=DEV) > 0.95)
        x *= 0.5 + torch.rand(shape[-2:-1] + (1,), generator=g, device=DEV)
    return x.to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _pages(lens, ps, gen, spare):
    """Block table of sequences with the given lengths over a pool in random order, its pages, and those not used."""
    need = [-(-n // ps) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=gen).tolist()
    rows, at = [], 0
    for n in need:
        rows.append(order[at:at + n])
        at += n
    return rows, len(order), order[at:]


def _table(rows, width):
    return _ints([r + [0] * (width - len(r)) for r in rows])


def _prepare_resize(case, seed):
    gen = torch.Generator().manual_seed(seed)
    old, new = _lengths(case)
    ps = case["ps"]
    taken = sum(max(0, -(-b // ps) + a // -ps) for a, b in zip(old, new))
    rows, pool, spare = _pages(old, ps, gen, taken + 5)
    width = max(-(-max(a, b) // ps) for a, b in zip(old, new)) + 1
    return dict(op="resize", old=_ints(old), new=_ints(new), ps=ps, table=_table(rows, width),
                free=_ints(spare + [0] * (pool - len(spare))), count=_ints([len(spare)]),
                rows=sum(max(0, b - a) for a, b in zip(old, new)), back=sum(max(0, a - b) for a, b in zip(old, new)),
                kind=torch.int64 if case["wide"] else torch.int32)


def _prepare_cache(case, seed):
    gen = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    ps, Hkv, D = case["ps"], case["Hkv"], case["D"]
    ctx, counts = _contexts(case)
    lens = [c + n for c, n in zip(ctx, counts)]
    rows, pool, _ = _pages(lens, ps, gen, 3)
    s = dict(op=case["op"], k=_rows((pool, ps, Hkv, D), g), v=_rows((pool, ps, Hkv, D), g, spread=False),
             table=_table(rows, max(1, max(map(len, rows)))), ctx=_ints(ctx), lens=_ints(lens))
    if case["op"] == "commit":
        paths = _paths(case)
        s["path"] = _ints([p + [0] * (case["path"] - len(p)) for p in paths])
        s["accepted"] = _ints([len(p) for p in paths])
        return s
    Hq = case["Hq"]
    s |= dict(q=_rows((sum(counts), Hq, D), g, spread=False), max_len=max(lens), total=sum(lens), scale=1.0 / math.sqrt(D),
              window=case["window"], sinks=case["sinks"], most=max(counts),
              # the packed row of token i of each sequence, short ones filled with row 0; and back
              at=torch.tensor([[sum(counts[:b]) + i if i < n else 0 for i in range(max(counts))] for b, n in enumerate(counts)],
                              device=DEV),
              seq=torch.tensor([b for b, n in enumerate(counts) for _ in range(n)], dtype=torch.int64, device=DEV),
              tok=torch.tensor([i for n in counts for i in range(n)], dtype=torch.int64, device=DEV))
    if case["op"] == "tree":
        s["parents"] = _ints([p for tree in _parents(case, counts) for p in tree])
    if own:
        from paged_kv_cache_298_gb300 import binding
        s["plan"] = binding.SpanPlan(counts, Hq, Hkv, D, DEV)
        n = binding.workspace_bytes_span(s["plan"], max_kv_len=s["max_len"], window=s["window"], sinks=s["sinks"],
                                         tree=case["op"] == "tree", total_kv=s["total"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return s


def prepare(case, seed):
    return _prepare_resize(case, seed) if case["op"] == "resize" else _prepare_cache(case, seed)


# ---- plain forms -------------------------------------------------------------------------------

def _resize_plain(s, old, new, rows):
    ps, table, free, count = s["ps"], s["table"], s["free"], s["count"]
    old, new = old.long(), new.long()
    had, has = (old + ps - 1) // ps, (new + ps - 1) // ps
    i = torch.arange(table.shape[1], device=DEV)
    # pages behind the new end go on top of the stack, in order; then the top ones are taken, in order
    gone = (i >= has[:, None]) & (i < had[:, None])
    end = free.numel()
    wide = torch.cat([free, free[:1]])
    place = torch.where(gone, count + gone.flatten().cumsum(0).view_as(gone) - 1, end)
    wide.scatter_(0, place.flatten().long(), table.flatten())
    come = (i >= had[:, None]) & (i < has[:, None])
    height = count + gone.sum() - come.sum()
    place = torch.where(come, height + come.flatten().cumsum(0).view_as(come) - 1, end)
    table.copy_(torch.where(come, wide[place], table))
    free.copy_(wide[:end])
    count.copy_(height)
    more = (new - old).clamp(min=0)
    indptr = torch.cat([torch.zeros_like(more[:1]), more.cumsum(0)])
    r = torch.arange(rows, device=DEV)
    b = torch.searchsorted(indptr[1:].contiguous(), r, right=True)
    pos = old[b] + r - indptr[b]
    slots = table[b, pos // ps].long() * ps + pos % ps
    return indptr.to(torch.int32), slots.to(s["kind"])


def _attend_plain(s, key_pos, see):
    """Attention of the tokens [seq, token] over the keys at key_pos [seq, key] that `see` [seq, token, key] lets through."""
    q, table = s["q"].float(), s["table"].long()
    ps, Hkv, D = s["k"].shape[1:]
    Hq = q.shape[1]
    at = key_pos.clamp(0, table.shape[1] * ps - 1)
    page = table.gather(1, at // ps)
    k, v = (s[x][page, at % ps].float().permute(0, 2, 1, 3) for x in "kv")                       # [seq, Hkv, key, D]
    B, T = s["at"].shape
    qb = q[s["at"]].view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)  # [seq, Hkv, G x token, D]
    w = (qb @ k.transpose(2, 3)).view(B, Hkv, Hq // Hkv, T, -1) * s["scale"]
    w = w.masked_fill_(~see[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    w = w.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = w.sum(-1, keepdim=True)
    out = (w.view(B, Hkv, -1, w.shape[-1]) @ v).view(B, Hkv, Hq // Hkv, T, D) / torch.where(total > 0, total, 1.0)
    return out.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D)[s["seq"], s["tok"]].to(torch.bfloat16)


def _ancestors(s):
    """Which nodes of its tree each node sees [seq, node, node], and how deep it is [seq, node]."""
    B, T = s["at"].shape
    up = torch.zeros((B, T, T + 1), device=DEV)
    up[s["seq"], s["tok"], torch.where(s["parents"] < 0, T, s["parents"].long())] = 1.0
    reach = up[..., :T] + torch.eye(T, device=DEV)
    for _ in range(max(1, (T - 1).bit_length())):  # twice the distance each time
        reach = (reach @ reach).clamp_(max=1.0)
    return reach > 0, reach.sum(-1).long() - 1


def _tree_plain(s):
    T, ctx = s["at"].shape[1], s["ctx"].long()
    reach, depth = _ancestors(s)
    t = torch.arange(s["max_len"], device=DEV)
    node = t - ctx[:, None]                                                                    # [seq, key]
    anc = reach.gather(2, node.clamp(0, T - 1)[:, None].expand(-1, T, -1)) & (node < T)[:, None]
    see = torch.where(node[:, None] < 0, torch.ones_like(anc), anc)
    if s["window"]:
        key_pos = torch.where(node < 0, t, ctx[:, None] + depth.gather(1, node.clamp(0, T - 1)))  # a node's is its depth's
        pos = ctx[:, None] + depth
        see = see & ((key_pos[:, None] < s["sinks"]) | (key_pos[:, None] > pos[..., None] - s["window"]))
    return _attend_plain(s, t.expand(len(ctx), -1), see)


def _window_plain(s):
    B, T = s["at"].shape
    ctx, sinks, window = s["ctx"].long()[:, None], s["sinks"], s["window"]
    i = torch.arange(sinks + window + T - 1, device=DEV)
    t = torch.where(i < sinks, i, ctx - window + 1 + i - sinks)                                # [seq, key]
    pos = ctx + torch.arange(T, device=DEV)
    inside = (t[:, None] > pos[..., None] - window) & (t[:, None] >= sinks)
    see = ((i < sinks) | inside) & (t[:, None] <= pos[..., None])
    return _attend_plain(s, t, see)


def _commit_plain(s):
    ps = s["k"].shape[1]
    j = torch.arange(s["path"].shape[1], device=DEV)
    to, come = s["ctx"].long()[:, None] + j, s["ctx"].long()[:, None] + s["path"].long()
    come = torch.where(j < s["accepted"][:, None], come, to)  # (a place behind the path takes its own row)
    page, slot, page0, slot0 = (x for t in (to, come) for x in (s["table"].long().gather(1, t // ps), t % ps))
    for x in "kv":
        s[x][page, slot] = s[x][page0, slot0]


def run(s):
    if own:
        from paged_kv_cache_298_gb300 import binding
        if s["op"] == "tree":
            return binding.decode_attn_paged_tree(s["q"], s["k"], s["v"], s["table"], s["lens"], s["parents"], s["plan"],
                                                  max_kv_len=s["max_len"], window=s["window"], sinks=s["sinks"],
                                                  scale=s["scale"], total_kv=s["total"], workspace=s["workspace"])
        if s["op"] == "window":
            return binding.decode_attn_paged_window(s["q"], s["k"], s["v"], s["table"], s["lens"], s["plan"],
                                                    max_kv_len=s["max_len"], window=s["window"], sinks=s["sinks"],
                                                    scale=s["scale"], total_kv=s["total"], workspace=s["workspace"])
        if s["op"] == "commit":
            binding.kv_commit_paged(s["k"], s["v"], s["table"], s["ctx"], s["path"], s["accepted"])
            return s["k"], s["v"]

        def resize(old, new, rows):
            return binding.kv_resize_paged(old, new, s["table"], s["free"], s["count"], page_size=s["ps"], total_rows=rows,
                                           slot_dtype=s["kind"])
    else:
        if s["op"] == "tree":
            return _tree_plain(s)
        if s["op"] == "window":
            return _window_plain(s)
        if s["op"] == "commit":
            _commit_plain(s)
            return s["k"], s["v"]

        def resize(old, new, rows):
            return _resize_plain(s, old, new, rows)
    # there and back: what was taken is returned (drafts that were rejected, requests that end), so that a pass ends as it began
    indptr, slots = resize(s["old"], s["new"], s["rows"])
    back_indptr, back_slots = resize(s["new"], s["old"], s["back"])
    return dict(indptr=indptr, slots=slots, back_indptr=back_indptr, back_slots=back_slots, table=s["table"], free=s["free"],
                count=s["count"])


# ---- work ----------------------------------------------------------------------------------------

def _depths(parents):
    out = []
    for p in parents:
        out.append(0 if p < 0 else out[p] + 1)
    return out


def work(case):
    if case["op"] == "resize":
        old, new = _lengths(case)
        ps = case["ps"]
        pages = sum(abs(-(-b // ps) + a // -ps) for a, b in zip(old, new))
        rows = sum(abs(b - a) for a, b in zip(old, new))
        # both ways: lengths read and boundaries written, a page id read and written for each page, a slot for each row
        return {"bytes": 2 * (12 * len(old) + 8 * pages) + rows * (8 if case["wide"] else 4), "flops": rows}
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "commit":
        moved = sum(j != n for p in _paths(case) for j, n in enumerate(p))
        return {"bytes": 8 * moved * Hkv * D, "flops": 0}
    ctx, counts = _contexts(case)
    window, sinks = case["window"], case["sinks"]
    trees = _parents(case, counts) if case["op"] == "tree" else None
    keys = pairs = 0
    for b, (c, n) in enumerate(zip(ctx, counts)):
        if n == 0:
            continue
        first = max(0, c - window + 1) if window else 0
        keys += c + n - max(0, first - sinks)
        for i, d in enumerate(_depths(trees[b]) if trees else range(n)):
            pairs += c + d + 1 if not window else c + d + 1 - max(0, c + d + 1 - window - sinks)
    return {"bytes": 4 * keys * Hkv * D + 4 * sum(counts) * case["Hq"] * D, "flops": 4 * pairs * case["Hq"] * D}


# ---- the definitions in 64 bits --------------------------------------------------------------------

def _exact_resize(case, s):
    free, count, table = s["free"].tolist(), s["count"].item(), s["table"].tolist()
    ps, old, new = case["ps"], s["old"].tolist(), s["new"].tolist()
    out = {}
    for name, before, after in (("", old, new), ("back_", new, old)):
        for b, (x, y) in enumerate(zip(before, after)):
            for i in range(-(-y // ps), -(-x // ps)):
                free[count] = table[b][i]
                count += 1
        count -= sum(max(0, -(-y // ps) + x // -ps) for x, y in zip(before, after))
        take, slots, indptr = count, [], [0]
        for b, (x, y) in enumerate(zip(before, after)):
            for i in range(-(-x // ps), -(-y // ps)):
                table[b][i] = free[take]
                take += 1
            slots += [table[b][t // ps] * ps + t % ps for t in range(x, y)]
            indptr.append(len(slots))
        out[name + "indptr"], out[name + "slots"] = _ints(indptr), torch.tensor(slots, dtype=s["kind"], device=DEV)
    return dict(out, table=_ints(table), free=_ints(free), count=_ints([count]))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "resize":
        return _exact_resize(case, s)
    ps, table = s["k"].shape[1], s["table"].long()
    if case["op"] == "commit":
        out = {x: s[x].double() for x in "kv"}
        for b, (c, path) in enumerate(zip(s["ctx"].tolist(), _paths(case))):
            to = torch.arange(c, c + len(path), device=DEV)
            come = c + torch.tensor(path, device=DEV)
            for x in "kv":
                out[x][table[b][to // ps], to % ps] = s[x][table[b][come // ps], come % ps].double()
        return out["k"], out["v"]
    ctx, counts = _contexts(case)
    trees = _parents(case, counts) if case["op"] == "tree" else None
    G = case["Hq"] // case["Hkv"]
    done, at = [], 0
    for b, (c, n) in enumerate(zip(ctx, counts)):
        if n == 0:
            continue
        place = torch.arange(c + n, device=DEV)
        k, v = (s[x][table[b][place // ps], place % ps].double() for x in "kv")
        depth = torch.tensor(_depths(trees[b]) if trees else list(range(n)), device=DEV)
        pos = torch.cat([place[:c], c + depth])                    # of each key in its own line of tokens
        see = torch.zeros((n, c + n), dtype=torch.bool, device=DEV)
        see[:, :c] = True
        if trees:
            line = torch.zeros((n, n), dtype=torch.bool)
            for i, p in enumerate(trees[b]):
                if p >= 0:
                    line[i] = line[p]
                line[i, i] = True
            see[:, c:] = line.to(DEV)
        else:
            see[:, c:] = torch.ones((n, n), dtype=torch.bool, device=DEV).tril()
        if case["window"]:
            see &= (pos < case["sinks"])[None] | (pos[None] > pos[c:, None] - case["window"])
        q = s["q"][at:at + n].double()
        at += n
        heads = []
        for h in range(case["Hq"]):
            w = q[:, h] @ k[:, h // G].T * s["scale"]
            heads.append(torch.softmax(w.masked_fill(~see, -math.inf), dim=1) @ v[:, h // G])
        done.append(torch.stack(heads, dim=1))
    return torch.cat(done)
