"""Cases of the cache and shared-prefix operators, each in its plain form and through the library.

Three operators over the paged K/V caches:

* ``append``: runs of new tokens are quantised into the e4m3 cache (codes and one bf16 factor per slot and kv head);
* ``read``: runs of the e4m3 cache are read back as bf16 rows;
* ``shared``: single-token attention of a batch whose sequences share a prefix, in one or several groups.

``own`` selects the library's calls; otherwise the plain form runs (float32 torch operations).
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ---- cases ----------------------------------------------------------------------------------

def _append(name, seqs, lo, hi, Hkv, D, ps, start, fused, mix):
    return dict(name=name, op="append", seqs=seqs, lo=lo, hi=hi, Hkv=Hkv, D=D, ps=ps, start=start, fused=fused, mix=mix)


def _read(name, seqs, lo, hi, Hkv, D, ps, start, mix):
    return dict(name=name, op="read", seqs=seqs, lo=lo, hi=hi, Hkv=Hkv, D=D, ps=ps, start=start, mix=mix)


def _shared(name, groups, seqs, Hq, Hkv, D, ps, prefix, lo, hi, pad, mix):
    return dict(name=name, op="shared", groups=groups, seqs=seqs, Hq=Hq, Hkv=Hkv, D=D, ps=ps, prefix=prefix, lo=lo, hi=hi, pad=pad,
                mix=mix)


def listed():
    return [
        # a decode step of a few sequences: one or two tokens each, launch latency
        _append("append_step", 16, 1, 2, 8, 128, 16, 2048, False, 1),
        # one chunk of each of several prompts, K and V being slices of a fused projection; odd lengths
        _append("append_chunks", 12, 100, 1021, 8, 128, 16, 301, True, 2),
        # whole prompts of a batch: the largest write, bound by memory
        _append("append_prompts", 16, 1500, 4096, 8, 128, 64, 0, False, 3),
        # other head dim and a page size that is no multiple of 8
        _append("append_d64_page12", 7, 33, 900, 4, 64, 12, 5, False, 4),
        # a short stored prefix of one sequence: latency
        _read("read_short", 1, 100, 100, 8, 128, 16, 0, 5),
        # ragged runs of a batch, wide heads, starting inside a page
        _read("read_ragged_d256", 9, 200, 1777, 4, 256, 32, 7, 6),
        # long stored prefixes restored before decoding: bound by memory
        _read("read_prefixes", 8, 3000, 8192, 8, 128, 64, 0, 7),
        # two sequences and a short prefix: launch latency
        _shared("shared_tiny", 1, 2, 8, 2, 64, 16, 128, 5, 70, 0, 8),
        # a small batch behind a system prompt, an ordinary serving step
        _shared("shared_b16", 1, 16, 32, 8, 128, 16, 2048, 1, 400, 0, 9),
        # a large ragged batch, padded by empty rows; the suffixes weigh more than the prefix
        _shared("shared_b128", 1, 128, 32, 8, 128, 16, 8192, 16, 1024, 3, 10),
        # a long document asked by many: the prefix is a large matrix product
        _shared("shared_long", 1, 64, 64, 8, 128, 64, 32768, 64, 2048, 0, 11),
        # three prompts shared by groups of unequal size, odd lengths, wide heads, pages of 12
        _shared("shared_groups", 3, 41, 16, 4, 256, 12, 3001, 1, 500, 1, 12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "shared", "shared"])
    D = rng.choice([64, 128, 128, 256])
    ps = rng.choice([8, 16, 16, 24, 32, 64, 128, 5, 12, 100])
    mix = rng.randrange(1 << 20)
    if op != "shared":
        Hkv = rng.choice([1, 2, 3, 4, 8])
        seqs = _log(rng, 1, 64)
        hi = _log(rng, 1, min(8192, 40000 * 1024 // (seqs * Hkv * D)))
        lo = rng.randint(1, hi)
        start = rng.choice([0, rng.randrange(0, 3000)])
        if op == "append":
            c = _append("", seqs, lo, hi, Hkv, D, ps, start, rng.random() < 0.4, mix)
        else:
            c = _read("", seqs, lo, hi, Hkv, D, ps, start, mix)
    else:
        Hkv = rng.choice([1, 2, 3, 4, 8])
        G = rng.choice([1, 2, 4, 8])
        seqs = _log(rng, 2, 160)
        groups = min(rng.choice([1, 1, 1, 2, 4]), seqs)
        prefix = _log(rng, 32, 32768)
        hi = _log(rng, 2, 2048)
        lo = rng.randint(1, hi)
        while seqs * G * Hkv * D * (prefix + hi) > 64 * 64 * 128 * 33000 or seqs * hi * Hkv * D > 64 * 1024 * 8 * 128:
            prefix, hi = max(32, prefix * 3 // 4), max(2, hi * 3 // 4)
            lo = min(lo, hi)
        c = _shared("", groups, seqs, G * Hkv, Hkv, D, ps, prefix, lo, hi, rng.choice([0, 0, min(2, seqs - 1)]), mix)
    del c["name"]
    return c


def _runs(case):
    """Tokens of every sequence's run."""
    r = random.Random(case["mix"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]


def _batch(case):
    """(group sizes, prefix length of each group, length behind the prefix of each sequence, -1: a padded, empty row)."""
    r = random.Random(case["mix"])
    n, left = case["groups"], case["seqs"]
    sizes = []
    for g in range(n):
        most = left - (n - g - 1)
        s = left if g == n - 1 else r.randint(1, max(1, min(most, 2 * left // (n - g) - 1)))
        sizes.append(s)
        left -= s
    prefixes = [case["prefix"]] + [r.randint(max(1, case["prefix"] // 3), case["prefix"]) for _ in range(n - 1)]
    suffix = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    for b in r.sample(range(case["seqs"]), case["pad"]):
        suffix[b] = -1
    return sizes, prefixes, suffix


# ---- inputs ----------------------------------------------------------------------------------

def _table(rows, ps, gen, spare=3):
    """Block table for sequences of the given lengths over a pool in random order, and the pool's pages."""
    need = [-(-n // ps) for n in rows]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=gen).tolist()
    width = max(1, max(need))
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [0] * (width - n))
        at += n
    return torch.tensor(table, dtype=torch.int32, device=DEV), pool


def _rows(shape, g, spread=True):
    """bf16 rows as projections give them: a scale of its own for each head, some channels larger than others."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    if spread:
        x *= 1.0 + 3.0 * (torch.rand(shape[-1], generator=g, device=DEV) > 0.95)
        x *= 0.5 + torch.rand(shape[-2:-1] + (1,), generator=g, device=DEV)
    return x.to(torch.bfloat16)


def _prepare_cache(case, seed):
    gen = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    Hkv, D, ps, B = case["Hkv"], case["D"], case["ps"], case["seqs"]
    runs = _runs(case)
    T = sum(runs)
    first = [case["start"] + (i * 5) % 11 if case["start"] else 0 for i in range(B)]
    table, pool = _table([f + n for f, n in zip(first, runs)], ps, gen)
    indptr = [0]
    for n in runs:
        indptr.append(indptr[-1] + n)
    s = dict(op=case["op"], T=T, table=table, indptr=torch.tensor(indptr, dtype=torch.int32, device=DEV),
             first=torch.tensor(first, dtype=torch.int32, device=DEV))
    shape = (pool, ps, Hkv, D)
    if case["op"] == "append":
        if case["fused"]:  # [T, query heads, then K and V heads] of one projection
            qkv = _rows((T, 6 * Hkv, D), g)
            s["k"], s["v"] = qkv[:, 4 * Hkv:5 * Hkv], qkv[:, 5 * Hkv:]
        else:
            s["k"], s["v"] = _rows((T, Hkv, D), g), _rows((T, Hkv, D), g)
        for x in "kv":
            s[x + "_codes"] = torch.zeros(shape, dtype=torch.uint8, device=DEV)
            s[x + "_scale"] = torch.ones((pool, Hkv, ps), dtype=torch.bfloat16, device=DEV)
    else:
        for x in "kv":
            codes = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(100.0).clamp_(-E4M3_MAX, E4M3_MAX)
            s[x + "_codes"] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
            s[x + "_scale"] = (torch.rand((pool, Hkv, ps), generator=g, device=DEV) * 0.02 + 0.004).to(torch.bfloat16)
    return s


def _prepare_shared(case, seed):
    gen = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    Hq, Hkv, D, ps, B = case["Hq"], case["Hkv"], case["D"], case["ps"], case["seqs"]
    sizes, prefixes, suffix = _batch(case)
    # whole pages of a group's prefix are shared; the page that a prefix ends in is each sequence's own copy
    whole = [p // ps for p in prefixes]
    group = [i for i, n in enumerate(sizes) for _ in range(n)]
    lens = [0 if n < 0 else prefixes[i] + n for i, n in zip(group, suffix)]
    held = [prefixes[i] + max(n, 0) for i, n in zip(group, suffix)]
    need = [-(-n // ps) - whole[i] for n, i in zip(held, group)]
    pool = sum(whole) + sum(need) + 3
    order = torch.randperm(pool, generator=gen).tolist()
    shared, at = [], 0
    for w in whole:
        shared.append(order[at:at + w])
        at += w
    width = max(whole[i] + n for i, n in zip(group, need)) + 1
    rows = []
    for i, n in zip(group, need):
        rows.append(shared[i] + order[at:at + n])
        rows[-1] += [0] * (width - len(rows[-1]))
        at += n
    table = torch.tensor(rows, dtype=torch.int32, device=DEV)
    k, v = _rows((pool, ps, Hkv, D), g), _rows((pool, ps, Hkv, D), g, spread=False)
    start = 0
    for i, n in enumerate(sizes):  # the copies of the page that the prefix ends in
        part = prefixes[i] - whole[i] * ps
        if part:
            pages = table[start:start + n, whole[i]].long()
            k[pages, :part] = k[pages[0], :part].clone()
            v[pages, :part] = v[pages[0], :part].clone()
        start += n
    q = _rows((B, Hq, D), g, spread=False)
    starts = [sum(sizes[:i]) for i in range(len(sizes))]
    most = max(sizes)
    s = dict(op="shared", q=q, k=k, v=v, table=table, scale=1.0 / math.sqrt(D), sizes=sizes,
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
             prefix=torch.tensor(prefixes, dtype=torch.int32, device=DEV),
             group=torch.tensor(group, device=DEV),
             # the group's sequences side by side, short groups filled with their last one
             member=torch.tensor([[a + min(j, n - 1) for j in range(most)] for a, n in zip(starts, sizes)], device=DEV),
             place=torch.tensor([b - starts[i] for b, i in enumerate(group)], device=DEV),
             max_prefix=max(prefixes), max_suffix=max(1, max(suffix)), total_suffix=sum(n for n in suffix if n > 0))
    if own:
        from paged_kv_cache_298_gb300 import binding
        s["plan"] = binding.SharedPlan(sizes, Hq, Hkv, D, DEV)
        n = binding.workspace_bytes_shared(s["plan"], max_prefix_len=s["max_prefix"], max_suffix_len=s["max_suffix"],
                                           total_suffix=s["total_suffix"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return s


def prepare(case, seed):
    return _prepare_shared(case, seed) if case["op"] == "shared" else _prepare_cache(case, seed)


# ---- plain forms -------------------------------------------------------------------------------

def _places(s):
    """Page and slot of every token of the runs."""
    row = torch.arange(s["T"], device=DEV)
    ends = s["indptr"][1:].contiguous()
    b = torch.searchsorted(ends, row.to(torch.int32), right=True)
    pos = s["first"][b].long() + row - s["indptr"][b].long()
    ps = s["k_codes"].shape[1]
    return s["table"][b, pos // ps].long(), pos % ps


def _append_plain(s):
    page, slot = _places(s)
    for x in "kv":
        rows = s[x].float()
        amax = rows.abs().amax(dim=-1)
        factor = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax)).to(torch.bfloat16)
        codes = (rows / factor.float()[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s[x + "_codes"][page, slot] = codes.view(torch.uint8)
        s[x + "_scale"][page, :, slot] = factor


def _read_plain(s):
    page, slot = _places(s)
    out = []
    for x in "kv":
        codes = s[x + "_codes"][page, slot].view(torch.float8_e4m3fn).float()
        out.append((codes * s[x + "_scale"][page, :, slot].float()[..., None]).to(torch.bfloat16))
    return tuple(out)


def _shared_plain(s):
    q, table, lens, prefix, group = s["q"].float(), s["table"].long(), s["lens"].long(), s["prefix"].long(), s["group"]
    B, Hq, D = q.shape
    ps, Hkv = s["k"].shape[1:3]
    G = Hq // Hkv
    ng, nb = s["member"].shape
    # the prefixes, once for a group
    t = torch.arange(s["max_prefix"], device=DEV)
    page = table[s["member"][:, 0]][:, t // ps]
    kp, vp = (s[x][page, t % ps].float().permute(0, 2, 1, 3) for x in "kv")                    # [group, Hkv, t, D]
    qg = q[s["member"]].view(ng, nb, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(ng, Hkv, nb * G, D)
    sp = (qg @ kp.transpose(2, 3)).view(ng, Hkv, nb, G, -1)[group, :, s["place"]] * s["scale"]  # [B, Hkv, G, t]
    sp = sp.masked_fill((t >= prefix[group][:, None])[:, None, None], -math.inf)
    # what each sequence has behind its prefix
    j = torch.arange(s["max_suffix"], device=DEV)
    pos = prefix[group][:, None] + j
    at = pos.clamp(max=table.shape[1] * ps - 1)
    page = table.gather(1, at // ps)
    ks, vs = (s[x][page, at % ps].float().permute(0, 2, 1, 3) for x in "kv")                   # [B, Hkv, j, D]
    inside = (pos < lens[:, None])[:, None, None]
    ss = (q.view(B, Hkv, G, D) @ ks.transpose(2, 3) * s["scale"]).masked_fill(~inside, -math.inf)
    # one softmax over both
    m = torch.maximum(sp.amax(-1, keepdim=True), ss.amax(-1, keepdim=True))
    wp, ws = (sp - m).exp(), (ss - m).exp()
    total = wp.sum(-1, keepdim=True) + ws.sum(-1, keepdim=True)
    wide = torch.zeros((ng, nb, Hkv, G, wp.shape[-1]), device=DEV)
    wide[group, s["place"]] = wp
    op = (wide.permute(0, 2, 1, 3, 4).reshape(ng, Hkv, nb * G, -1) @ vp).view(ng, Hkv, nb, G, D)[group, :, s["place"]]
    out = (op + ws @ vs) / total
    out = torch.where((lens > 0)[:, None, None, None], out, torch.zeros_like(out))
    return out.reshape(B, Hq, D).to(torch.bfloat16)


def run(s):
    if own:
        from paged_kv_cache_298_gb300 import binding
        if s["op"] == "append":
            binding.kv_append_paged_fp8_multi(s["k"], s["v"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["table"],
                                              s["indptr"], s["first"])
        elif s["op"] == "read":
            return binding.kv_read_paged_fp8(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["table"], s["indptr"],
                                             s["first"], total_tokens=s["T"])
        else:
            return binding.decode_attn_paged_shared(s["q"], s["k"], s["v"], s["table"], s["lens"], s["prefix"], s["plan"],
                                                    max_prefix_len=s["max_prefix"], max_suffix_len=s["max_suffix"],
                                                    total_suffix=s["total_suffix"], scale=s["scale"], workspace=s["workspace"])
    else:
        if s["op"] == "append":
            _append_plain(s)
        elif s["op"] == "read":
            return _read_plain(s)
        else:
            return _shared_plain(s)
    return dict(k=s["k_codes"].view(torch.float8_e4m3fn), v=s["v_codes"].view(torch.float8_e4m3fn), k_scale=s["k_scale"],
                v_scale=s["v_scale"])


# ---- work ----------------------------------------------------------------------------------------

def work(case):
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] != "shared":
        rows = sum(_runs(case)) * Hkv
        return {"bytes": 2 * rows * (3 * D + 2), "flops": (6 if case["op"] == "append" else 2) * rows * D}
    sizes, prefixes, suffix = _batch(case)
    group = [i for i, n in enumerate(sizes) for _ in range(n)]
    keys = sum(prefixes) + sum(n for n in suffix if n > 0)
    seen = sum(prefixes[i] + n for i, n in zip(group, suffix) if n >= 0)
    return {"bytes": 4 * keys * Hkv * D + 4 * case["seqs"] * case["Hq"] * D, "flops": 4 * case["Hq"] * D * seen}


# ---- the definitions in 64 bits --------------------------------------------------------------------

def _run_places(s):
    indptr, first, ps = s["indptr"].tolist(), s["first"].tolist(), s["k_codes"].shape[1]
    page, slot = [], []
    for b, p in enumerate(first):
        pos = torch.arange(p, p + indptr[b + 1] - indptr[b], device=DEV)
        page.append(s["table"][b][pos // ps].long())
        slot.append(pos % ps)
    return torch.cat(page), torch.cat(slot)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        # the quotient that a code stands for, before its rounding to 8 bits, by the stored factor
        page, slot = _run_places(s)
        out = {}
        for x in "kv":
            rows = s[x].double()
            top = rows.abs().max(dim=-1).values / E4M3_MAX
            top = torch.where(top == 0, torch.ones_like(top), top)
            held = top.to(torch.bfloat16).double().unsqueeze(-1)
            codes = s[x + "_codes"].view(torch.float8_e4m3fn).double()
            codes.index_put_((page, slot), torch.clamp(rows / held, -E4M3_MAX, E4M3_MAX))
            scale = s[x + "_scale"].double().transpose(1, 2).contiguous()
            scale.index_put_((page, slot), top)
            out[x], out[x + "_scale"] = codes, scale.transpose(1, 2).contiguous()
        return out
    if case["op"] == "read":
        page, slot = _run_places(s)
        return tuple(s[x + "_codes"].view(torch.float8_e4m3fn).double()[page, slot]
                     * s[x + "_scale"].double().transpose(1, 2)[page, slot].unsqueeze(-1) for x in "kv")
    B, Hq, D = s["q"].shape
    ps, Hkv = s["k"].shape[1:3]
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        if n:
            t = torch.arange(n, device=DEV)
            page = s["table"][b][t // ps].long()
            k, v = (s[x][page, t % ps].double().repeat_interleave(Hq // Hkv, dim=1) for x in "kv")
            w = torch.softmax(torch.einsum("hd,thd->ht", s["q"][b].double(), k) * s["scale"], dim=1)
            out[b] = torch.einsum("ht,thd->hd", w, v)
    return out
