"""Runs of tokens in the e4m3 GQA cache on the GPU: the quantised write and the read-back, byte for
byte against plain 64-bit arithmetic.

Why the comparison is exact: the factor is a binary32 quotient rounded to bf16.  A code is the
quotient of two bf16 values rounded to 4 significant bits (or to a multiple of 2^-9): the border
between two codes has 5 significant bits, its product with the factor at most 13, so a quotient
that is no tie lies at least 2^-14 of itself away from the border and its rounding to binary32 on
the way changes nothing; a tie is a quotient that binary32 holds exactly.  Read back, code times factor
has 12 significant bits, exact in binary32, and is rounded once."""
import numpy as np
import pytest
import torch

from paged_kv_cache_298_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    binding.get_device_errors(clear=True)
    yield


def make(lens, starts, Hkv, D, ps, seed, spare=3):
    """Rows, empty caches and the runs' tensors, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    need = [-(-(s + n) // ps) for s, n in zip(starts, lens)]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=g).tolist()
    table = torch.full((len(lens), max(1, max(need, default=1))), -7, dtype=torch.int32)   # unused entries: outside the pool
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    k = torch.randn((T, Hkv, D), generator=g) * torch.logspace(-4, 4, max(T, 1))[:T, None, None]
    v = torch.randn((T, Hkv, D), generator=g)
    if T:
        v[0] = 0                                       # an all-zero row: factor 1
        v[T // 2] = torch.round(v[T // 2] * 4) * 112   # quotients on the borders between codes
    indptr = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    codes = [torch.randint(0, 255, (pool, ps, Hkv, D), generator=g, dtype=torch.uint8) for _ in "kv"]
    scale = [(torch.rand((pool, Hkv, ps), generator=g) + 0.01).to(torch.bfloat16) for _ in "kv"]
    return k.to(torch.bfloat16), v.to(torch.bfloat16), codes, scale, table, indptr, torch.tensor(starts, dtype=torch.int32)


def plain_places(table, indptr, pos, ps):
    for b in range(table.shape[0]):
        for i in range(int(indptr[b + 1]) - int(indptr[b])):
            p = int(pos[b]) + i
            yield int(indptr[b]) + i, int(table[b, p // ps]), p % ps


def plain_write(rows, codes, scale, table, indptr, pos):
    codes, scale = codes.clone(), scale.clone()
    ps = codes.shape[1]
    x = rows.double()
    amax = rows.float().abs().amax(-1)
    s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax)).to(torch.bfloat16)
    c = (x / s.double()[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for r, page, slot in plain_places(table, indptr, pos, ps):
        codes[page, slot] = c[r]
        scale[page, :, slot] = s[r]
    return codes, scale


def on(*ts):
    return [t.cuda() for t in ts]


def write(k, v, codes, scale, table, indptr, pos):
    dk, dv, kc, vc, ks, vs, t, i, p = on(k, v, *codes, *scale, table, indptr, pos)
    binding.kv_append_paged_fp8_multi(dk, dv, kc, vc, ks, vs, t, i, p)
    return kc.cpu(), vc.cpu(), ks.cpu(), vs.cpu()


def same(a, b):
    if a.dtype == torch.bfloat16:
        a, b = a.contiguous().view(torch.int16), b.contiguous().view(torch.int16)
    return torch.equal(a, b)


RUNS = [
    # lens, starts, Hkv, D, page size
    ([1], [0], 1, 128, 16),
    ([1], [4095], 8, 64, 64),                        # one token far in its sequence
    ([3, 0, 5, 1], [0, 7, 15, 31], 2, 64, 16),       # an empty run
    ([0, 0, 40], [3, 3, 3], 8, 128, 8),              # empty runs first
    ([17, 130, 64], [5, 0, 60], 3, 128, 12),         # odd heads, pages of 12
    ([33, 1, 100], [0, 999, 63], 4, 256, 64),
    ([50, 3], [2, 90], 8, 256, 1),                   # pages of one slot
    ([700], [10], 8, 128, 16),
    ([2] * 70, list(range(70)), 2, 128, 5),          # more runs than a warp probes at once
    ([1] * 1100, [0] * 1100, 1, 64, 16),             # three rounds of the search
    ([257, 511], [0, 1], 5, 64, 100),
]


@pytest.mark.parametrize("lens,starts,Hkv,D,ps", RUNS, ids=[f"n{sum(r[0])}_B{len(r[0])}_H{r[2]}_D{r[3]}_ps{r[4]}" for r in RUNS])
def test_write_and_read_back_are_exact(lens, starts, Hkv, D, ps):
    k, v, codes, scale, table, indptr, pos = make(lens, starts, Hkv, D, ps, 900 + D + ps)
    got = write(k, v, codes, scale, table, indptr, pos)
    kc, ks = plain_write(k, codes[0], scale[0], table, indptr, pos)
    vc, vs = plain_write(v, codes[1], scale[1], table, indptr, pos)
    for a, b, what in zip(got, (kc, vc, ks, vs), ("k codes", "v codes", "k factors", "v factors")):
        assert same(a, b), what
    ko, vo = binding.kv_read_paged_fp8(*on(kc, vc, ks, vs, table, indptr, pos), total_tokens=sum(lens))
    for out, c, s, rows in ((ko, kc, ks, k), (vo, vc, vs, v)):
        want = torch.empty_like(rows)
        for r, page, slot in plain_places(table, indptr, pos, ps):
            want[r] = (c[page, slot].view(torch.float8_e4m3fn).double() * s[page, :, slot].double()[:, None]).to(torch.bfloat16)
        assert same(out.cpu(), want)
        # a value is off by half a code's step (2^-4 of itself, or 2^-10 factors below the normal codes), one bf16
        # rounding (2^-8), and what saturation cuts where bf16 rounded the factor down (2^-8, in the top step)
        x, y = rows.double(), out.cpu().double()
        step = rows.float().abs().amax(-1, keepdim=True).double() / 448 * 2.0 ** -10 * 1.01
        assert bool(((y - x).abs() <= x.abs() * (2.0 ** -4 + 2.0 ** -7) + step).all())
    assert binding.get_device_errors() == 0


def test_every_code_and_extreme_factors_read_back():
    table, indptr, pos = torch.tensor([[0]], dtype=torch.int32), torch.tensor([0, 8], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    codes = torch.arange(256, dtype=torch.uint8).repeat(8).view(1, 8, 1, 256)
    scale = torch.tensor([1.0, 0.0037, 3e38, 1e-38, 1e-40, float("inf"), float("nan"), -2.5]).to(torch.bfloat16).view(1, 1, 8)
    ko, vo = binding.kv_read_paged_fp8(*on(codes, codes, scale, scale, table, indptr, pos), total_tokens=8)
    c = codes.view(torch.float8_e4m3fn).double()[0]
    want = (c * scale.double().view(8, 1, 1)).to(torch.float32).to(torch.bfloat16)
    for o in (ko.cpu(), vo.cpu()):
        assert torch.equal(o.isnan(), want.isnan())
        assert torch.equal(torch.nan_to_num(o.float(), 0, 1e39, -1e39), torch.nan_to_num(want.float(), 0, 1e39, -1e39))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_write_equals_the_single_token_append_on_extreme_rows(D):
    """Zeros, subnormal, tiny, huge, infinite and NaN rows: the same bytes as kv_append_paged_fp8."""
    g = torch.Generator().manual_seed(D)
    x = torch.randn((12, 2, D), generator=g)
    mags = torch.tensor([0.0, 1e-40, 3e-39, 1e-37, 1e-36, 1e-20, 448.0, 1e30, 3e38, 1.0, 1.0, 1e-38])
    x = (x * mags[:, None, None]).clamp(-3.3e38, 3.3e38)
    x[9, 0, 3], x[9, 1, 5] = float("inf"), float("-inf")
    x[10, 0, 0], x[10, 1, D - 1] = float("nan"), float("nan")
    x = x.to(torch.bfloat16).cuda()
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(12, 1)
    one = [torch.zeros((12, 1, 2, D), dtype=torch.uint8, device="cuda") for _ in "kv"] + \
          [torch.zeros((12, 2, 1), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    many = [t.clone() for t in one]
    zero = torch.zeros(12, dtype=torch.int32, device="cuda")
    binding.kv_append_paged_fp8(x, x, *one, table, zero)
    binding.kv_append_paged_fp8_multi(x, x, *many, table, torch.arange(13, dtype=torch.int32, device="cuda"), zero)
    for a, b in zip(one, many):
        assert same(a, b)


def test_strided_rows_of_a_fused_projection():
    """K and V as slices of one [T, heads, D] tensor, read back into slices of another; what lies between stays."""
    T, Hkv, D, ps = 37, 2, 128, 16
    k, v, codes, scale, table, indptr, pos = make([20, 17], [3, 0], Hkv, D, ps, 41)
    fused = torch.full((T, 6, D), 5.0, dtype=torch.bfloat16)
    fused[:, 2:4], fused[:, 4:] = k, v
    want = write(k, v, codes, scale, table, indptr, pos)
    f = fused.cuda()
    dev = on(*codes, *scale, table, indptr, pos)
    binding.kv_append_paged_fp8_multi(f[:, 2:4], f[:, 4:], *dev)
    for a, b in zip(dev[:4], want):
        assert same(a.cpu(), b)
    ko, vo = binding.kv_read_paged_fp8(*dev, total_tokens=T)
    out = torch.full((T, 6, D), 5.0, dtype=torch.bfloat16, device="cuda")
    r = binding.kv_read_paged_fp8(*dev, k_out=out[:, 2:4], v_out=out[:, 4:])
    assert r[0].data_ptr() == out[:, 2:4].data_ptr()
    assert torch.equal(out[:, 2:4], ko) and torch.equal(out[:, 4:], vo) and bool((out[:, :2] == 5).all())
    # head-major rows: [Hkv, T, D] seen as [T, Hkv, D]
    hm = k.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    again = on(*codes, *scale, table, indptr, pos)
    binding.kv_append_paged_fp8_multi(hm, v.cuda(), *again)
    for a, b in zip(again[:4], want):
        assert same(a.cpu(), b)


def test_rows_outside_every_run_are_left():
    """indptr starts past 0 and ends before total_tokens (a call sized for more tokens than it gets)."""
    Hkv, D, ps = 2, 64, 8
    k, v, codes, scale, table, _, pos = make([10, 20], [0, 4], Hkv, D, ps, 42)
    indptr = torch.tensor([4, 9, 21], dtype=torch.int32)
    got = write(k, v, codes, scale, table, indptr, pos)
    kc, ks = plain_write(k, codes[0], scale[0], table, indptr, pos)
    assert same(got[0], kc) and same(got[2], ks)
    out = torch.full((30, Hkv, D), -3.0, dtype=torch.bfloat16, device="cuda")
    binding.kv_read_paged_fp8(*on(*got, table, indptr, pos), k_out=out, v_out=out.clone())
    assert bool((out[:4] == -3).all()) and bool((out[21:] == -3).all()) and not bool((out[4:21] == -3).all(-1).any())
    none = torch.zeros(3, dtype=torch.int32)
    for a, b in zip(write(k, v, codes, scale, table, none, pos), (*codes, *scale)):
        assert same(a, b)
    assert binding.get_device_errors() == 0


def test_bad_pages_and_positions_are_flagged():
    Hkv, D, ps = 2, 128, 4
    k, v, codes, scale, table, indptr, pos = make([6, 6, 6], [0, 0, 0], Hkv, D, ps, 43)
    pool = codes[0].shape[0]
    table[0, 1] = pool          # rows 4, 5
    table[1, 0] = -1            # rows 6 .. 9
    pos[2] = -2                 # rows 12, 13 in front of the sequence
    good = [0, 1, 2, 3, 10, 11, 14, 15, 16, 17]
    kc, ks = codes[0].clone(), scale[0].clone()
    got = write(k, v, codes, scale, table, indptr, pos)
    flags = binding.get_device_errors()
    assert flags & binding.DEVERR_PAGE and flags & binding.DEVERR_SEQLEN
    places = {0: (0, 0), 1: (0, 1), 2: (0, 2), 3: (0, 3), 10: (1, 4), 11: (1, 5), 14: (2, 0), 15: (2, 1), 16: (2, 2), 17: (2, 3)}
    amax = k.float().abs().amax(-1)
    s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax)).to(torch.bfloat16)
    c = (k.double() / s.double()[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for r in good:
        b, p = places[r]
        page = int(table[b, p // ps])
        kc[page, p % ps], ks[page, :, p % ps] = c[r], s[r]
    assert same(got[0], kc) and same(got[2], ks)
    ko, _ = binding.kv_read_paged_fp8(*on(*got, table, indptr, pos), total_tokens=18)
    ko = ko.cpu()
    bad = [r for r in range(18) if r not in good]
    assert bool((ko[bad] == 0).all()) and not bool((ko[good] == 0).all(-1).any())
    flags = binding.get_device_errors()
    assert flags & binding.DEVERR_PAGE and flags & binding.DEVERR_SEQLEN
    # past the table's end
    pos[2] = table.shape[1] * ps - 1
    write(k, v, codes, scale, table, indptr, pos)
    assert binding.get_device_errors() & binding.DEVERR_SEQLEN


def test_offsets_past_32_bits():
    """A pool of more than 2^32 codes: the run lies in its last pages."""
    Hkv, D, ps, pool = 8, 256, 64, 33000
    kc = torch.empty((pool, ps, Hkv, D), dtype=torch.uint8, device="cuda")
    vc = torch.empty_like(kc)
    ks = torch.empty((pool, Hkv, ps), dtype=torch.bfloat16, device="cuda")
    vs = torch.empty_like(ks)
    table = torch.tensor([[pool - 1, pool - 2]], dtype=torch.int32, device="cuda")
    indptr, pos = torch.tensor([0, 100], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.randn((100, Hkv, D), device="cuda").to(torch.bfloat16)
    kc[:2], kc[-2:] = 1, 2
    binding.kv_append_paged_fp8_multi(x, x, kc, vc, ks, vs, table, indptr, pos)
    ko, vo = binding.kv_read_paged_fp8(kc, vc, ks, vs, table, indptr, pos, total_tokens=100)
    assert bool((kc[:2] == 1).all()) and bool((kc[-2, 36:] == 2).all())
    assert float((ko.float() - x.float()).norm() / x.float().norm()) < 2.0 ** -4 and torch.equal(ko, vo)
    assert binding.get_device_errors() == 0


def test_graph_replay_with_new_rows_and_runs():
    """A captured write and read-back replayed with other rows, boundaries and positions, on another stream than the
    default one."""
    Hkv, D, ps = 4, 128, 16
    k, v, codes, scale, table, indptr, pos = make([30, 30, 30], [0, 16, 33], Hkv, D, ps, 44)
    dk, dv, kc, vc, ks, vs, t, i, p = on(k, v, *codes, *scale, table, indptr, pos)
    ko, vo = torch.zeros_like(dk), torch.zeros_like(dv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        binding.kv_append_paged_fp8_multi(dk, dv, kc, vc, ks, vs, t, i, p)
        binding.kv_read_paged_fp8(kc, vc, ks, vs, t, i, p, k_out=ko, v_out=vo)

    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    k2, v2, _, _, _, _, _ = make([30, 30, 30], [0, 16, 33], Hkv, D, ps, 45)
    indptr2, pos2 = torch.tensor([0, 25, 28, 60], dtype=torch.int32), torch.tensor([2, 20, 10], dtype=torch.int32)
    dk.copy_(k2), dv.copy_(v2), i.copy_(indptr2), p.copy_(pos2)
    for a, b in zip((kc, vc, ks, vs), (*codes, *scale)):
        a.copy_(b)
    before = ko[60:].clone()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    want, ws = plain_write(k2, codes[0], scale[0], table, indptr2, pos2)
    assert same(kc.cpu(), want) and same(ks.cpu(), ws)
    direct, _ = binding.kv_read_paged_fp8(kc, vc, ks, vs, t, i, p, total_tokens=90)
    assert torch.equal(ko[:60], direct[:60]) and torch.equal(ko[60:], before)


def test_binding_refuses():
    k, v, codes, scale, table, indptr, pos = make([10, 20], [0, 4], 2, 64, 8, 48)
    good = on(k, v, *codes, *scale, table, indptr, pos)
    for i, bad in ((0, good[0].float()), (0, good[0][:-1]), (1, good[1][..., :32]), (2, good[2].float()), (3, good[3][:-1]),
                   (4, good[4].float()), (5, good[5][:, :1]), (6, good[6].long()), (6, good[6][:1]), (7, good[7][:2]),
                   (8, good[8].long())):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            binding.kv_append_paged_fp8_multi(*args)
        if i >= 2:
            with pytest.raises(ValueError):
                binding.kv_read_paged_fp8(*args[2:], total_tokens=30)
    for i in range(9):
        args = list(good)
        args[i] = args[i].cpu()
        with pytest.raises(binding.DapError):
            binding.kv_append_paged_fp8_multi(*args)
    with pytest.raises(ValueError):
        binding.kv_read_paged_fp8(*good[2:])
    with pytest.raises(ValueError):
        binding.kv_read_paged_fp8(*good[2:], total_tokens=-1)
    with pytest.raises(ValueError):
        binding.kv_read_paged_fp8(*good[2:], total_tokens=30, k_out=good[0][:-1])
    # more rows than 32 bits count, refused before anything else happens
    many = good[0][:1].expand(2 ** 31, 2, 64)
    for call in (lambda: binding.kv_append_paged_fp8_multi(many, many, *good[2:]),
                 lambda: binding.kv_read_paged_fp8(*good[2:], k_out=many, v_out=many),
                 lambda: binding.kv_read_paged_fp8(*good[2:], total_tokens=2 ** 31)):
        with pytest.raises(ValueError):
            call()
    # rows whose strides break the 16-byte rule
    odd = torch.zeros((30, 2, 68), dtype=torch.bfloat16, device="cuda")[..., :64]
    with pytest.raises(binding.DapError) as e:
        binding.kv_append_paged_fp8_multi(odd, odd, *good[2:])
    assert e.value.status == 5
    assert binding.get_device_errors() == 0


def test_two_streams_at_once():
    cases = [make([200, 300], [0, 5], 8, 128, 16, 46 + j) for j in range(2)]
    dev = [on(c[0], c[1], *c[2], *c[3], *c[4:]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for d, st in zip(dev, streams):
            binding.kv_append_paged_fp8_multi(*d, stream=st)
    torch.cuda.synchronize()
    for c, d in zip(cases, dev):
        want, ws = plain_write(c[0], c[2][0], c[3][0], *c[4:])
        assert same(d[2].cpu(), want) and same(d[4].cpu(), ws)


def test_prompts_then_decode_equals_token_by_token():
    """Decoding over a cache filled by one run write gives the bits that a cache filled token by token gives."""
    lens = [70, 33, 129]
    k, v, codes, scale, table, indptr, pos = make(lens, [0, 0, 0], 2, 128, 16, 47)
    a = on(*codes, *scale)
    b = [t.clone() for t in a]
    dk, dv, t, i, p = on(k, v, table.clamp(min=0), indptr, pos)
    binding.kv_append_paged_fp8_multi(dk, dv, *a, t, i, p)
    for n in range(max(lens)):
        live = [j for j, m in enumerate(lens) if n < m]
        rows = torch.tensor([int(indptr[j]) + n for j in live], device="cuda")
        binding.kv_append_paged_fp8(dk[rows].contiguous(), dv[rows].contiguous(), *b, t[live].contiguous(),
                                    torch.full((len(live),), n, dtype=torch.int32, device="cuda"))
    for x, y in zip(a, b):
        assert same(x, y)
    q = torch.randn((3, 8, 128), device="cuda").to(torch.bfloat16)
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    outs = [binding.decode_attn_paged_fp8kv(q, *c, t, L, max_kv_len=129, num_splits=2) for c in (a, b)]
    assert torch.equal(*outs)
