"""The run write's quotients over everything that decides them, byte for byte against 64-bit division.

A code depends on the significands of its value and of its row's maximum (7 bits each beside the leading one) and on the
distance of their exponents; the maximum's own exponent only shifts, inside the range where the kernel divides by a reciprocal
and a correction step (maxima of 2^-90 .. 2^90).  So all 128 x 128 pairs of significands at every distance that gives a code
other than zero, and rows on both sides of both ends of the range, are all there is.  The comparison is exact: a quotient that
is no tie between codes lies at least 2^-14 of itself away from one (test_fp8_runs_gpu), further than binary32 rounds."""
import pytest
import torch

from paged_kv_cache_298_gb300 import binding

pytestmark = pytest.mark.gpu

SIG = 1 + torch.arange(128, dtype=torch.float64) / 128


def write(rows):
    """The codes and factors of bf16 rows [T, D], one kv head, pages of 64."""
    T, D = rows.shape
    n = -(-T // 64)
    x = rows.view(T, 1, D).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    codes = [torch.zeros((n, 64, 1, D), dtype=torch.uint8, device="cuda") for _ in "kv"]
    scale = [torch.zeros((n, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    binding.kv_append_paged_fp8_multi(x, x, *codes, *scale, torch.arange(n, **i32).view(1, n), torch.tensor([0, T], **i32),
                                      torch.zeros(1, **i32))
    assert binding.get_device_errors(clear=True) == 0
    assert torch.equal(codes[0], codes[1]) and torch.equal(scale[0].view(torch.int16), scale[1].view(torch.int16))
    return codes[0].view(-1, D)[:T].cpu(), scale[0].view(-1)[:T].cpu()


def check(rows64):
    rows = rows64.to(torch.bfloat16)
    assert torch.equal(rows.double(), rows64)   # (bf16 holds them)
    codes, scale = write(rows)
    amax = rows64.abs().amax(-1)
    s = (amax.float() / 448.0).to(torch.bfloat16)
    assert torch.equal(scale.view(torch.int16), s.view(torch.int16))
    want = (rows64 / s.double()[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    bad = (codes != want).nonzero()
    assert len(bad) == 0, f"{len(bad)} codes, the first at {bad[0].tolist()}: value {float(rows64[tuple(bad[0])])!r}, maximum {float(amax[bad[0, 0]])!r}"


def rows_of(top, D, distance):
    """Rows with each maximum of `top` in front, then values of every significand `distance` powers of two below (both signs in
    turn), as many rows of D as that takes."""
    step = D // 2 if D < 256 else 128
    out = []
    for i in range(0, 128, step):
        v = SIG[i:i + step] * 2.0 ** -distance * 2.0 ** torch.floor(torch.log2(top))[:, None]
        v = torch.where(v > top[:, None], v / 2, v)   # (inside the row's maximum)
        v = v * torch.where((torch.arange(step) + i + distance) % 2 == 0, 1.0, -1.0)
        out.append(torch.cat([top[:, None], v, torch.zeros((len(top), D - 1 - step), dtype=torch.float64)], dim=1))
    return torch.cat(out)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_all_pairs_of_significands(D):
    # codes go down to 2^-9 of a factor, the maximum is about 448 of them: 19 powers of two, and below half of one zero
    check(torch.cat([rows_of(SIG * 8, D, d) for d in range(22)]))


@pytest.mark.parametrize("D", [64, 256])
def test_both_sides_of_the_range_of_the_reciprocal(D):
    tops = []
    for e in (-90, 90):
        at = 2.0 ** e
        tops += [at, at * (1 + 1 / 128), at * (1 + 2 / 128), at * (1 - 1 / 256), at * (1 - 2 / 256), at * 1.75, at * 0.875, at * 2, at / 2]
    check(torch.cat([rows_of(torch.tensor(tops, dtype=torch.float64), D, d) for d in range(0, 22, 3)]))
