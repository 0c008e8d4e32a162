"""Refusals of the e4m3 cache's run write and read-back that need no GPU: the documented status
comes back before CUDA is touched, and the binding refuses tensors it cannot pass."""
import ctypes

import pytest
import torch

from paged_kv_cache_298_gb300 import binding

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p((1 << 20) + 2)
SHAPE, UNSUPPORTED, NULL, ALIGN = 2, 3, 1, 5


def call(write, **kw):
    a = dict(k=FAKE, v=FAKE, kst=1024, ksh=128, vst=1024, vsh=128, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, P=64, ps=16,
             table=FAKE, maxp=8, indptr=FAKE, pos=FAKE, T=20, B=2, Hkv=8, D=128)
    a.update(kw)
    lib = binding.load()
    cache = (a["kc"], a["vc"], a["ks"], a["vs"], a["P"], a["ps"], a["table"], a["maxp"], a["indptr"], a["pos"], a["T"],
             a["B"], a["Hkv"], a["D"])
    strides = (a["kst"], a["ksh"], a["vst"], a["vsh"])
    if write:
        return lib.kv_append_paged_fp8_multi(a["k"], a["v"], *strides, *cache, None)
    return lib.kv_read_paged_fp8(*cache, a["k"], a["v"], *strides, None)


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(B=-1), SHAPE), (dict(B=0), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=0), SHAPE),
    (dict(P=0), SHAPE), (dict(ps=0), SHAPE), (dict(maxp=0), SHAPE), (dict(kst=-8), SHAPE), (dict(vsh=-8), SHAPE),
    (dict(kst=0), SHAPE), (dict(vst=0), SHAPE), (dict(ksh=0), SHAPE), (dict(vsh=0), SHAPE),
    (dict(D=32), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(D=512), UNSUPPORTED),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(kc=None), NULL), (dict(vc=None), NULL), (dict(ks=None), NULL),
    (dict(vs=None), NULL), (dict(table=None), NULL), (dict(indptr=None), NULL), (dict(pos=None), NULL),
    (dict(k=ODD), ALIGN), (dict(v=ODD), ALIGN), (dict(kc=ODD), ALIGN), (dict(vc=ODD), ALIGN),
    (dict(ks=ctypes.c_void_p((1 << 20) + 1)), ALIGN), (dict(table=ODD), ALIGN), (dict(indptr=ODD), ALIGN),
    (dict(pos=ODD), ALIGN), (dict(kst=1028), ALIGN), (dict(ksh=132), ALIGN), (dict(vst=1026), ALIGN),
    (dict(vsh=129), ALIGN),
])
def test_bad_arguments(write, kw, status):
    assert call(write, **kw) == status


@pytest.mark.parametrize("write", [True, False])
def test_no_tokens_is_nothing_to_do(write):
    assert call(write, T=0) == 0
    assert call(write, T=0, B=0) == 0


def test_binding_refuses_cpu_tensors():
    rows = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    codes = torch.zeros((3, 16, 2, 64), dtype=torch.uint8)
    scale = torch.ones((3, 2, 16), dtype=torch.bfloat16)
    table, ind, pos = (torch.zeros(s, dtype=torch.int32) for s in ((1, 2), (2,), (1,)))
    with pytest.raises(binding.DapError):
        binding.kv_append_paged_fp8_multi(rows, rows, codes, codes, scale, scale, table, ind, pos)
    with pytest.raises(binding.DapError):
        binding.kv_read_paged_fp8(codes, codes, scale, scale, table, ind, pos, total_tokens=4)
