"""Windowed and tree attention, commits and resizes that are given their outputs and workspace take no device memory: none from
torch's allocator, and, after a device's first call, none from the driver."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_FRESH = r"""
import json, sys, torch
sys.path.insert(0, sys.argv[1])
from paged_kv_cache_298_gb300 import binding
torch.cuda.set_device(0)
i32 = dict(dtype=torch.int32, device="cuda")
B, Hq, Hkv, D, ps, ctx = 6, 32, 8, 128, 16, 900
forms = []
table = torch.arange(B * 64, **i32).view(B, 64)
k, v = (torch.randn((B * 64, ps, Hkv, D), device="cuda").to(torch.bfloat16) for _ in "kv")
for n in (1, 3, 40, 64):
    plan = binding.SpanPlan([n] * B, Hq, Hkv, D, "cuda")
    q = torch.randn((B * n, Hq, D), device="cuda").to(torch.bfloat16)
    parents = torch.arange(-1, n - 1, **i32).repeat(B)
    lens = torch.full((B,), ctx + n, **i32)
    for S in (0, 3):
        kw = dict(max_kv_len=1000, window=300, sinks=4, num_splits=S)
        ws = [torch.empty(max(1, binding.workspace_bytes_span(plan, tree=t, **kw)), dtype=torch.uint8, device="cuda") for t in (0, 1)]
        forms.append((q, lens, parents, plan, kw, ws, torch.empty_like(q)))
old, new = torch.full((B,), 20, **i32), torch.full((B,), 400, **i32)
pool = (torch.zeros((B, 64), **i32), torch.arange(1000, **i32), torch.full((1,), 900, **i32))
indptr, slots = torch.empty(B + 1, **i32), torch.empty(B * 380, dtype=torch.int64, device="cuda")
empty = torch.empty(0, dtype=torch.int64, device="cuda")
path, count = torch.arange(1, 9, **i32).repeat(B, 1), torch.full((B,), 8, **i32)
base = torch.full((B,), ctx, **i32)
def step():
    for q, lens, parents, plan, kw, ws, out in forms:
        binding.decode_attn_paged_window(q, k, v, table, lens, plan, workspace=ws[0], out=out, **kw)
        binding.decode_attn_paged_tree(q, k, v, table, lens, parents, plan, workspace=ws[1], out=out, **kw)
    binding.kv_commit_paged(k, v, table, base, path, count)
    binding.kv_resize_paged(old, new, *pool, page_size=ps, total_rows=B * 380, indptr=indptr, slots=slots)
    binding.kv_resize_paged(new, old, *pool, page_size=ps, indptr=indptr, slots=empty)
    torch.cuda.synchronize()
step()
seen = []
for _ in range(3):
    seen.append((torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]))
    step()
seen.append((torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]))
print(json.dumps({"seen": seen, "errors": binding.get_device_errors(),
                  "finite": all(bool(torch.isfinite(f[-1].float()).all()) for f in forms)}))
"""


def test_given_buffers_mean_no_allocation():
    r = subprocess.run([sys.executable, "-c", _FRESH, ROOT], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert res["errors"] == 0 and res["finite"]
    assert all(s == res["seen"][0] for s in res["seen"]), res["seen"]
