"""Calls that are given their outputs and workspace take no device memory: none from torch's allocator, and, after a device's
first call, none from the driver."""
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
B, Hq, Hkv, D, ps, P, S = 20, 32, 8, 128, 16, 1000, 40
n = -(-(P + S) // ps)
table = torch.arange(n, **i32).repeat(B, 1)
own = torch.arange(B * 4, **i32).view(B, 4) + n
table[:, P // ps:] = own[:, :n - P // ps]
k, v = (torch.randn((n + B * 4, ps, Hkv, D), device="cuda").to(torch.bfloat16) for _ in "kv")
part = P % ps
for x in (k, v):
    x[table[:, P // ps].long(), :part] = x[0, :part].clone()
q = torch.randn((B, Hq, D), device="cuda").to(torch.bfloat16)
lens, prefix = torch.full((B,), P + S, **i32), torch.full((1,), P, **i32)
plan = binding.SharedPlan([B], Hq, Hkv, D, "cuda")
kw = dict(max_prefix_len=P, max_suffix_len=S)
forms = [dict(kw, prefix_splits=a, suffix_splits=b) for a, b in ((0, 0), (5, 1), (16, 2), (3, 1))]
ws = torch.empty(max(binding.workspace_bytes_shared(plan, **f) for f in forms), dtype=torch.uint8, device="cuda")
out = torch.empty_like(q)
T = 300
codes = [torch.zeros((20, ps, Hkv, D), dtype=torch.uint8, device="cuda") for _ in "kv"]
scale = [torch.zeros((20, Hkv, ps), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
rows = [torch.randn((T, Hkv, D), device="cuda").to(torch.bfloat16) for _ in "kv"]
back = [torch.empty_like(r) for r in rows]
run = (torch.arange(20, **i32).view(1, 20), torch.tensor([0, T], **i32), torch.zeros(1, **i32))
def step():
    for f in forms:
        binding.decode_attn_paged_shared(q, k, v, table, lens, prefix, plan, workspace=ws, out=out, **f)
    binding.kv_append_paged_fp8_multi(*rows, *codes, *scale, *run)
    binding.kv_read_paged_fp8(*codes, *scale, *run, k_out=back[0], v_out=back[1])
    torch.cuda.synchronize()
step()
seen = []
for _ in range(3):
    seen.append((torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]))
    step()
seen.append((torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]))
print(json.dumps({"seen": seen, "errors": binding.get_device_errors(), "finite": bool(torch.isfinite(out.float()).all())}))
"""


def test_given_buffers_mean_no_allocation():
    r = subprocess.run([sys.executable, "-c", _FRESH, ROOT], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert res["errors"] == 0 and res["finite"]
    assert all(s == res["seen"][0] for s in res["seen"]), res["seen"]
