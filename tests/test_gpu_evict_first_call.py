"""The first eviction calls of a process made while a graph is captured: what
they ask of the device, or set on it, once per process must not need a stream."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
import paged_kv_cache_247_gb300 as pkv
S, H, n, budget = 1, 2, 40000, 9000
w = torch.rand((S, H, n), device="cuda")
lens = torch.full((S,), n, dtype=torch.int32, device="cuda")
keep = torch.zeros((S, H, budget), dtype=torch.int32, device="cuda")
kc = torch.rand((n // 16, H, 16, 64), device="cuda").half()
vc, was = kc.clone(), kc.clone()
table = torch.arange(n // 16, dtype=torch.int32, device="cuda")[None]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    pkv.kv_evict_select(keep, w, lens, n, recent=7, sinks=3)
    pkv.kv_compact(kc, vc, table, keep, lens)
g.replay()
torch.cuda.synchronize()
rank = w.clone()
rank[..., :3] = rank[..., n - 7:] = 2.0
want = torch.argsort(rank, dim=-1, descending=True, stable=True)[..., :budget].sort(-1).values
assert torch.equal(keep.long(), want)
rows = lambda c: c.transpose(0, 1).reshape(H, n, 64)
moved = torch.stack([rows(was)[h, want[0, h]] for h in range(H)])
assert torch.equal(rows(kc)[:, :budget], moved) and torch.equal(rows(vc)[:, :budget], moved)
assert pkv.device_status() == 0
print("captured")
"""


def test_captured(lib, cuda_device):
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.strip() == "captured"
