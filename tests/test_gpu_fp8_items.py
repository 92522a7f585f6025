"""Attention over a cache held in 8 bits where a CTA goes through many work items,
where their number passes the launch's CTAs, and where the running references move
in every tile.  Cases, reference and tolerance are those of test_gpu_fp8."""

import numpy as np
import pytest
import torch

import paged_kv_cache_247_gb300 as pkv
from paged_kv_cache_247_gb300 import workloads as W
from test_gpu_fp8 import Case, _clean_status, _random_masks  # noqa: F401 (an autouse fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("hq,hkv,D,most", [
    (8, 8, 64, 4),      # 4 rows
    (24, 12, 128, 4),   # 8 rows
    (32, 16, 64, 8),    # 16 rows
    (24, 8, 128, 9),    # 27 rows, of a sequence with few drafts fewer than 17
    (40, 8, 128, 11),   # 55 rows: some of the warpgroups without a row
    (20, 4, 64, 25),    # 125 rows: two chunks, the second of any size
])
def test_trees_with_many_items(cuda_device, dtype, hq, hkv, D, most):
    rng = np.random.default_rng(hq + D + most)
    lens = [int(n) for n in rng.integers(0, 420, 44)]
    drafts = [min(n, int(rng.integers(0, most + 1))) for n in lens]
    drafts[5] = min(lens[5], most)
    c = Case(hq + D, dtype, hq, hkv, D, 16, lens, drafts, _random_masks(rng, drafts))
    whole = c.check(max_query_len=most)
    c.check(max_query_len=most, partition_size=128)
    assert torch.equal(whole, c.run(max_query_len=most))


def test_more_items_than_ctas(cuda_device):
    """A bound far above the contexts, cut into small partitions: most items are
    empty, and a CTA stands for several."""
    rng = np.random.default_rng(7)
    lens = [int(n) for n in rng.integers(0, 500, 40)]
    c = Case(21, "bf16", 16, 8, 64, 16, lens)
    wide = torch.full((40, 2048), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.t_tables.shape[1]] = c.t_tables
    c.t_tables = wide
    c.check(max_context_len=32768, partition_size=128)  # 81,920 items


@pytest.mark.parametrize("dtype,hq,hkv,D,drafts", [
    ("bf16", 4, 4, 128, None), ("fp16", 16, 1, 64, None), ("bf16", 24, 1, 128, None),
    ("fp16", 40, 1, 128, None), ("bf16", 16, 4, 64, [16, 3])])
@pytest.mark.parametrize("down", [False, True])
def test_references_that_move(cuda_device, dtype, hq, hkv, D, drafts, down):
    """Keys that grow along the context, so that the largest logit of every tile
    passes the ones before by far (or, turned round, none does)."""
    lens = [1500, 700]
    masks = None if drafts is None else _random_masks(np.random.default_rng(2), drafts)
    c = Case(31 + D, dtype, hq, hkv, D, 16, lens, drafts, masks)
    at = torch.cat([torch.arange(n, device="cuda") for n in lens]).float() / 1500
    at = 1 - at if down else at
    k = torch.cat([torch.ones((n, hkv, D), device="cuda") for n in lens]) * (0.1 + 12 * at)[:, None, None]
    k += 0.05 * c.k.float()
    q = c.q.float()
    q = q.abs() * 1.5 / D ** 0.5 * 4  # every query along the keys: logits up to about 100
    c.q = q.to(c.dt)
    pkv.kv_append_fp8(k.to(W.DTYPES[dtype]), c.v, *c.caches, c.slots)
    c.check()
    c.check(partition_size=256)
