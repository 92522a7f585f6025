"""The eviction calls on batches that hold nothing yet: a bound of zero
positions, and prompt rows that are all padding.  The plain calls take them."""

import pytest
import torch

import paged_kv_cache_247_gb300 as pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status(lib, cuda_device):
    pkv.device_status(clear=True)
    yield
    assert pkv.device_status(clear=True) == 0


def _empty(cuda_device, queries):
    q = torch.ones((queries, 8, 64), dtype=torch.float16, device=cuda_device)
    cache = torch.ones((4, 2, 16, 64), dtype=torch.float16, device=cuda_device)
    table = torch.zeros((3, 1), dtype=torch.int32, device=cuda_device)
    lens = torch.zeros(3, dtype=torch.int32, device=cuda_device)
    return q, cache, table, lens, torch.empty((3, 2, 0), device=cuda_device)


def test_decode_weights(cuda_device):
    q, cache, table, lens, weights = _empty(cuda_device, 3)
    plain = pkv.paged_attn_decode(torch.full_like(q, 7.0), q, cache, cache, table, lens, 0.1, 0)
    out = pkv.paged_attn_decode_weights(torch.full_like(q, 7.0), weights, q, cache, cache, table,
                                        lens, 0.1, 0)
    assert (plain == 0).all() and torch.equal(out, plain)


@pytest.mark.parametrize("width", [0, 5])
def test_prefill_weights(cuda_device, width):
    q, cache, table, lens, _ = _empty(cuda_device, 4)        # four rows behind the last sequence
    start = torch.zeros(4, dtype=torch.int32, device=cuda_device)
    weights = torch.full((3, 2, width), 2.0, device=cuda_device)
    out = torch.full_like(q, 7.0)
    pkv.paged_attn_prefill(out, q, start, cache, cache, table, lens, 0.1, 0, 1)
    pkv.paged_attn_prefill_weights(out, weights, q, start, cache, cache, table, lens, 0.1, 0, 1)
    assert (out == 7.0).all() and (weights == 2.0).all()


def test_select(cuda_device):
    _, _, _, lens, weights = _empty(cuda_device, 1)
    new = torch.full((3,), 5, dtype=torch.int32, device=cuda_device)
    keep = pkv.kv_evict_select(torch.zeros((3, 2, 9), dtype=torch.int32, device=cuda_device), weights,
                               lens, 0, recent=2, sinks=1, new_lens=new)
    assert (keep == -1).all() and (new == 0).all()


def test_compact(cuda_device):
    _, cache, table, lens, weights = _empty(cuda_device, 1)
    keep = torch.full((3, 2, 9), -1, dtype=torch.int32, device=cuda_device)
    pkv.kv_compact(cache, cache.clone(), table, keep, lens, weights=weights)
    assert (cache == 1).all()
