"""Every attention call at a scale of zero and below: the formula has no
restriction on it (zero gives every visible key the same weight, a negative
scale prefers the keys that a positive one shuns), and weights that a call
accumulates have to stay numbers.

Outputs are held to the tolerances of the other parity tests, accumulated
weights to the bound derived in tests/test_gpu_evict.py, which holds for any
sign of the logits."""

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_247_gb300 as pkv
from paged_kv_cache_247_gb300 import workloads as W
from _gpu_util import assert_within_tol, oracle_decode, to_f64
from test_gpu_evict import _check_weights, _chunk_case, _old_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status(lib, cuda_device):
    pkv.device_status(clear=True)
    yield
    pkv.set_decode_path(0)
    assert pkv.device_status(clear=True) == 0


SCALES = [0.0, -0.0, -0.125, -1.0]


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype,hq,hkv,D,B,lens,chunks", [
    ("bf16", 8, 2, 128, 16, [700, 130, 1], [300, 130, 1]),    # two row tiles, whole and partial chunks
    ("fp16", 12, 4, 64, 32, [257, 64], [257, 5]),             # a group of 3
    ("fp16", 4, 4, 128, 8, [513], [400]),
])
def test_prefill(cuda_device, dtype, hq, hkv, D, B, lens, chunks, scale):
    case, q, start = _chunk_case(D + B, dtype, hq, hkv, D, B, lens, chunks, cuda_device)
    case.scale = scale
    ref = oracle.paged_prefill_attention(to_f64(q), to_f64(case.k_cache), to_f64(case.v_cache),
                                         case.block_tables.cpu().numpy(),
                                         case.context_lens.cpu().numpy(), start.cpu().numpy(), scale)
    args = (q, start, case.k_cache, case.v_cache, case.block_tables, case.context_lens, scale,
            case.max_context_len, max(chunks))
    out = pkv.paged_attn_prefill(torch.full_like(q, float("nan")), *args)
    assert_within_tol(out, ref, q.dtype, "prefill")
    weights = _old_weights(len(lens), hkv, case.max_context_len, 9)
    old = weights.clone()
    again = pkv.paged_attn_prefill_weights(torch.full_like(q, float("nan")), weights, *args)
    assert torch.equal(again, out)
    _check_weights(weights, old, case, q, chunks, 1.0)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype,hq,hkv,D,part", [
    ("bf16", 8, 2, 128, 0), ("fp16", 4, 4, 64, 128), ("bf16", 34, 2, 64, 0)])
def test_decode(cuda_device, dtype, hq, hkv, D, part, scale):
    lens = [700, 1, 0, 129]
    case = W.make_decode_case(hq, 4, hq, hkv, D, 16, dtype, lens, pool_factor=1.2, poison=True,
                              device=cuda_device)
    case.scale = scale
    ref = oracle_decode(case)
    args = (case.q, case.k_cache, case.v_cache, case.block_tables, case.context_lens, scale, 700)
    for path in (1, 2):
        pkv.set_decode_path(path)
        out = pkv.paged_attn_decode(torch.full_like(case.q, float("nan")), *args, partition_size=part)
        assert_within_tol(out, ref, case.q.dtype, f"decode path {path}")
    weights = _old_weights(4, hkv, 700, 3)
    old = weights.clone()
    out = pkv.paged_attn_decode_weights(torch.full_like(case.q, float("nan")), weights, *args,
                                        partition_size=part)
    assert_within_tol(out, ref, case.q.dtype, "decode with weights")
    _check_weights(weights, old, case, case.q, [1] * 4, 1.0)


def test_zero_scale_keeps_non_finite_queries(cuda_device):
    """Zero times a NaN or an infinity is no number: such a query's row is NaN
    and the others are not."""
    case, q, start = _chunk_case(7, "bf16", 4, 2, 128, 16, [200], [60], cuda_device)
    q[3, 1, 5], q[40, 2, 0] = float("nan"), float("inf")
    out = pkv.paged_attn_prefill(torch.zeros_like(q), q, start, case.k_cache, case.v_cache,
                                 case.block_tables, case.context_lens, 0.0, 200, 60)
    bad = torch.zeros((60, 4), dtype=torch.bool, device=cuda_device)
    bad[3, 1] = bad[40, 2] = True
    assert (torch.isnan(out).any(-1) ^ bad).nonzero().tolist() == []
