"""Every decode call with a partition size far above its contexts, up to the
largest int32 multiple: bit for bit the unsplit call."""

import pytest
import torch

import paged_kv_cache_247_gb300 as pkv
from paged_kv_cache_247_gb300 import workloads as W
from _gpu_util import assert_within_tol, oracle_decode
from test_gpu_evict import _check_weights, _old_weights
from test_partitions import LARGEST

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status(lib, cuda_device):
    pkv.device_status(clear=True)
    yield
    pkv.set_decode_path(0)
    assert pkv.device_status(clear=True) == 0


@pytest.mark.parametrize("part", [LARGEST, LARGEST - 128, 1 << 30])
@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 128), (4, 4, 64)])
def test_unsplit(cuda_device, hq, hkv, D, part):
    lens = [700, 1, 0, 129, 128]
    case = W.make_decode_case(hq, 5, hq, hkv, D, 16, "bf16", lens, pool_factor=1.2, poison=True,
                              device=cuda_device)
    args = (case.q, case.k_cache, case.v_cache, case.block_tables, case.context_lens, case.scale, 700)
    old = _old_weights(5, hkv, 700, 3)
    outs, weights = [], []
    for size in (768, part):
        for path in (1, 2):
            pkv.set_decode_path(path)
            outs.append(pkv.paged_attn_decode(torch.full_like(case.q, float("nan")), *args,
                                              partition_size=size))
        weights.append(old.clone())
        outs.append(pkv.paged_attn_decode_weights(torch.full_like(case.q, float("nan")), weights[-1],
                                                  *args, partition_size=size))
    for a, b in zip(outs[:3], outs[3:]):
        assert torch.equal(a, b)
        assert_within_tol(b, oracle_decode(case), case.q.dtype, "out")
    assert torch.equal(*weights)
    _check_weights(weights[1], old, case, case.q, [1] * 5, 1.0)
    k, v = (torch.randn((5, hkv, 700, D), device="cuda").bfloat16() for _ in range(2))
    a, b = (pkv.contiguous_attn_decode(torch.empty_like(case.q), case.q, k, v, case.context_lens,
                                       case.scale, partition_size=size) for size in (704, part))
    assert torch.equal(a, b)
