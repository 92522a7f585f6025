"""Rows at the upper end of their type in a cache held in 8 bits: what is documented of the
elements that round above it."""

import pytest
import torch

import paged_kv_cache_247_gb300 as pkv
from paged_kv_cache_247_gb300 import workloads as W
from test_gpu_fp8 import _clean_status, _empty_cache  # noqa: F401 (an autouse fixture)

pytestmark = pytest.mark.gpu

# dtype, the largest element that keeps within the type, the next of the type, what that is held as.
# The next one lies half way between the codes' 1.875 and 2 times a power of two, whose last bits are
# 1 and 0: the tie goes up.
ENDS = [("fp16", 63456.0, 63488.0, 2.0 ** 16), ("bf16", 1.9296875 * 2.0 ** 127, 1.9375 * 2.0 ** 127, 2.0 ** 128)]


@pytest.mark.parametrize("dtype,last,over,held", ENDS)
def test_read_back_and_appended_again(cuda_device, dtype, last, over, held):
    dt = W.DTYPES[dtype]
    x = torch.zeros((4, 1, 64), dtype=torch.float64, device="cuda")
    x[0, 0, :3] = torch.tensor([last, -last, 3.0])
    x[1, 0, :3] = torch.tensor([over, last, 3.0])
    x[2, 0, 5] = -over
    x[3] = torch.finfo(dt).max
    x = x.to(dt)
    assert torch.isfinite(x).all()
    caches = _empty_cache(2, 1, 8, 64)
    pkv.kv_append_fp8(x, x, *caches, torch.arange(4, device="cuda"))
    value = caches[0][0, 0, :4].double() * caches[2][0, 0, :4].double()
    even = 61440.0 if dtype == "fp16" else 1.875 * 2.0 ** 127
    assert value[0, 0] == even and value[0, 1] == -even
    assert value[1, 0] == held and value[1, 1] == even and value[2, 5] == -held and (value[3] == held).all()
    out = torch.zeros((2, 1, 8, 64), dtype=dt, device="cuda")
    again = out.clone()
    pkv.block_read_fp8(out, again, *caches, torch.tensor([[0, 0]], device="cuda"))
    rows = out[0, 0, :4]
    want = torch.where(value.abs() == held, torch.copysign(torch.full_like(value, float("inf")), value), value)
    assert torch.equal(rows.double(), want)
    twice = _empty_cache(2, 1, 8, 64)
    pkv.kv_append_fp8(rows[:, None], rows[:, None], *twice, torch.arange(4, device="cuda"))
    assert torch.equal(twice[0].view(torch.uint8)[0, 0, 0], caches[0].view(torch.uint8)[0, 0, 0])
    assert torch.equal(twice[2][0, 0, 0], caches[2][0, 0, 0])
    assert torch.isnan(twice[2][0, 0, 1:4]).all()


@pytest.mark.parametrize("dtype,last,over,held", ENDS)
def test_an_output_that_comes_to_it(cuda_device, dtype, last, over, held):
    """One position: the output is its V row, infinity where that is held above the type."""
    dt = W.DTYPES[dtype]
    k = torch.ones((2, 1, 64), dtype=dt, device="cuda")
    v = torch.full((2, 1, 64), last, dtype=torch.float64, device="cuda")
    v[1] = over
    v = v.to(dt)
    caches = _empty_cache(2, 1, 8, 64)
    pkv.kv_append_fp8(k, v, *caches, torch.tensor([0, 8], device="cuda"))
    q = torch.ones((2, 2, 64), dtype=dt, device="cuda")
    out = pkv.paged_attn_decode_fp8(torch.empty_like(q), q, *caches, torch.tensor([[0], [1]], dtype=torch.int32, device="cuda"),
                                    torch.ones(2, dtype=torch.int32, device="cuda"), 0.125, 1)
    even = 61440.0 if dtype == "fp16" else 1.875 * 2.0 ** 127
    assert (out[0].double() == even).all() and torch.isinf(out[1]).all()
