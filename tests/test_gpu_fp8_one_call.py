"""A call over an 8-bit cache that splits its contexts and is given no workspace goes into the
library once, and gives what it gives with one."""

import numpy as np
import pytest
import torch

import paged_kv_cache_247_gb300 as pkv
from test_gpu_fp8 import Case, _clean_status, _random_masks  # noqa: F401 (an autouse fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("drafts", [None, [5, 3]])
def test_one_call_into_the_library(cuda_device, lib, monkeypatch, drafts):
    masks = None if drafts is None else _random_masks(np.random.default_rng(1), drafts)
    c = Case(3, "bf16", 8, 2, 128, 16, [900, 300], drafts, masks)
    size = pkv.tree_fp8_workspace_size(c.q.shape[0], 5 if drafts else 1, 2, 8, 2, 128, 900, 128)
    want = c.run(partition_size=128, workspace=torch.empty(size, dtype=torch.uint8, device="cuda"))
    name = "pkv_paged_attn_tree_fp8" if drafts else "pkv_paged_attn_decode_fp8"
    inner, calls = getattr(lib, name), []

    def counted(*args):
        calls.append(inner(*args))
        return calls[-1]

    monkeypatch.setattr(lib, name, counted)
    for part in (128, 128, 1024):
        got = c.run(partition_size=part)
        assert torch.equal(got, want) or part == 1024
    assert calls == [0, 0, 0]
