"""The README's Python blocks run as they stand, one after another: the short
decode example, and the loop that evicts, taken through two evictions."""

import os
import re

import pytest
import torch

import paged_kv_cache_247_gb300 as pkv
from paged_kv_cache_247_gb300 import workloads as W
from _gpu_util import assert_within_tol, oracle_decode

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_readme_blocks(lib, cuda_device):
    pkv.device_status(clear=True)
    with open(README) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    assert len(blocks) == 2
    names, gen, rows = {}, torch.Generator(device="cuda").manual_seed(3), []
    exec(blocks[0], names)
    H, D = names["H"], names["D"]

    def project(step):
        q, k, v = (torch.randn((1, n, D), generator=gen, device="cuda").bfloat16()
                   for n in (4 * H, H, H))
        rows.append(v.clone())
        return q, k, v

    evicted = []
    select = pkv.kv_evict_select

    def counted(*args, **kwargs):
        evicted.append(len(rows))
        return select(*args, **kwargs)

    names.update(steps=6200, project=project)
    pkv.kv_evict_select = counted
    try:
        exec(blocks[1], names)
    finally:
        pkv.kv_evict_select = select
    # full at 4,096 positions, and again 2,048 later
    assert len(evicted) == 2 and evicted[1] - evicted[0] == 2048
    held = 2048 + 6200 - 4096 - 2048
    assert names["lens"].tolist() == [held] and names["alloc"].seq_info(1)[0] == held
    assert names["positions"].tolist() == [6200]
    table = torch.from_numpy(names["alloc"].block_table([1], 256)).cuda()
    case = W.DecodeCase(q=names["q"], k_cache=names["k_cache"], v_cache=names["v_cache"],
                        block_tables=table, context_lens=names["lens"], scale=D ** -0.5,
                        block_size=names["B"], max_context_len=4096)
    assert_within_tol(names["out"], oracle_decode(case), torch.bfloat16, "the last step")
    # the first four rows and the newest ones are still there, the oldest others are not all
    at = table[0].long()
    kept = names["v_cache"][at[:-(-held // 16)]].transpose(1, 2).reshape(-1, H, D)[:held]
    assert torch.equal(kept[:4], torch.cat(rows[:4]))
    assert torch.equal(kept[-56 - 256:], torch.cat(rows[-56 - 256:]))
    weights = names["weights"]
    assert (weights[0, :, :held] > 0).all() and (weights[0, :, held:] == 0).all()
    assert pkv.device_status(clear=True) == 0
