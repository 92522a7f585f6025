"""Launches that do not fit the GPU's limits are refused on the host before
anything is enqueued: checked without a GPU, where a call that got past its
checks would report a CUDA error instead."""

import pytest

from test_evict_host import UNSUPPORTED, _prefill


@pytest.mark.parametrize("maxctx,S,heads", [
    (1 << 30, 128, 2),           # 2^23 tiles of 128 positions: 2^31 CTAs
    (1 << 20, 65535, 5),         # 2^13 tiles
])
def test_prefill_weights_grid(lib, maxctx, S, heads):
    got = _prefill(lib, maxctx=maxctx, ws=maxctx, mbps=maxctx // 128, B=128, S=S, Hq=4 * heads,
                   Hkv=heads, T=16, mql=8, wkb=16 * 4 * heads * 4)
    assert got == UNSUPPORTED
