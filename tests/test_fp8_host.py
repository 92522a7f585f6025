"""The calls of a cache held in 8 bits on a machine without a GPU: refusals on
the host, before anything is enqueued, and the workspace sizes."""

import ctypes
import math

import pytest
import torch

import paged_kv_cache_247_gb300 as pkv

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
NONE = ctypes.c_size_t(-1).value


def _append(lib, **over):
    a = dict(k=16, ks=256, v=16, vs=256, kc=16, vc=16, ksc=16, vsc=16, slot=16, T=3, Hkv=2, D=128,
             B=16, NB=4, dtype=1)
    a.update(over)
    return lib.pkv_kv_append_fp8(a["k"], a["ks"], a["v"], a["vs"], a["kc"], a["vc"], a["ksc"],
                                 a["vsc"], a["slot"], a["T"], a["Hkv"], a["D"], a["B"], a["NB"],
                                 a["dtype"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(T=0, k=None), 0),
    (dict(T=-1), INVALID), (dict(Hkv=0), INVALID), (dict(NB=0), INVALID), (dict(dtype=2), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(B=24), UNSUPPORTED),
    (dict(ks=255), INVALID), (dict(ks=248), INVALID), (dict(vs=260), INVALID),
    (dict(k=8), INVALID), (dict(vc=24), INVALID), (dict(ksc=8), INVALID), (dict(slot=20), INVALID),
    (dict(v=None), INVALID), (dict(vsc=None), INVALID), (dict(slot=None), INVALID),
    (dict(T=1 << 27, Hkv=2), UNSUPPORTED),            # 2^31 parts of 16 elements
])
def test_append_refusals(lib, over, expect):
    assert _append(lib, **over) == expect


def _read(lib, **over):
    a = dict(ko=16, vo=16, NO=3, kc=16, vc=16, ksc=16, vsc=16, pairs=16, P=2, Hkv=2, D=64, B=16,
             NB=4, dtype=0)
    a.update(over)
    return lib.pkv_block_read_fp8(a["ko"], a["vo"], a["NO"], a["kc"], a["vc"], a["ksc"], a["vsc"],
                                  a["pairs"], a["P"], a["Hkv"], a["D"], a["B"], a["NB"],
                                  a["dtype"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(P=0, pairs=None), 0),
    (dict(P=-1), INVALID), (dict(NO=0), INVALID), (dict(NB=0), INVALID), (dict(dtype=-1), INVALID),
    (dict(D=32), UNSUPPORTED), (dict(B=4), UNSUPPORTED),
    (dict(ko=8), INVALID), (dict(pairs=20), INVALID), (dict(vsc=2), INVALID), (dict(vo=None), INVALID),
    (dict(P=1 << 24, Hkv=2), UNSUPPORTED),
])
def test_read_refusals(lib, over, expect):
    assert _read(lib, **over) == expect


def _norm_rope(lib, **over):
    a = dict(qo=16, qos=1024, ko=16, kos=256, q=16, qs=1024, k=16, ks=256, qw=16, kw=16, eps=1e-6,
             pos=16, ps=3, axes=1, pa=None, freq=16, rot=64, inter=0, f=1.0, T=3, Hq=8, Hkv=2,
             D=128, dtype=0)
    a.update(over)
    return lib.pkv_qk_norm_rope(
        a["qo"], a["qos"], a["ko"], a["kos"], a["q"], a["qs"], a["k"], a["ks"], a["qw"], a["kw"],
        a["eps"], a["pos"], a["ps"], a["axes"], a["pa"], a["freq"], a["rot"], a["inter"], a["f"],
        a["T"], a["Hq"], a["Hkv"], a["D"], a["dtype"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(T=0, q=None), 0),
    (dict(T=-1), INVALID), (dict(rot=0), INVALID), (dict(rot=63), INVALID), (dict(rot=130), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(dtype=5), INVALID), (dict(f=math.nan), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=math.inf), INVALID),
    (dict(axes=0), INVALID), (dict(axes=256), INVALID), (dict(ps=2), INVALID),
    (dict(axes=3, pa=bytes([0, 1, 2, 3] * 8)), INVALID),   # no axis 3
    (dict(qs=1020), INVALID), (dict(qs=1016), INVALID), (dict(kos=248), INVALID),
    (dict(q=16, qo=16, qos=2048), INVALID), (dict(k=32, ko=32, ks=512), INVALID),
    (dict(q=8), INVALID), (dict(kw=8), INVALID), (dict(freq=20), INVALID), (dict(pos=18), INVALID),
    (dict(ko=None), INVALID),
    (dict(Hq=70000, qs=70000 * 128, qos=70000 * 128), UNSUPPORTED),
])
def test_norm_rope_refusals(lib, over, expect):
    assert _norm_rope(lib, **over) == expect


def _decode(lib, **over):
    a = dict(out=16, q=16, k=16, v=16, ks=16, vs=16, tables=16, mbps=4, lens=16, maxctx=64, S=2,
             Hq=8, Hkv=2, D=128, B=16, NB=10, scale=0.1, dtype=0, part=0, ws=None, wsb=0)
    a.update(over)
    return lib.pkv_paged_attn_decode_fp8(
        a["out"], a["q"], a["k"], a["v"], a["ks"], a["vs"], a["tables"], a["mbps"], a["lens"],
        a["maxctx"], a["S"], a["Hq"], a["Hkv"], a["D"], a["B"], a["NB"], a["scale"], a["dtype"],
        a["part"], a["ws"], a["wsb"], None)


def _tree(lib, **over):
    a = dict(out=16, q=16, T=9, start=16, mql=8, masks=16, k=16, v=16, ks=16, vs=16, tables=16,
             mbps=4, lens=16, maxctx=64, S=2, Hq=8, Hkv=2, D=64, B=16, NB=10, scale=0.1, dtype=0,
             part=0, ws=None, wsb=0)
    a.update(over)
    return lib.pkv_paged_attn_tree_fp8(
        a["out"], a["q"], a["T"], a["start"], a["mql"], a["masks"], a["k"], a["v"], a["ks"],
        a["vs"], a["tables"], a["mbps"], a["lens"], a["maxctx"], a["S"], a["Hq"], a["Hkv"], a["D"],
        a["B"], a["NB"], a["scale"], a["dtype"], a["part"], a["ws"], a["wsb"], None)


_BOTH = [
    (dict(S=0, q=None), 0),
    (dict(S=-1), INVALID), (dict(Hq=7), INVALID), (dict(dtype=7), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(B=24), UNSUPPORTED), (dict(part=96), INVALID), (dict(part=-128), INVALID),
    (dict(scale=math.nan), INVALID), (dict(maxctx=-1), INVALID), (dict(mbps=3), INVALID),
    (dict(mbps=0, maxctx=0), INVALID), (dict(NB=0), INVALID),
    (dict(out=8), INVALID), (dict(q=None), INVALID), (dict(k=24), INVALID), (dict(ks=8), INVALID),
    (dict(vs=None), INVALID), (dict(tables=2), INVALID), (dict(lens=None), INVALID),
    (dict(maxctx=(1 << 30) + 1, mbps=1 << 27), UNSUPPORTED),
    (dict(NB=1 << 26, Hkv=2), UNSUPPORTED),                # rows of the pool beyond 32 bits
    (dict(maxctx=512, mbps=32, part=128), WORKSPACE),
    (dict(maxctx=512, mbps=32, part=128, ws=24, wsb=1 << 20), INVALID),
    (dict(S=65536, maxctx=64), UNSUPPORTED),
]


@pytest.mark.parametrize("over,expect", _BOTH)
def test_decode_refusals(lib, over, expect):
    assert _decode(lib, **over) == expect


@pytest.mark.parametrize("over,expect", _BOTH + [
    (dict(T=0, q=None), 0), (dict(mql=0, q=None), 0),
    (dict(T=-1), INVALID), (dict(mql=-1), INVALID), (dict(mql=65), UNSUPPORTED),
    (dict(start=None), INVALID), (dict(masks=None), INVALID), (dict(masks=20), INVALID),
    (dict(start=18), INVALID),
])
def test_tree_refusals(lib, over, expect):
    assert _tree(lib, **over) == expect


def test_workspace_sizes(lib):
    decode, tree = lib.pkv_decode_fp8_workspace_size, lib.pkv_tree_fp8_workspace_size
    # partial outputs, maxima and sums per row, head and partition
    assert decode(8, 32, 8, 128, 32768, 512) == 8 * 32 * 64 * (128 + 2) * 4
    assert decode(8, 32, 8, 128, 4096, 4096) == 0
    assert tree(20, 9, 3, 32, 8, 64, 300, 128) == 20 * 32 * 3 * (64 + 2) * 4
    assert decode(8, 32, 8, 96, 100, 0) == NONE and decode(8, 32, 8, 128, 100, 64) == NONE
    assert tree(20, 65, 3, 32, 8, 64, 300, 128) == NONE
    with pytest.raises(ValueError, match="sizes"):
        pkv.decode_fp8_workspace_size(8, 30, 8, 128, 100)
    with pytest.raises(ValueError, match="32 bits"):
        pkv.tree_fp8_workspace_size(8, 1 << 40, 8, 32, 8, 128, 100)


def test_binding_refuses_host_tensors():
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    cache = torch.zeros((3, 2, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.zeros((3, 2, 16, 1), dtype=torch.bfloat16)
    i64, i32 = torch.zeros(2, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_append_fp8(x, x, cache, cache, scales, scales, i64)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.block_read_fp8(x, x, cache, cache, scales, scales, i64)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.qk_norm_rope(x, x, x, x, i32, torch.ones(8, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attn_decode_fp8(x, x, cache, cache, scales, scales, i32[None], i32, 1.0, 4)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attn_tree_fp8(x, x, i32, i64, cache, cache, scales, scales, i32[None], i32, 1.0,
                                4, 1)
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        pkv.kv_append_fp8(x.float(), x, cache, cache, scales, scales, i64)
