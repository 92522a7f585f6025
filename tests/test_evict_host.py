"""The eviction calls on a machine without a GPU: refusals on the host, the
rotary frequencies, and the allocator's shrinking of sequences."""

import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_247_gb300 as pkv

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def _rope(lib, **over):
    a = dict(qo=16, qos=1024, q=16, qs=1024, k=16, ks=256, v=16, vs=256, pos=16, freq=16, rot=64,
             inter=0, f=1.0, kc=16, vc=16, slot=16, T=3, Hq=8, Hkv=2, D=128, B=16, NB=4, dtype=0)
    a.update(over)
    return lib.pkv_rope_kv_append(
        a["qo"], a["qos"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["freq"],
        a["rot"], a["inter"], a["f"], a["kc"], a["vc"], a["slot"], a["T"], a["Hq"], a["Hkv"],
        a["D"], a["B"], a["NB"], a["dtype"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(T=0, q=None), 0),
    (dict(T=-1), INVALID),
    (dict(rot=0), INVALID), (dict(rot=63), INVALID), (dict(rot=130), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(B=24), UNSUPPORTED), (dict(dtype=5), INVALID),
    (dict(f=math.nan), INVALID),
    (dict(qs=1020), INVALID),             # not a multiple of 16 bytes
    (dict(qs=1016), INVALID),             # shorter than a token's row
    (dict(ks=248), INVALID),
    (dict(qo=16, q=16, qos=2048), INVALID),  # in place with another stride
    (dict(q=8), INVALID), (dict(kc=8), INVALID), (dict(freq=20), INVALID),
    (dict(pos=18), INVALID), (dict(slot=12), INVALID), (dict(slot=None), INVALID),
    (dict(Hq=70000, qs=70000 * 128, qos=70000 * 128), UNSUPPORTED),
    (dict(NB=0), INVALID),
])
def test_rope_refusals(lib, over, expect):
    assert _rope(lib, **over) == expect


def _decode(lib, **over):
    a = dict(out=16, w=16, ws=64, decay=1.0, q=16, k=16, v=16, tables=16, mbps=4, lens=16,
             maxctx=64, S=2, Hq=8, Hkv=2, D=128, B=16, NB=10, scale=0.1, dtype=0, part=0, wk=16,
             wkb=1 << 20)
    a.update(over)
    return lib.pkv_paged_attn_decode_weights(
        a["out"], a["w"], a["ws"], a["decay"], a["q"], a["k"], a["v"], a["tables"], a["mbps"],
        a["lens"], a["maxctx"], a["S"], a["Hq"], a["Hkv"], a["D"], a["B"], a["NB"], a["scale"],
        a["dtype"], a["part"], a["wk"], a["wkb"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(S=0, q=None), 0),
    (dict(w=None), INVALID), (dict(w=18), INVALID), (dict(ws=63), INVALID),
    (dict(decay=math.inf), INVALID), (dict(scale=math.nan), INVALID),
    (dict(Hq=66), UNSUPPORTED),             # a group of 33
    (dict(part=96), UNSUPPORTED),           # not whole 128-key tiles
    (dict(part=48), INVALID),
    (dict(wk=None), WORKSPACE), (dict(wkb=100), WORKSPACE), (dict(wk=24), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(mbps=3), INVALID), (dict(Hq=7), INVALID),
])
def test_decode_weights_refusals(lib, over, expect):
    assert _decode(lib, **over) == expect


def test_decode_weights_workspace(lib):
    size = lib.pkv_decode_weights_workspace_size
    # unsplit: two rows of logits per query head of the group and CTA (one CTA per
    # (sequence, KV head) here), padded to 16 bytes
    assert size(2, 8, 2, 128, 61, 0) == 4 * (4 * 2 * 4 * 64)
    # split in three: the partial outputs, maxima and sums, every logit, and the
    # scratch of 12 CTAs for sequences of one partition
    assert size(2, 8, 2, 64, 300, 128) == 4 * (2 * 8 * 3 * 66 + 2 * 8 * 300 + 12 * 2 * 4 * 128)
    # 512 items on 152 SMs (assumed here): 4 rounds of 128 CTAs
    assert size(64, 32, 8, 128, 8192, 8192) == 4 * (128 * 2 * 4 * 8192)
    assert size(2, 8, 2, 128, 0, 0) == 0
    for bad in ((2, 66, 2, 128, 64, 0), (2, 8, 2, 128, 64, 96), (2, 8, 2, 96, 64, 0),
                (2, 7, 2, 128, 64, 0), (2, 8, 2, 128, (1 << 30) + 1, 0)):
        assert size(*bad) == ctypes.c_size_t(-1).value
    assert lib.pkv_prefill_weights_workspace_size(5, 8) == 160
    assert lib.pkv_prefill_weights_workspace_size(-1, 8) == ctypes.c_size_t(-1).value


def _prefill(lib, **over):
    a = dict(out=16, w=16, ws=64, decay=1.0, window=0, q=16, T=16, qs=16, mql=8, k=16, v=16,
             tables=16, mbps=4, lens=16, maxctx=64, S=2, Hq=8, Hkv=2, D=128, B=16, NB=10,
             scale=0.1, dtype=1, wk=16, wkb=16 * 8 * 4)
    a.update(over)
    return lib.pkv_paged_attn_prefill_weights(
        a["out"], a["w"], a["ws"], a["decay"], a["window"], a["q"], a["T"], a["qs"], a["mql"],
        a["k"], a["v"], a["tables"], a["mbps"], a["lens"], a["maxctx"], a["S"], a["Hq"], a["Hkv"],
        a["D"], a["B"], a["NB"], a["scale"], a["dtype"], a["wk"], a["wkb"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(S=0, q=None), 0), (dict(T=0, q=None), 0), (dict(mql=0), 0),
    (dict(window=-1), INVALID), (dict(w=None), INVALID), (dict(ws=63), INVALID),
    (dict(decay=math.nan), INVALID), (dict(wkb=16 * 8 * 4 - 1), WORKSPACE),
    (dict(wk=None), WORKSPACE), (dict(wk=8), INVALID), (dict(Hq=258), UNSUPPORTED),
    (dict(B=4), UNSUPPORTED),
])
def test_prefill_weights_refusals(lib, over, expect):
    assert _prefill(lib, **over) == expect


def _select(lib, **over):
    a = dict(keep=16, new=None, w=16, ws=64, lens=32, maxctx=64, S=2, H=2, budget=16, recent=4,
             sinks=2)
    a.update(over)
    return lib.pkv_kv_evict_select(a["keep"], a["new"], a["w"], a["ws"], a["lens"], a["maxctx"],
                                   a["S"], a["H"], a["budget"], a["recent"], a["sinks"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(S=0, keep=None), 0),
    (dict(budget=0), INVALID), (dict(recent=15), INVALID), (dict(recent=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(sinks=13), INVALID), (dict(ws=60), INVALID),
    (dict(maxctx=-1), INVALID), (dict(keep=None), INVALID), (dict(w=18), INVALID),
    (dict(new=32), INVALID),              # context_lens itself: other heads still read it
    (dict(S=70000), UNSUPPORTED), (dict(budget=(1 << 30) + 1), UNSUPPORTED),
])
def test_select_refusals(lib, over, expect):
    assert _select(lib, **over) == expect


def _compact(lib, **over):
    a = dict(k=16, v=16, w=16, ws=64, src=16, mb=4, dst=16, db=1, keep=16, budget=16, lens=16,
             maxctx=64, S=2, H=2, D=128, B=16, NB=10, dtype=0)
    a.update(over)
    return lib.pkv_kv_compact(a["k"], a["v"], a["w"], a["ws"], a["src"], a["mb"], a["dst"],
                              a["db"], a["keep"], a["budget"], a["lens"], a["maxctx"], a["S"],
                              a["H"], a["D"], a["B"], a["NB"], a["dtype"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(S=0, k=None), 0),
    (dict(budget=0), INVALID), (dict(budget=17), INVALID),  # more than the destination holds
    (dict(mb=3), INVALID), (dict(ws=63), INVALID), (dict(w=18), INVALID),
    (dict(D=32), UNSUPPORTED), (dict(B=12), UNSUPPORTED), (dict(dtype=2), INVALID),
    (dict(k=8), INVALID), (dict(keep=None), INVALID), (dict(dst=17), INVALID),
    (dict(H=70000), UNSUPPORTED), (dict(NB=0), INVALID),
])
def test_compact_refusals(lib, over, expect):
    assert _compact(lib, **over) == expect


def test_binding_refuses_host_tensors():
    half = torch.zeros((2, 4, 64), dtype=torch.float16)
    cache = torch.zeros((3, 2, 16, 64), dtype=torch.float16)
    i32 = torch.zeros(2, dtype=torch.int32)
    w = torch.zeros((2, 2, 48))
    table = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkv.rope_kv_append(half, half, half[:, :2], half[:, :2], i32,
                           torch.zeros(32, dtype=torch.float64), cache, cache, i32.long())
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkv.paged_attn_decode_weights(half, w, half, cache, cache, table, i32, 0.1, 48)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkv.paged_attn_prefill_weights(half, w, half, i32, cache, cache, table, i32, 0.1, 48, 1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkv.kv_evict_select(torch.zeros((2, 2, 8), dtype=torch.int32), w, i32, 48)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkv.kv_compact(cache, cache, table, torch.zeros((2, 2, 8), dtype=torch.int32), i32)


def test_rope_frequencies():
    plain = pkv.rope_frequencies(8, base=16.0, device="cpu")
    assert plain.dtype == torch.float64
    assert torch.allclose(plain, torch.tensor([1, 0.5, 0.25, 0.125], dtype=torch.float64))
    assert torch.allclose(pkv.rope_frequencies(8, 16.0, "linear", 4.0, device="cpu"), plain / 4)
    raised = pkv.rope_frequencies(8, 16.0, "base", 4.0, device="cpu")
    assert raised[0] == 1 and math.isclose(raised[-1], 0.125 / 4)
    assert (raised[1:-1] < plain[1:-1]).all() and (raised[1:-1] > plain[1:-1] / 4).all()
    # 1, 0.5, 0.25, 0.125 radians over 16 pi positions: 8, 4, 2, 1 turns
    bands = pkv.rope_frequencies(8, 16.0, "bands", 4.0, original_len=16 * math.pi, low=1.0,
                                 high=4.0, device="cpu")
    mixed = 0.25 / 3 + 0.25 / 4 * 2 / 3
    assert torch.allclose(bands, torch.tensor([1, 0.5, mixed, 0.125 / 4], dtype=torch.float64))
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, base=1.0),
                dict(rot_dim=8, factor=0.5), dict(rot_dim=8, scaling="other"),
                dict(rot_dim=8, scaling="bands"), dict(rot_dim=2, scaling="base")):
        with pytest.raises(ValueError):
            pkv.rope_frequencies(device="cpu", **bad)


# ---- the allocator ---------------------------------------------------------


def test_shrink_frees_the_tail(lib):
    a = pkv.BlockAllocator(10, 4)
    a.add_seq(1, 18)                       # five blocks
    before = a.block_table([1], 5)[0]
    a.shrink_seqs([1], [7])
    assert a.seq_info(1) == (7, 2)
    assert a.block_table([1], 2)[0].tolist() == before[:2].tolist()
    assert a.stats()["free_blocks"] == 8 and a.stats()["cow_copies"] == 0
    a.shrink_seqs([1], [7])                # nothing to do
    slot, src, dst = a.append_slot(1)      # goes on in the last kept block
    assert slot == before[1] * 4 + 3 and (src, dst) == (-1, -1)
    a.shrink_seqs([1], [0])
    assert a.seq_info(1) == (0, 0) and a.stats()["free_blocks"] == 10


def test_shrink_replaces_shared_blocks(lib):
    a = pkv.BlockAllocator(12, 4)
    a.add_seq(1, 12)
    a.fork(1, 2)
    a.fork(1, 3)
    shared = a.block_table([1], 3)[0].tolist()
    a.shrink_seqs([1, 2], [5, 12])         # 2 keeps its length: untouched
    t1, t2 = a.block_table([1, 2], 3).tolist()
    assert t2 == shared and t1[2] == -1 and not set(t1[:2]) & set(shared)
    assert [a.refcount(b) for b in shared] == [2, 2, 2]
    # both remaining owners at once: neither gets a block the other reads
    a.shrink_seqs([2, 3], [8, 4])
    t2, t3 = a.block_table([2, 3], 2).tolist()
    assert not set(t2) & set(shared) and t3[0] not in shared and t3[0] not in t2
    assert [a.refcount(b) for b in shared] == [0, 0, 0]
    assert a.stats()["used_blocks"] == 2 + 2 + 1


def test_shrink_is_all_or_nothing(lib):
    a = pkv.BlockAllocator(4, 4)
    a.add_seq(1, 12)
    a.fork(1, 2)
    state = (a.block_table([1, 2], 3).tolist(), a.stats())
    with pytest.raises(pkv.OutOfBlocks):
        a.shrink_seqs([1], [8])            # needs two fresh blocks, one is free
    for ids, lens, status in (([1, 9], [4, 4], 6), ([1, 1], [4, 4], 1), ([1], [13], 1),
                              ([1], [-1], 1)):
        with pytest.raises(pkv.PagedKVError) as e:
            a.shrink_seqs(ids, lens)
        assert e.value.status == status
    with pytest.raises(ValueError):
        a.shrink_seqs([1, 2], [4])
    assert (a.block_table([1, 2], 3).tolist(), a.stats()) == state
    a.shrink_seqs([], [])
    a.shrink_seqs([1], [4])                # one fresh block: fits
    assert a.stats()["free_blocks"] == 0


@pytest.mark.parametrize("seed", range(4))
def test_shrink_conserves_blocks(lib, seed):
    rng = np.random.default_rng(seed)
    a = pkv.BlockAllocator(200, 4)
    live = {}
    for step in range(300):
        op = rng.integers(4)
        if op == 0 and len(live) < 12:
            live[step] = int(rng.integers(0, 40))
            try:
                a.add_seq(step, live[step])
            except pkv.OutOfBlocks:
                del live[step]
        elif op == 1 and live and len(live) < 12:
            parent = int(rng.choice(list(live)))
            a.fork(parent, step)
            live[step] = live[parent]
        elif op == 2 and live:
            some = [int(s) for s in rng.permutation(list(live))[:3]]
            lens = [int(rng.integers(0, live[s] + 1)) for s in some]
            shared = {b for s in live for b in a.block_table([s], 20)[0] if b >= 0 and a.refcount(b) > 1}
            try:
                a.shrink_seqs(some, lens)
            except pkv.OutOfBlocks:
                continue
            for s, n in zip(some, lens):
                table = [b for b in a.block_table([s], 20)[0] if b >= 0]
                assert len(table) == -(-n // 4) == a.seq_info(s)[1]
                if n < live[s]:
                    assert not set(table) & shared
                    assert all(a.refcount(b) == 1 for b in table)
                live[s] = n
        elif live:
            gone = int(rng.choice(list(live)))
            a.free_seq(gone)
            del live[gone]
        owners = {}
        for s in live:
            for b in a.block_table([s], 20)[0]:
                if b >= 0:
                    owners[b] = owners.get(b, 0) + 1
        assert all(a.refcount(b) == n for b, n in owners.items())
        assert a.stats()["used_blocks"] == len(owners)
    for s in list(live):
        a.free_seq(s)
    assert a.stats()["free_blocks"] == 200
