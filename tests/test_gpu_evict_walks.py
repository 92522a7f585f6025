"""The eviction operators on launches large enough that a CTA (or a warp) goes
through several pieces of work: decode with weights on several times as many
(sequence, KV head) pairs as SMs, compaction by one, two and four warps per
CTA, and rotary appends of several tokens per CTA.  Tolerances as derived in
tests/test_gpu_evict.py."""

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_247_gb300 as pkv
from paged_kv_cache_247_gb300 import workloads as W
from _gpu_util import assert_within_tol, oracle_decode, raw_bytes, to_f64
from test_gpu_evict import _check_rotated, _check_weights, _keep_of, _old_weights, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status(lib, cuda_device):
    pkv.device_status(clear=True)
    yield
    assert pkv.device_status(clear=True) == 0


@pytest.mark.parametrize("dtype,hq,hkv,D,B,longest,part", [
    ("bf16", 32, 8, 128, 16, 300, 384),      # unsplit, a group of 4
    ("bf16", 32, 8, 128, 16, 700, 128),      # empty, unsplit and split items in turn
    ("fp16", 40, 40, 64, 8, 290, 384),       # single heads
    ("bf16", 96, 8, 64, 32, 500, 128),       # a group of 12
    ("fp16", 256, 8, 128, 16, 260, 384),     # a group of 32
    ("fp16", 160, 8, 128, 64, 400, 256),     # a group of 20: most sequences whole, some in two
])
def test_decode_weights_many_items(cuda_device, dtype, hq, hkv, D, B, longest, part):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    S = 4 * sms // hkv + 3                               # five items a CTA, or more
    rng = np.random.default_rng(hq + D)
    lens = rng.integers(0, longest + 1, S)
    lens[::7] = 0
    lens[3::11] = rng.integers(1, 4, len(lens[3::11]))
    lens[S // 2], lens[S - 1] = longest, 129
    case = W.make_decode_case(hq + B, S, hq, hkv, D, B, dtype, lens.tolist(), pool_factor=1.1,
                              poison=True, device=cuda_device)
    weights = _old_weights(S, hkv, longest + 3, 5)
    old = weights.clone()
    ws = torch.full((pkv.decode_weights_workspace_size(S, hq, hkv, D, longest, part) // 4,),
                    float("nan"), device="cuda")
    out = torch.full_like(case.q, float("nan"))
    args = (case.k_cache, case.v_cache, case.block_tables, case.context_lens)
    pkv.paged_attn_decode_weights(out, weights, case.q, *args, case.scale, longest, decay=0.5,
                                  partition_size=part, workspace=ws)
    # a few sequences by the oracle
    some = sorted({0, 3, S // 2, S - 2, S - 1} | {int(s) for s in rng.choice(S, 5)})
    assert_within_tol(out[some], oracle_decode(case, seqs=some), case.q.dtype, "out")
    _check_weights(weights, old, case, case.q, [1] * S, 0.5, seqs=some)
    # and every one, bit for bit, by calls so small that no CTA takes a second item
    step = max(1, sms // (hkv * -(-longest // part)))
    for a in range(0, S, step):
        b = min(S, a + step)
        w, o = old[a:b].clone(), torch.full_like(case.q[a:b], float("nan"))
        pkv.paged_attn_decode_weights(o, w, case.q[a:b].contiguous(), *args[:2],
                                      case.block_tables[a:b].contiguous(),
                                      case.context_lens[a:b].contiguous(), case.scale, longest,
                                      decay=0.5, partition_size=part)
        assert torch.equal(o, out[a:b]), (a, b)
        assert torch.equal(w, weights[a:b]), (a, b)


@pytest.mark.parametrize("dtype,S,H,D,B,budget,fresh", [
    ("fp16", 13, 8, 128, 16, 400, False),    # 104 pairs: four warps per CTA
    ("bf16", 26, 8, 64, 8, 401, True),       # 208: two
    ("bf16", 40, 8, 128, 16, 390, True),     # 320: one
    ("fp16", 20, 40, 64, 32, 300, False),    # 800: one, shorter rings
    ("bf16", 17, 40, 128, 128, 333, False),
])
def test_compact_many_pairs(cuda_device, dtype, S, H, D, B, budget, fresh):
    lens = [(budget + 300 - 37 * s) % (budget + 301) for s in range(S)]
    case = W.make_decode_case(D + B, S, H, H, D, B, dtype, lens, pool_factor=2.2, poison=True,
                              device=cuda_device)
    keep = _keep_of(lens, H, budget, 4)
    src = case.block_tables.cpu().numpy()
    dst = np.ascontiguousarray(src[:, :-(-budget // B)])
    if fresh:
        used = set(src[src >= 0].tolist())
        free = [b for b in range(case.num_blocks) if b not in used]
        for s in range(S):
            for i in range(s % 2, -(-min(lens[s], budget) // B), 2):
                dst[s, i] = free.pop()
    weights = _old_weights(S, H, max(lens) + 3, 2)
    k0, v0, w0 = raw_bytes(case.k_cache), raw_bytes(case.v_cache), to_f64(weights)
    pkv.kv_compact(case.k_cache, case.v_cache, case.block_tables,
                   torch.from_numpy(keep).to(cuda_device), case.context_lens, weights=weights,
                   dst_tables=torch.from_numpy(dst).to(cuda_device), max_context_len=max(lens))
    for cache, was in ((case.k_cache, k0), (case.v_cache, v0)):
        ref = oracle.compact(was.reshape(cache.shape), src, dst, keep, lens)
        assert np.array_equal(raw_bytes(cache).reshape(cache.shape), ref)
    assert np.array_equal(to_f64(weights), oracle.compact_weights(w0, keep, lens))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,hq,hkv,D,rot,T", [
    ("bf16", 8, 2, 64, 32, 2049),            # two tokens a CTA, and one in the last
    ("fp16", 4, 1, 64, 64, 5003),            # four
    ("bf16", 6, 2, 128, 32, 8197),           # six, as many as give each thread its two units
    ("fp16", 2, 1, 64, 16, 9001),            # eight, the most
])
def test_rope_many_tokens(cuda_device, dtype, hq, hkv, D, rot, T, interleaved):
    dt, B = W.DTYPES[dtype], 16
    rng = np.random.default_rng(T)
    qkv = _randn((T, hq + 2 * hkv, D), 3, dt)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    before = to_f64(qkv)
    NB = -(-T // B) + 3
    kc, vc = _randn((NB, hkv, B, D), 8, dt), _randn((NB, hkv, B, D), 9, dt)
    kc0, vc0 = to_f64(kc), to_f64(vc)
    slots = rng.permutation(NB * B)[:T].astype(np.int64)
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    slots[rng.choice(T, T // 9, replace=False)] = -1
    pos[rng.choice(T, T // 7, replace=False)] = -1
    freq = pkv.rope_frequencies(rot)
    pkv.rope_kv_append(q, q, k, v, torch.from_numpy(pos).to(cuda_device), freq, kc, vc,
                       torch.from_numpy(slots).to(cuda_device), interleaved=interleaved)
    f64, real = freq.cpu().numpy(), pos >= 0
    now = to_f64(qkv)
    assert np.array_equal(now[:, hq:], before[:, hq:])
    assert np.array_equal(now[~real], before[~real])
    _check_rotated(q[torch.from_numpy(real)], before[real, :hq], pos[real], f64, interleaved, 1.0, dt)
    stored = real & (slots >= 0)
    blk, off = slots[stored] // B, slots[stored] % B
    _check_rotated(kc[torch.from_numpy(blk), :, torch.from_numpy(off)],
                   before[stored, hq:hq + hkv], pos[stored], f64, interleaved, 1.0, dt)
    vc0[blk, :, off] = before[stored, hq + hkv:]
    assert np.array_equal(to_f64(vc), vc0)
    kc_now = to_f64(kc)
    kc_now[blk, :, off] = kc0[blk, :, off]
    assert np.array_equal(kc_now, kc0)
