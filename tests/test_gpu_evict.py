"""The eviction operators on the GPU against the fp64 oracle.

Tolerances.  Byte moves and choices are exact.  A rotated element is rounded
once to its type (off by at most half a step, eps / 2 relative) after fp32
arithmetic: cos and sin within 2^-22 (the reduced angle is rounded to fp32,
2^-26 turns = 2^-23.3 radians, and sincospif adds 2 ulp), two products and a
sum, so 2^-21 (|first| + |second|) in all.  An attention weight is
2^(x - lse): the logit is an fp32 sum of D exact products, off by at most
(D / 16 + 8) 2^-23 of the sum of their magnitudes a (16 products per MMA
step, each step's alignment and rounding below 2^-23 of the running sum, and
the scaling), lse as much again; the exponential, the logarithm, the
differences at magnitudes below 64 and the fp32 sums add less than 2^-17
relative.  So |err| <= w (2 (D / 16 + 8) 2^-23 max a + 2^-17), plus 2^-24 of
the decayed old weight.
"""

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_247_gb300 as pkv
from paged_kv_cache_247_gb300 import _lib
from paged_kv_cache_247_gb300 import workloads as W
from _gpu_util import assert_within_tol, oracle_decode, raw_bytes, to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status(lib, cuda_device):
    pkv.device_status(clear=True)
    yield
    assert pkv.device_status(clear=True) == 0


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, seed, dtype):
    return torch.randn(shape, generator=_gen(seed), device="cuda").to(dtype)


# ---- rotary positions with append --------------------------------------------------------------


def _check_rotated(got, x, positions, inv_freq, interleaved, factor, dtype):
    """Within the bound above, per element (x: the rows before, fp64)."""
    ref = oracle.rope(x, positions, inv_freq, interleaved, factor)
    mag = oracle.rope(np.abs(x), np.zeros_like(positions), inv_freq, interleaved, 1.0)
    half, r = len(inv_freq), 2 * len(inv_freq)
    pair = np.zeros_like(x)
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, half), slice(half, r))
    pair[..., a] = pair[..., b] = mag[..., a] + mag[..., b]
    # subnormal fp16 results round by an absolute half step
    bound = (torch.finfo(dtype).eps / 2 * np.abs(ref) + abs(factor) * pair * 2.0 ** -21
             + (2.0 ** -25 if dtype == torch.float16 else 0.0) * (pair > 0))
    g = to_f64(got)
    assert (np.abs(g - ref) <= bound * (1 + 1e-6)).all(), np.abs(g - ref).max()
    assert np.array_equal(g[..., r:], x[..., r:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,hq,hkv,D,B,rot,T,packed,inplace", [
    ("fp16", 8, 8, 64, 16, 64, 1, False, False),
    ("bf16", 32, 8, 128, 16, 128, 37, True, False),
    ("fp16", 12, 4, 128, 8, 64, 65, True, True),
    ("bf16", 5, 5, 64, 32, 34, 9, False, True),      # pairs that do not fill 16-byte chunks
    ("fp16", 3, 1, 128, 128, 2, 130, True, False),
    ("bf16", 40, 40, 128, 64, 96, 300, False, False),
    ("fp16", 7, 1, 64, 16, 46, 31, True, True),
])
def test_rope_append(cuda_device, dtype, hq, hkv, D, B, rot, T, packed, inplace, interleaved):
    dt = W.DTYPES[dtype]
    rng = np.random.default_rng(T * 7 + rot)
    if packed:
        qkv = _randn((T, hq + 2 * hkv, D), 3, dt)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = (_randn((T, n, D), 4 + n, dt) for n in (hq, hkv, hkv))
    q64, k64, v64 = to_f64(q), to_f64(k), to_f64(v)
    NB = -(-T // B) + 3
    kc, vc = _randn((NB, hkv, B, D), 8, dt), _randn((NB, hkv, B, D), 9, dt)
    kc0, vc0 = to_f64(kc), to_f64(vc)
    slots = rng.permutation(NB * B)[:T].astype(np.int64)
    pos = rng.integers(0, 1 << 21, T).astype(np.int32)
    pos[0] = 0
    if T > 4:
        slots[1], pos[2], slots[3] = -1, -1, -7   # not stored; padding; not stored
    freq = pkv.rope_frequencies(rot, 500000.0)
    q_out = q if inplace else torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    before = to_f64(q_out)
    res = pkv.rope_kv_append(q_out, q, k, v, torch.from_numpy(pos).to(cuda_device), freq, kc, vc,
                             torch.from_numpy(slots).to(cuda_device), interleaved=interleaved,
                             attn_factor=1.25)
    assert res is q_out
    f64 = freq.cpu().numpy()
    real = pos >= 0
    _check_rotated(q_out[torch.from_numpy(real)], q64[real], pos[real], f64, interleaved, 1.25, dt)
    assert np.array_equal(to_f64(q_out)[~real], before[~real])   # padding rows as they were
    stored = real & (slots >= 0)
    blk, off = slots[stored] // B, slots[stored] % B
    _check_rotated(kc[torch.from_numpy(blk), :, torch.from_numpy(off)], k64[stored], pos[stored],
                   f64, interleaved, 1.25, dt)
    vc0[blk, :, off] = v64[stored]
    assert np.array_equal(to_f64(vc), vc0)
    kc_now = to_f64(kc)
    kc_now[blk, :, off] = kc0[blk, :, off]
    assert np.array_equal(kc_now, kc0)                           # other slots as they were
    if packed and not inplace:
        assert np.array_equal(to_f64(q), q64)


def test_rope_far_positions(cuda_device):
    """The angle is reduced in 64 bits: positions up to 2^31 - 1."""
    pos = np.array([0, 1, 1 << 20, 999999937, 2147483647], dtype=np.int32)
    T = len(pos)
    q, k, v = (_randn((T, 2, 64), i, torch.float16) for i in range(3))
    freq = pkv.rope_frequencies(64)
    kc = torch.zeros((1, 2, 16, 64), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    out = pkv.rope_kv_append(torch.empty_like(q), q, k, v, torch.from_numpy(pos).cuda(), freq, kc,
                             vc, torch.arange(T, device="cuda"))
    _check_rotated(out, to_f64(q), pos, freq.cpu().numpy(), False, 1.0, torch.float16)


def test_rope_refuses_and_flags(cuda_device):
    T, D = 4, 64
    q = _randn((T, 4, D), 0, torch.bfloat16)
    k, v = _randn((T, 2, D), 1, torch.bfloat16), _randn((T, 2, D), 2, torch.bfloat16)
    kc = torch.zeros((2, 2, 8, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freq = pkv.rope_frequencies(D)
    slots = torch.arange(T, device="cuda")
    call = lambda **o: pkv.rope_kv_append(*[o.get(n, d) for n, d in (  # noqa: E731
        ("q_out", torch.empty_like(q)), ("q", q), ("k", k), ("v", v), ("positions", pos),
        ("inv_freq", freq), ("k_cache", kc), ("v_cache", vc), ("slots", slots))])
    for bad in (dict(positions=pos.long()), dict(inv_freq=freq.float()), dict(slots=slots.int()),
                dict(k=k.half()), dict(v=v[:3]), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(q_out=torch.empty((T, 3, D), dtype=q.dtype, device="cuda")),
                dict(positions=pos.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(pkv.PagedKVError):
        call(inv_freq=pkv.rope_frequencies(2 * D))
    assert torch.count_nonzero(kc) == 0
    call(slots=torch.tensor([0, 16, 1, 1 << 40], device="cuda"))   # two beyond the 16 slots
    assert pkv.device_status(clear=True) == _lib.DEV_BAD_SLOT
    assert np.array_equal(to_f64(vc)[0, :, :2], to_f64(v)[[0, 2]].transpose(1, 0, 2))
    assert torch.count_nonzero(vc[0, :, 2:]) == 0 and torch.count_nonzero(vc[1]) == 0


# ---- attention with accumulated weights ---------------------------------------------------------


def _weights_bound(case_q, k_cache, w, scale, D):
    a = abs(scale) * D * float(case_q.abs().max()) * float(k_cache[k_cache == k_cache].abs().max())
    # the sum of magnitudes is far below the product of the maxima: Cauchy-Schwarz over the rows
    a = min(a, abs(scale) * float(case_q.float().norm(dim=-1).max())
            * float(torch.nan_to_num(k_cache.float()).norm(dim=-1).max()))
    return np.abs(w) * (2 * (D / 16 + 8) * 2.0 ** -23 * a + 2.0 ** -17)


def _check_weights(got, old, case, q, query_counts, decay, window=0, seqs=None):
    """Held positions by the oracle, the others untouched."""
    S = case.context_lens.shape[0]
    tables, lens = case.block_tables.cpu().numpy(), case.context_lens.cpu().numpy()
    k64 = to_f64(case.k_cache)
    g, o = to_f64(got), to_f64(old)
    D, row = q.shape[2], 0
    q64 = to_f64(q)
    for s in range(S):
        n, l = int(lens[s]), int(query_counts[s])
        if seqs is None or s in seqs:
            if n == 0 or l == 0:
                assert np.array_equal(g[s], o[s], equal_nan=True), s
            else:
                w = oracle.attention_weights(q64[row:row + l], k64, tables[s], n, case.scale, window)
                base = decay * o[s, :, :n] if decay else 0.0
                bound = _weights_bound(q, case.k_cache, w, case.scale, D) + 2.0 ** -24 * np.abs(base)
                err = np.abs(g[s, :, :n] - (w + base))
                assert (err <= bound + 2.0 ** -23 * np.abs(w + base)).all(), (s, (err - bound).max())
                assert np.array_equal(g[s, :, n:], o[s, :, n:], equal_nan=True), s
        row += l


def _old_weights(S, H, width, seed):
    return torch.rand((S, H, width), generator=_gen(seed), device="cuda") * 3


@pytest.mark.parametrize("dtype,hq,hkv,D,B,lens,part,decay,slack", [
    ("fp16", 8, 8, 64, 16, [1, 0, 200, 17, 128, 129], 0, 1.0, 3),
    ("bf16", 32, 8, 128, 16, [1000, 1, 127, 0, 513], 0, 0.9, 0),
    ("bf16", 12, 4, 128, 8, [1500, 300, 1], 256, 1.0, 1),          # split, a group of 3
    ("fp16", 16, 1, 64, 128, [700, 129, 5], 128, 0.5, 7),          # split at head size 64
    ("fp16", 32, 1, 128, 32, [385, 384, 383], 0, 1.0, 0),          # the largest group
    ("bf16", 34, 2, 64, 64, [90, 700], 0, 0.0, 2),                 # a group of 17
    ("fp16", 5, 5, 128, 16, [33], 0, 0.0, 5),
    ("bf16", 14, 2, 64, 8, [4097, 2049, 3], 0, 1.0, 1),            # a group of 7
])
def test_decode_weights(cuda_device, dtype, hq, hkv, D, B, lens, part, decay, slack):
    S = len(lens)
    case = W.make_decode_case(hq + B, S, hq, hkv, D, B, dtype, lens, pool_factor=1.4, poison=True,
                              device=cuda_device)
    weights = _old_weights(S, hkv, case.max_context_len + slack, 5)
    if decay == 0.0:
        weights.fill_(float("nan"))                 # overwritten unread
    old = weights.clone()
    out = torch.full_like(case.q, float("nan"))
    # whatever the workspace held before
    ws = torch.full((pkv.decode_weights_workspace_size(S, hq, hkv, D, case.max_context_len, part)
                     // 4,), float("nan"), device="cuda")
    res = pkv.paged_attn_decode_weights(out, weights, case.q, case.k_cache, case.v_cache,
                                        case.block_tables, case.context_lens, case.scale,
                                        case.max_context_len, decay=decay, partition_size=part,
                                        workspace=ws)
    assert res is out
    assert_within_tol(out, oracle_decode(case), case.q.dtype, "out")
    _check_weights(weights, old, case, case.q, [1] * S, decay)
    # the attention is the plain call's, bit for bit, where that runs the same kernel and split
    if pkv.decode_uses_tensor_cores(S, hq, hkv, D, case.max_context_len, part):
        ref = pkv.paged_attn_decode(torch.empty_like(out), case.q, case.k_cache, case.v_cache,
                                    case.block_tables, case.context_lens, case.scale,
                                    case.max_context_len, partition_size=part)
        assert torch.equal(out, ref)


def test_decode_weights_loose_bound_and_bad_inputs(cuda_device):
    """A bound far above every context, a context beyond it, a bad block id."""
    case = W.make_decode_case(3, 3, 8, 2, 64, 16, "fp16", [40, 0, 9], pool_factor=2.0, poison=True,
                              max_blocks_per_seq=200, device=cuda_device)
    weights = _old_weights(3, 2, 3200, 6)
    old, out = weights.clone(), torch.empty_like(case.q)
    args = (case.q, case.k_cache, case.v_cache, case.block_tables, case.context_lens, case.scale)
    pkv.paged_attn_decode_weights(out, weights, *args, 3200)
    assert_within_tol(out, oracle_decode(case), case.q.dtype, "out")
    _check_weights(weights, old, case, case.q, [1] * 3, 1.0)
    for bad in (weights[:, :, :100], weights[:2], weights.double()):
        with pytest.raises(ValueError):
            pkv.paged_attn_decode_weights(out, bad.contiguous(), *args, 3200)
    with pytest.raises(ValueError):
        pkv.paged_attn_decode_weights(out, weights, *args, 3200, partition_size=96)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_attn_decode_weights(out, weights, *args, 3200,
                                      workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    # the bound cuts the longest context short
    case.context_lens[0] = 60
    pkv.paged_attn_decode_weights(out, weights, *args, 40)
    assert pkv.device_status(clear=True) == _lib.DEV_BAD_CONTEXT_LEN
    assert torch.equal(weights[0, :, 40:], old[0, :, 40:])
    case.context_lens[0] = 40
    case.block_tables[0, 1] = case.num_blocks
    pkv.paged_attn_decode_weights(out, weights, *args, 3200)
    assert pkv.device_status(clear=True) == _lib.DEV_BAD_BLOCK_ID


def _chunk_case(seed, dtype, hq, hkv, D, B, lens, chunks, device, pad_rows=0):
    case = W.make_decode_case(seed, len(lens), hq, hkv, D, B, dtype, lens, pool_factor=1.3,
                              poison=True, device=device)
    total = int(sum(chunks))
    q = _randn((total + pad_rows, hq, D), seed + 1, case.q.dtype)
    q[total:] = float("nan")                       # rows behind the last sequence
    start = torch.tensor(np.concatenate([[0], np.cumsum(chunks)]), dtype=torch.int32, device=device)
    return case, q, start


@pytest.mark.parametrize("dtype,hq,hkv,D,B,lens,chunks,window,decay,pad", [
    ("fp16", 8, 8, 64, 16, [1, 40, 200], [1, 40, 7], 0, 1.0, 0),
    ("bf16", 32, 8, 128, 16, [300, 129, 64], [200, 1, 64], 0, 1.0, 5),
    ("fp16", 12, 4, 128, 8, [150, 260, 31], [150, 0, 3], 0, 0.5, 2),      # a group of 3; no queries
    ("bf16", 8, 2, 64, 32, [500, 130], [131, 130], 16, 1.0, 1),           # only the last 16 count
    ("bf16", 40, 40, 128, 16, [97, 140], [97, 140], 32, 0.0, 0),
    ("fp16", 128, 1, 64, 64, [140, 20], [20, 3], 0, 1.0, 0),              # one query per tile
    ("bf16", 66, 2, 128, 128, [300, 1], [5, 1], 1, 0.9, 3),               # a group of 33
    ("fp16", 5, 1, 64, 16, [700], [513], 100, 1.0, 4),
])
def test_prefill_weights(cuda_device, dtype, hq, hkv, D, B, lens, chunks, window, decay, pad):
    case, q, start = _chunk_case(D + B, dtype, hq, hkv, D, B, lens, chunks, cuda_device, pad)
    S, total = len(lens), int(sum(chunks))
    weights = _old_weights(S, hkv, case.max_context_len + 2, 9)
    if decay == 0.0:
        weights.fill_(float("nan"))
    old = weights.clone()
    out = torch.full_like(q, 3.0)
    args = (q, start, case.k_cache, case.v_cache, case.block_tables, case.context_lens, case.scale,
            case.max_context_len, max(chunks))
    pkv.paged_attn_prefill_weights(out, weights, *args, window=window, decay=decay,
                                   workspace=torch.full((q.shape[0] * hq,), float("nan"),
                                                        device="cuda"))
    plain = torch.full_like(q, 3.0)
    pkv.paged_attn_prefill(plain, *args)
    assert torch.equal(out, plain)                  # the same attention, bit for bit
    assert (out[total:] == 3.0).all()               # rows behind the last sequence as they were
    _check_weights(weights, old, case, q[:total], chunks, decay, window)
    again = old.clone()
    pkv.paged_attn_prefill_weights(out, again, *args, window=window, decay=decay)
    assert torch.equal(again, weights) or decay == 0.0 and torch.equal(
        torch.nan_to_num(again), torch.nan_to_num(weights))


def test_prefill_weights_agree_with_decode(cuda_device):
    """One query per sequence: the chunk call and the decode call."""
    lens = [700, 1, 129, 64]
    case, q, start = _chunk_case(5, "bf16", 16, 4, 128, 16, lens, [1] * 4, cuda_device)
    a, b = (torch.zeros((4, 4, 700), device="cuda") for _ in range(2))
    pkv.paged_attn_prefill_weights(torch.empty_like(q), a, q, start, case.k_cache, case.v_cache,
                                   case.block_tables, case.context_lens, case.scale, 700, 1)
    pkv.paged_attn_decode_weights(torch.empty_like(q), b, q, case.k_cache, case.v_cache,
                                  case.block_tables, case.context_lens, case.scale, 700)
    _check_weights(a, torch.zeros_like(a), case, q, [1] * 4, 1.0)
    _check_weights(b, torch.zeros_like(b), case, q, [1] * 4, 1.0)
    assert torch.allclose(a.sum(-1), torch.full((4, 4), 4.0, device="cuda"), rtol=1e-4)


def test_prefill_weights_neighbour_nan(cuda_device):
    """NaN queries of another sequence and of another group's heads, which
    share MMA tiles with a group of 3, stay out of a sequence's weights."""
    lens, chunks = [90, 50], [30, 20]
    case, q, start = _chunk_case(11, "fp16", 6, 2, 64, 16, lens, chunks, cuda_device)
    q[:30, 3:] = float("nan")                       # sequence 0: KV head 1's queries
    q[30:] = float("nan")                           # sequence 1: all of them
    weights = torch.zeros((2, 2, 90), device="cuda")
    pkv.paged_attn_prefill_weights(torch.empty_like(q), weights, q, start, case.k_cache,
                                   case.v_cache, case.block_tables, case.context_lens, case.scale,
                                   90, 30)
    w = oracle.attention_weights(np.nan_to_num(to_f64(q[:30])), to_f64(case.k_cache),
                                 case.block_tables[0].cpu().numpy(), 90, case.scale)[0]
    bound = _weights_bound(torch.nan_to_num(q), case.k_cache, w, case.scale, 64)
    assert (np.abs(to_f64(weights)[0, 0] - w) <= bound + 2.0 ** -23 * w).all()
    assert torch.isnan(weights[0, 1]).all() and torch.isnan(weights[1, :, :50]).all()
    assert (weights[1, :, 50:] == 0).all()


# ---- choice --------------------------------------------------------------------------------------


def _check_select(weights, lens, budget, recent, sinks, max_ctx=None):
    S, H, width = weights.shape
    keep = torch.full((S, H, budget), -5, dtype=torch.int32, device="cuda")
    new = torch.full((S,), -5, dtype=torch.int32, device="cuda")
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    before = weights.clone()
    pkv.kv_evict_select(keep, weights, lens_t, width if max_ctx is None else max_ctx, recent=recent,
                        sinks=sinks, new_lens=new)
    assert new.tolist() == [min(n, budget) for n in lens]
    assert torch.equal(weights.view(torch.int32), before.view(torch.int32))
    w, k = weights.cpu().numpy(), keep.cpu().numpy()
    for s in range(S):
        for h in range(H):
            ref = oracle.evict_select(w[s, h], lens[s], budget, recent, sinks)
            assert k[s, h].tolist() == ref + [-1] * (budget - len(ref)), (s, h)


@pytest.mark.parametrize("lens,H,budget,recent,sinks,slack", [
    ([1, 0, 5, 64, 65], 2, 64, 16, 4, 0),
    ([2, 3], 1, 1, 0, 0, 1),
    ([2, 3, 100], 3, 1, 1, 0, 5),
    ([100, 33], 2, 7, 0, 7, 0),
    ([4097, 2000, 9000], 2, 1025, 100, 3, 2),
    ([20000], 5, 19999, 0, 0, 3),
    ([1030] * 3, 4, 1029, 1000, 0, 0),
])
@pytest.mark.parametrize("kind", ["heavy", "ties", "special", "negative"])
def test_select(cuda_device, lens, H, budget, recent, sinks, slack, kind):
    width = max(lens) + slack
    g = _gen(budget)
    w = torch.exp(3 * torch.randn((len(lens), H, width), generator=g, device="cuda"))
    if kind == "ties":
        w = torch.randint(0, 3, w.shape, generator=g, device="cuda").float()
    elif kind == "special":
        pick = torch.randint(0, 8, w.shape, generator=g, device="cuda")
        for i, x in enumerate((float("nan"), float("inf"), float("-inf"), 0.0, -0.0)):
            w[pick == i] = x
    elif kind == "negative":
        w = torch.log(w)
    _check_select(w, lens, budget, recent, sinks)


def test_select_long_row(cuda_device):
    w = torch.exp(2 * torch.randn((1, 2, 200001), generator=_gen(1), device="cuda"))
    w[0, 1] = 0.25                                   # all equal: the lowest positions
    _check_select(w, [200001], 70000, 1000, 4)


def test_select_row_longer_than_shared_memory(cuda_device):
    w = torch.exp(2 * torch.randn((1, 1, 420000), generator=_gen(2), device="cuda"))
    _check_select(w, [419999], 100000, 7, 0)


@pytest.mark.parametrize("S,H,n", [
    (1, 1, 780000),      # 16 CTAs a row, each with close to all of an SM's shared memory
    (1, 2, 1000003),     # 16 CTAs a row, keys read again in every pass
    (40, 8, 60001),      # one CTA a row, keys read again
])
def test_select_keys_per_cta(cuda_device, S, H, n):
    """Shares of a row up to and beyond what a CTA holds in shared memory."""
    w = torch.exp(2 * torch.randn((S, H, n + 1), generator=_gen(n), device="cuda"))
    w[0, 0, ::3] = 1.5                               # ties on both sides of the CTAs' bounds
    _check_select(w, [n] + [max(1, n - 977 * s) for s in range(1, S)], n // 3, 500, 4)


@pytest.mark.parametrize("S,H", [(1, 3), (20, 8), (40, 8), (90, 8)])
def test_select_rows_per_launch(cuda_device, S, H):
    """Every number of CTAs per row, sequences below and above the budget."""
    lens = [(700 + 613 * s) % 9000 + 1 for s in range(S)]
    w = torch.rand((S, H, 9001), generator=_gen(S), device="cuda")
    _check_select(w, lens, 1200, 64, 2)


def test_select_refuses_and_flags(cuda_device):
    w = torch.rand((2, 2, 50), device="cuda")
    keep = torch.empty((2, 2, 10), dtype=torch.int32, device="cuda")
    lens = torch.tensor([50, 70], dtype=torch.int32, device="cuda")
    for bad in (dict(keep=keep.long()), dict(weights=w.half()), dict(lens=lens.long()),
                dict(keep=keep[:1]), dict(new_lens=lens[:1]), dict(max_ctx=51)):
        with pytest.raises(ValueError):
            pkv.kv_evict_select(bad.get("keep", keep), bad.get("weights", w), bad.get("lens", lens),
                                bad.get("max_ctx", 50), new_lens=bad.get("new_lens"))
    for bad in (dict(recent=11), dict(sinks=-1), dict(new_lens=lens)):
        with pytest.raises(pkv.PagedKVError):
            pkv.kv_evict_select(keep, w, lens, 50, **bad)
    pkv.kv_evict_select(keep, w, lens, 50)           # 70 > 50: taken as 50
    assert pkv.device_status(clear=True) == _lib.DEV_BAD_CONTEXT_LEN
    ref = oracle.evict_select(w[1, 0].cpu().numpy(), 50, 10, 0, 0)
    assert keep[1, 0].tolist() == ref


# ---- compaction ----------------------------------------------------------------------------------


def _keep_of(lens, H, budget, seed):
    rng = np.random.default_rng(seed)
    keep = np.full((len(lens), H, budget), -1, dtype=np.int32)
    for s, n in enumerate(lens):
        for h in range(H):
            m = min(n, budget)
            keep[s, h, :m] = np.sort(rng.permutation(n)[:m])
    return keep


@pytest.mark.parametrize("dtype,H,D,B,lens,budget,fresh,weighted", [
    ("fp16", 2, 64, 16, [100, 30, 0, 1], 40, False, True),
    ("bf16", 8, 128, 16, [1000, 513, 512], 512, False, True),
    ("fp16", 3, 128, 8, [300, 77], 33, True, True),
    ("bf16", 1, 64, 128, [2000], 1999, False, False),
    ("fp16", 5, 64, 32, [65, 64, 63], 1, False, True),
    ("bf16", 2, 128, 64, [3000, 129], 1500, True, False),
])
def test_compact(cuda_device, dtype, H, D, B, lens, budget, fresh, weighted):
    case = W.make_decode_case(D + B, len(lens), H, H, D, B, dtype, lens, pool_factor=2.5,
                              pool_blocks=None, poison=True, device=cuda_device)
    S = len(lens)
    keep = _keep_of(lens, H, budget, 4)
    src = case.block_tables.cpu().numpy()
    dst = src.copy()
    if fresh:                                        # every second kept block is another one
        used = set(src[src >= 0].tolist())
        free = [b for b in range(case.num_blocks) if b not in used]
        for s in range(S):
            for i in range(0, -(-min(lens[s], budget) // B), 2):
                dst[s, i] = free.pop()
    dst = np.ascontiguousarray(dst[:, :max(1, -(-min(budget, max(lens)) // B))])
    weights = _old_weights(S, H, max(lens) + 3, 2) if weighted else None
    k0, v0 = raw_bytes(case.k_cache), raw_bytes(case.v_cache)
    shape = case.k_cache.shape
    w0 = to_f64(weights) if weighted else None
    pkv.kv_compact(case.k_cache, case.v_cache, case.block_tables,
                   torch.from_numpy(keep).to(cuda_device), case.context_lens, weights=weights,
                   dst_tables=torch.from_numpy(dst).to(cuda_device) if fresh or budget < max(lens)
                   else None, max_context_len=max(lens))
    for cache, was in ((case.k_cache, k0), (case.v_cache, v0)):
        ref = oracle.compact(was.reshape(shape), src, dst, keep, lens)
        assert np.array_equal(raw_bytes(cache).reshape(shape), ref)
    if weighted:
        assert np.array_equal(to_f64(weights), oracle.compact_weights(w0, keep, lens))


def test_compact_refuses_and_flags(cuda_device):
    case = W.make_decode_case(2, 2, 2, 2, 64, 16, "fp16", [60, 40], pool_factor=2.0,
                              device=cuda_device)
    keep = torch.from_numpy(_keep_of([60, 40], 2, 16, 1)).cuda()
    args = (case.k_cache, case.v_cache, case.block_tables)
    for bad in ((keep.long(), case.context_lens), (keep[:1], case.context_lens),
                (keep[:, :1].contiguous(), case.context_lens), (keep, case.context_lens[:1])):
        with pytest.raises(ValueError):
            pkv.kv_compact(*args, *bad)
    with pytest.raises(ValueError):
        pkv.kv_compact(*args, keep, case.context_lens, weights=torch.zeros((2, 2, 50), device="cuda"),
                       max_context_len=60)
    with pytest.raises(pkv.PagedKVError):            # two blocks for 33 rows
        pkv.kv_compact(*args, torch.zeros((2, 2, 33), dtype=torch.int32, device="cuda"),
                       case.context_lens, dst_tables=case.block_tables[:, :2].contiguous())
    k0 = to_f64(case.k_cache)
    src = case.block_tables.cpu().numpy()
    for entry, flag in ((3, 64), (5, 2), (4, -1)):   # beyond the sequence; below its index
        was = int(keep[0, 1, entry])
        keep[0, 1, entry] = flag
        fresh = [t.clone() for t in (case.k_cache, case.v_cache)]
        pkv.kv_compact(*fresh, case.block_tables, keep, case.context_lens)
        assert pkv.device_status(clear=True) == _lib.DEV_BAD_KEEP
        good = keep.cpu().numpy().copy()
        good[0, 1, entry] = entry                    # skipped: the row stays
        assert np.array_equal(to_f64(fresh[0]), oracle.compact(k0, src, src, good, [60, 40]))
        keep[0, 1, entry] = was
    tables = case.block_tables.clone()
    tables[1, 2] = -1                                # positions 32 .. 39 of sequence 1
    fresh = [t.clone() for t in (case.k_cache, case.v_cache)]
    pkv.kv_compact(*fresh, tables, keep, case.context_lens)
    assert pkv.device_status(clear=True) == _lib.DEV_BAD_BLOCK_ID
    with pytest.raises(ValueError):
        pkv.kv_compact(*fresh, tables, keep, case.context_lens.cpu())


def test_offsets_beyond_32_bits(cuda_device):
    """Blocks whose rows lie past 2^32 elements into the caches."""
    H, B, D = 8, 128, 128
    NB = (1 << 32) // (H * B * D) + 8
    kc, vc = (torch.empty((NB, H, B, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    T = 300
    table = torch.tensor([[NB - 1, 0, NB - 3]], dtype=torch.int32, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = table[0].long()[pos.long() // B] * B + pos.long() % B
    q, k, v = (_randn((T, H, D), i, torch.bfloat16) for i in range(3))
    freq = pkv.rope_frequencies(D)
    qr = pkv.rope_kv_append(torch.empty_like(q), q, k, v, pos, freq, kc, vc, slots)
    k_rows = kc[table[0].long()].transpose(1, 2).reshape(-1, H, D)[:T]
    _check_rotated(k_rows, to_f64(k), pos.cpu().numpy(), freq.cpu().numpy(), False, 1.0,
                   torch.bfloat16)
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    small = W.DecodeCase(q=qr[-1:].contiguous(), k_cache=kc[table[0].long()],
                         v_cache=vc[table[0].long()],
                         block_tables=torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"),
                         context_lens=lens, scale=D ** -0.5, block_size=B, max_context_len=T)
    weights = torch.zeros((1, H, T), device="cuda")
    out = torch.empty_like(small.q)
    pkv.paged_attn_decode_weights(out, weights, small.q, kc, vc, table, lens, small.scale, T)
    assert_within_tol(out, oracle_decode(small), torch.bfloat16, "decode")
    _check_weights(weights, torch.zeros_like(weights), small, small.q, [1], 1.0)
    both = torch.zeros_like(weights)
    start = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    tail = qr[-40:].contiguous()
    pkv.paged_attn_prefill_weights(torch.empty_like(tail), both, tail, start, kc, vc, table, lens,
                                   small.scale, T, 40)
    _check_weights(both, torch.zeros_like(both), small, tail, [40], 1.0)
    keep = pkv.kv_evict_select(torch.empty((1, H, 200), dtype=torch.int32, device="cuda"), weights,
                               lens, T, recent=10)
    kept = keep[0].long()                            # [H, 200]
    want = torch.stack([k_rows[kept[h], h] for h in range(H)])
    want_v = torch.stack([v[kept[h], h] for h in range(H)])
    pkv.kv_compact(kc, vc, table, keep, lens)
    for cache, ref in ((kc, want), (vc, want_v)):
        got = cache[table[0, :2].long()].transpose(0, 1).reshape(H, -1, D)[:, :200]
        assert torch.equal(got, ref)


# ---- the operators together ----------------------------------------------------------------------


@pytest.mark.parametrize("dtype,hq,hkv,D,B", [("bf16", 16, 4, 128, 16), ("fp16", 6, 6, 64, 8)])
def test_a_run_that_evicts(cuda_device, dtype, hq, hkv, D, B):
    """Prompts of forked samples, decode steps, and an eviction whenever the
    longest sequence passes its budget, against the oracle replaying it: rows
    rotated at their positions, shared blocks left to their other owners."""
    dt = W.DTYPES[dtype]
    budget, recent, sinks, high = 48, 8, 2, 60
    prompt, steps, width = [55, 31], 24, 80
    alloc = pkv.BlockAllocator(60, B)
    kc, vc = (torch.full((60, hkv, B, D), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    freq = pkv.rope_frequencies(D, scaling="linear", factor=2.0)
    f64 = freq.cpu().numpy()
    scale = D ** -0.5
    mbs = -(-width // B)
    gpu = lambda x, t: torch.from_numpy(np.ascontiguousarray(x)).to(cuda_device, t)  # noqa: E731

    # prompts
    seed = 100
    q, k, v = (_randn((sum(prompt), n, D), seed + n, dt) for n in (hq, hkv, hkv + 1))
    v = v[:, :hkv]
    for s, n in enumerate(prompt):
        alloc.add_seq(s, n)
    slots = np.concatenate([alloc.seq_slots(s, 0, n) for s, n in enumerate(prompt)])
    pos = np.concatenate([np.arange(n) for n in prompt])
    qr = pkv.rope_kv_append(torch.empty_like(q), q, k, v, gpu(pos, torch.int32), freq, kc, vc,
                            gpu(slots, torch.int64))
    tables = alloc.block_table([0, 1], mbs)
    start = gpu(np.concatenate([[0], np.cumsum(prompt)]), torch.int32)
    w2 = torch.zeros((2, hkv, width), device="cuda")
    out = torch.empty_like(qr)
    pkv.paged_attn_prefill_weights(out, w2, qr, start, kc, vc, gpu(tables, torch.int32),
                                   gpu(prompt, torch.int32), scale, width, max(prompt), window=20)
    assert torch.isfinite(out).all()
    k64, v64 = to_f64(kc), to_f64(vc)
    for s in range(2):
        ref = oracle.attention_weights(to_f64(qr)[start[s]:start[s + 1]], k64, tables[s], prompt[s],
                                       scale, 20)
        assert np.allclose(to_f64(w2)[s, :, :prompt[s]], ref, rtol=2e-4, atol=1e-7)

    # four samples: two of each prompt, sharing its blocks
    alloc.fork(0, 2)
    alloc.fork(1, 3)
    ids = [0, 1, 2, 3]
    weights = w2[[0, 1, 0, 1]].contiguous()
    lens = np.array([prompt[0], prompt[1]] * 2)
    seen = lens.copy()                               # positions go on counting
    evictions = 0
    for step in range(steps):
        if lens.max() + 1 > high:
            tables = alloc.block_table(ids, mbs)
            keep = torch.empty((4, hkv, budget), dtype=torch.int32, device="cuda")
            new = torch.empty(4, dtype=torch.int32, device="cuda")
            lens_t = gpu(lens, torch.int32)
            pkv.kv_evict_select(keep, weights, lens_t, width, recent=recent, sinks=sinks, new_lens=new)
            w_np, k_np = weights.cpu().numpy(), keep.cpu().numpy()
            for s in range(4):
                for h in range(hkv):
                    ref = oracle.evict_select(w_np[s, h], int(lens[s]), budget, recent, sinks)
                    assert k_np[s, h, :len(ref)].tolist() == ref
            after = np.minimum(lens, budget)
            alloc.shrink_seqs(ids, after)
            dst = alloc.block_table(ids, mbs)
            k_old, v_old = to_f64(kc), to_f64(vc)
            w_old = to_f64(weights)
            pkv.kv_compact(kc, vc, gpu(tables, torch.int32), keep, lens_t, weights=weights,
                           dst_tables=gpu(dst, torch.int32), max_context_len=width)
            assert np.array_equal(to_f64(kc), oracle.compact(k_old, tables, dst, k_np, lens),
                                  equal_nan=True)
            assert np.array_equal(to_f64(vc), oracle.compact(v_old, tables, dst, k_np, lens),
                                  equal_nan=True)
            assert np.array_equal(to_f64(weights), oracle.compact_weights(w_old, k_np, lens))
            assert new.tolist() == after.tolist()
            lens = after
            evictions += 1
        slots, pairs = alloc.append_slots(ids)
        if len(pairs):
            pkv.block_copy(kc, vc, gpu(pairs, torch.int64))
        tables = alloc.block_table(ids, mbs)
        q, k, v = (_randn((4, n, D), seed + 7 * step + i, dt) for i, n in enumerate((hq, hkv, hkv)))
        k64, v64 = to_f64(kc), to_f64(vc)
        qr = pkv.rope_kv_append(torch.empty_like(q), q, k, v, gpu(seen, torch.int32), freq, kc, vc,
                                gpu(slots, torch.int64))
        lens, seen = lens + 1, seen + 1
        _check_rotated(qr, to_f64(q), seen - 1, f64, False, 1.0, dt)
        out = torch.empty_like(qr)
        old = weights.clone()
        pkv.paged_attn_decode_weights(out, weights, qr, kc, vc, gpu(tables, torch.int32),
                                      gpu(lens, torch.int32), scale, width, decay=0.95)
        case = W.DecodeCase(q=qr, k_cache=kc, v_cache=vc, block_tables=gpu(tables, torch.int32),
                            context_lens=gpu(lens, torch.int32), scale=scale, block_size=B,
                            max_context_len=width)
        assert_within_tol(out, oracle_decode(case), dt, f"step {step}")
        _check_weights(weights, old, case, qr, [1] * 4, 0.95)
    assert evictions >= 2
    for s in ids:
        alloc.free_seq(s)
    assert alloc.stats()["free_blocks"] == 60


def test_arguments_beyond_32_bits(cuda_device):
    """Not cut down to their low bits: 2**32 recent positions are not none."""
    big = 2**32
    keep = torch.zeros((1, 2, 4), dtype=torch.int32, device="cuda")
    w = torch.ones((1, 2, 64), device="cuda")
    lens = torch.tensor([40], dtype=torch.int32, device="cuda")
    kc = torch.zeros((4, 2, 16, 64), dtype=torch.float16, device="cuda")
    q = torch.zeros((1, 2, 64), dtype=torch.float16, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for call in (
            lambda: pkv.kv_evict_select(keep, w, lens, 64, recent=big),
            lambda: pkv.kv_evict_select(keep, w, lens, 64, sinks=-big),
            lambda: pkv.kv_compact(kc, kc.clone(), table, keep, lens, max_context_len=big + 64),
            lambda: pkv.paged_attn_decode_weights(torch.empty_like(q), w, q, kc, kc, table, lens,
                                                  0.1, 64, partition_size=big),
            lambda: pkv.paged_attn_prefill_weights(torch.empty_like(q), w, q, start, kc, kc,
                                                   table, lens, 0.1, 64, 1, window=-big),
            lambda: pkv.paged_attn_prefill_weights(torch.empty_like(q), w, q, start, kc, kc,
                                                   table, lens, 0.1, 64, big)):
        with pytest.raises(ValueError):
            call()


def test_two_calls_at_once(cuda_device):
    """The same operators on two streams at a time, each with its own batch."""
    cases = [W.make_decode_case(20 + i, 6, 16, 4, 128, 16, "bf16", [2000, 1, 700, 129, 0, 1500],
                                pool_factor=1.1, device=cuda_device) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(c.q) for c in cases]
    weights = [_old_weights(6, 4, 2000, i) for i in range(2)]
    olds = [w.clone() for w in weights]
    keeps = [torch.empty((6, 4, 300), dtype=torch.int32, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s, o, w, old, k in zip(cases, streams, outs, weights, olds, keeps):
            with torch.cuda.stream(s):
                w.copy_(old)
                pkv.paged_attn_decode_weights(o, w, c.q, c.k_cache, c.v_cache, c.block_tables,
                                              c.context_lens, c.scale, 2000)
                pkv.kv_evict_select(k, w, c.context_lens, 2000, recent=20, sinks=1)
    torch.cuda.synchronize()
    for c, o, w, old, k in zip(cases, outs, weights, olds, keeps):
        assert_within_tol(o, oracle_decode(c), c.q.dtype, "out")
        _check_weights(w, old, c, c.q, [1] * 6, 1.0)
        w_np, k_np = w.cpu().numpy(), k.cpu().numpy()
        for s, n in enumerate(c.context_lens.tolist()):
            for h in range(4):
                ref = oracle.evict_select(w_np[s, h], n, 300, 20, 1)
                assert k_np[s, h].tolist() == ref + [-1] * (300 - len(ref))


def test_chain_captured_on_another_stream(cuda_device):
    """rope -> decode with weights -> select -> compact in one graph, replayed
    with new inputs, against the same calls made eagerly; two graphs share one
    workspace."""
    lens0, budget = [300, 129, 40], 128
    case = W.make_decode_case(8, 3, 16, 4, 128, 16, "bf16", lens0, pool_factor=1.2,
                              device=cuda_device)
    ws = torch.empty(pkv.decode_weights_workspace_size(3, 16, 4, 128, 300), dtype=torch.uint8,
                     device="cuda")
    q, k, v = (_randn((3, n, 128), n, torch.bfloat16) for n in (16, 4, 5))
    v = v[:, :4].contiguous()
    freq = pkv.rope_frequencies(128)
    pos = torch.tensor([1000, 2000, 3000], dtype=torch.int32, device="cuda")
    slots = W.last_position_slots(case).to(cuda_device)
    kc0, vc0 = case.k_cache.clone(), case.v_cache.clone()
    weights = _old_weights(3, 4, 300, 3)
    w0 = weights.clone()
    keep = torch.empty((3, 4, budget), dtype=torch.int32, device="cuda")
    qr, out = torch.empty_like(q), torch.empty_like(q)

    def chain():
        pkv.rope_kv_append(qr, q, k, v, pos, freq, case.k_cache, case.v_cache, slots)
        pkv.paged_attn_decode_weights(out, weights, qr, case.k_cache, case.v_cache,
                                      case.block_tables, case.context_lens, case.scale, 300,
                                      workspace=ws)
        pkv.kv_evict_select(keep, weights, case.context_lens, 300, recent=16)
        pkv.kv_compact(case.k_cache, case.v_cache, case.block_tables, keep, case.context_lens,
                       weights=weights, max_context_len=300)

    def reset():
        case.k_cache.copy_(kc0)
        case.v_cache.copy_(vc0)
        weights.copy_(w0)

    def result():
        torch.cuda.synchronize()
        return [t.clone() for t in (out, weights, keep, case.k_cache, case.v_cache)]

    stream = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(stream):
        chain()
        stream.synchronize()
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                chain()
            graphs.append(g)
    for seed in (1, 2):
        q.copy_(_randn(q.shape, 50 + seed, q.dtype))
        reset()
        chain()
        want = result()
        for g in graphs:
            reset()
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                g.replay()
            for a, b in zip(result(), want):
                assert torch.equal(a.view(torch.int16 if a.dtype != torch.int32 else a.dtype),
                                   b.view(torch.int16 if b.dtype != torch.int32 else b.dtype))
