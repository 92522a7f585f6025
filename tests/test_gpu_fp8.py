"""The cache held in 8 bits on the GPU against the fp64 oracle.

Tolerances.  Codes, scales and the bf16 values read back are exact; fp16 read
back is the one rounding of an exact product.  A normalised and turned element:
the root mean square within 2^-21 relative (an fp32 sum of D squares, rsqrtf
within 2 ulp, three products), the turn within 2^-21 (|first| + |second|) of
its pair as for rope_kv_append, and one rounding to the type (eps / 2); so
eps / 2 |y| + 2^-20 (|first| + |second|).

Attention: out = sum_t p_t v_t.  A logit is an fp32 sum of D products of exact
numbers, off by at most dx = (D / 16 + 8) 2^-23 of the sum a of their magnitudes,
and the running maximum cancels, so each weight is off by 2 dx relative (its own
logit and the sum's), by 2^-17 for the exponential and the fp32 sums, and by
2^-11 for the rounding of the products' left factor to 11 bits or more; weights
below 2^-23 of the largest may be lost, 2^-23 of the largest |v| for each
position.  The result is rounded once (eps / 2).  Together
  |err| <= eps / 2 |out| + (2 dx + 2^-17 + 2^-11) sum_t p_t |v_t| + n 2^-23 max |v|.
"""

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_247_gb300 as pkv
from paged_kv_cache_247_gb300 import _lib
from paged_kv_cache_247_gb300 import workloads as W
from _gpu_util import to_f64

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _clean_status(lib, cuda_device):
    pkv.device_status(clear=True)
    yield
    assert pkv.device_status(clear=True) == 0


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, seed, dtype):
    x = torch.randn(shape, generator=_gen(seed), device="cuda")
    return (x * torch.exp(torch.randn(shape[:-1] + (1,), generator=_gen(seed + 99), device="cuda"))).to(dtype)


def _codes(t):
    return t.cpu().view(torch.uint8).numpy()


def _empty_cache(NB, H, B, D, fill=0):
    k = torch.full((NB, H, B, D), fill, dtype=torch.uint8, device="cuda").view(E4M3)
    s = torch.full((NB, H, B, 1), 0.5, dtype=torch.bfloat16, device="cuda")
    return k, k.clone(), s, s.clone()


# ---- append and read back ----------------------------------------------------------------------


def _special_rows(dtype, D):
    """Rows at the borders of the scale and of the codes."""
    tiny = 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -133
    big = torch.finfo(dtype).max
    x = torch.zeros((14, D), dtype=torch.float64)
    x[1, 0], x[2, 1], x[3, 2] = tiny, big, -big
    x[4, :4] = torch.tensor([448.0, 3.0625, -432.0, 2.0 ** -7])
    x[5, :3] = torch.tensor([450.0, 416.0, -2.0 ** -10])     # above 448 (rounds down in fp16, not in bf16)
    x[6, 0], x[7, D - 1], x[8, 5] = float("nan"), float("inf"), float("-inf")
    x[9] = torch.linspace(-448, 448, D).double()
    x[10, :2] = torch.tensor([224.0, -225.0])
    x[11] = 2.0 ** -14
    x[12, 0], x[12, 1:] = 256.0, 17 * 2.0 ** -4             # ties of the codes: 17/16
    x[13] = -0.0
    return x.to(dtype).cuda()


@pytest.mark.parametrize("dtype,H,D,B,T,packed", [
    ("bf16", 8, 128, 16, 1, False), ("fp16", 1, 64, 8, 1, True), ("bf16", 5, 64, 32, 37, True),
    ("fp16", 40, 128, 16, 65, False), ("bf16", 1, 128, 128, 300, True), ("fp16", 3, 64, 64, 1000, False),
    ("bf16", 12, 128, 8, 513, True),
])
def test_append(cuda_device, dtype, H, D, B, T, packed):
    dt = W.DTYPES[dtype]
    rng = np.random.default_rng(T)
    if packed:
        qkv = _randn((T, 3 * H, D), 3, dt)
        k, v = qkv[:, H:2 * H], qkv[:, 2 * H:]
    else:
        k, v = _randn((T, H, D), 4, dt), _randn((T, H, D), 5, dt)
    special = _special_rows(dt, D)
    flat = min(T * H, len(special))
    rows = torch.arange(flat, device="cuda")
    k[rows // H, rows % H] = special[:flat]
    v[rows // H, rows % H] = special.flip(0)[:flat]
    NB = -(-T // B) + 2
    kc, vc, ks, vs = _empty_cache(NB, H, B, D, fill=0x31)
    slots = rng.permutation(NB * B)[:T].astype(np.int64)
    if T > 2:
        slots[1], slots[T - 1] = -1, -9
    pkv.kv_append_fp8(k, v, kc, vc, ks, vs, torch.from_numpy(slots).cuda())
    there = slots >= 0
    blk, off = slots[there] // B, slots[there] % B
    for x, cache, scales in ((k, kc, ks), (v, vc, vs)):
        codes, s = oracle.quantise(to_f64(x)[there])
        want_c = np.full((NB, H, B, D), 0x31, dtype=np.uint8)
        want_s = np.full((NB, H, B, 1), 0.5)
        want_c[blk, :, off], want_s[blk, :, off, 0] = codes, s
        assert np.array_equal(_codes(cache), want_c)
        assert np.array_equal(to_f64(scales), want_s, equal_nan=True)


def test_append_bad_slot(cuda_device):
    k = _randn((4, 2, 64), 1, torch.float16)
    kc, vc, ks, vs = _empty_cache(2, 2, 8, 64)
    pkv.kv_append_fp8(k, k, kc, vc, ks, vs, torch.tensor([3, 16, 1 << 40, -1], device="cuda"))
    assert pkv.device_status(clear=True) == _lib.DEV_BAD_SLOT
    changed = (ks != 0.5).squeeze(-1).any(1)
    assert changed.sum() == 1 and changed[0, 3] and not (vs[1] != 0.5).any()


@pytest.mark.parametrize("dtype,H,D,B,P", [
    ("bf16", 8, 128, 16, 7), ("fp16", 1, 64, 8, 1), ("fp16", 5, 128, 128, 3), ("bf16", 3, 64, 32, 129)])
def test_read_back(cuda_device, dtype, H, D, B, P):
    dt = W.DTYPES[dtype]
    rng = np.random.default_rng(P)
    NB, NO = P + 3, P + 2
    kc, vc, ks, vs = _empty_cache(NB, H, B, D)
    for seed, c, s in ((1, kc, ks), (2, vc, vs)):
        c.view(torch.uint8).copy_(torch.randint(0, 256, c.shape, generator=_gen(seed), device="cuda"))
        e = torch.randint(-30, 12, s.shape, generator=_gen(seed + 5), device="cuda")
        s.copy_(torch.exp2(e.double()))
        s.view(-1)[0] = float("nan")
    src = rng.integers(0, NB, P)
    src[-1] = src[0]                                          # a source read twice
    pairs = np.stack([src, rng.permutation(NO)[:P]], 1).astype(np.int64)
    ko = torch.full((NO, H, B, D), 7.0, dtype=dt, device="cuda")
    vo = ko.clone()
    pkv.block_read_fp8(ko, vo, kc, vc, ks, vs, torch.from_numpy(pairs).cuda())
    values = oracle.e4m3_values()
    for out, c, s in ((ko, kc, ks), (vo, vc, vs)):
        want = np.full((NO, H, B, D), 7.0)
        want[pairs[:, 1]] = (values[_codes(c)] * to_f64(s))[pairs[:, 0]]
        want = torch.from_numpy(want).to(dt).double().numpy()  # (bf16: exact; fp16: the one rounding)
        assert np.array_equal(to_f64(out), want, equal_nan=True)


def test_read_bad_blocks(cuda_device):
    kc, vc, ks, vs = _empty_cache(3, 2, 8, 64, fill=0x38)
    ko = torch.zeros((2, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    pairs = torch.tensor([[3, 0], [0, 2], [-1, 0], [2, 1], [0, 1 << 40]], device="cuda")
    pkv.block_read_fp8(ko, vo, kc, vc, ks, vs, pairs)
    assert pkv.device_status(clear=True) == _lib.DEV_BAD_BLOCK_ID
    assert not ko[0].any() and (ko[1] == 0.5).all() and (vo[1] == 0.5).all()


def test_block_copy_of_codes_and_scales(cuda_device):
    """Copy-on-write of an 8-bit block: codes and scales, a call each."""
    kc, vc, ks, vs = _empty_cache(6, 2, 16, 64)
    k = _randn((32, 2, 64), 3, torch.bfloat16)
    pkv.kv_append_fp8(k, k, kc, vc, ks, vs, torch.arange(32, device="cuda"))
    pairs = torch.tensor([[1, 4], [0, 5]], device="cuda")
    pkv.block_copy(kc, vc, pairs)
    pkv.block_copy(ks, vs, pairs)
    for t in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs):
        assert torch.equal(t[4], t[1]) and torch.equal(t[5], t[0])


# ---- norms with rotary positions ---------------------------------------------------------------


def _norm_rope_ref(x, weight, eps, positions, axes, inv_freq, interleaved, factor):
    y = x if weight is None else oracle.norm(x, weight, eps)
    out, mag = np.array(y), np.zeros_like(y)
    half = len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = positions[axes[i]].astype(np.float64) * f
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        out[..., a] = factor * (y[..., a] * c - y[..., b] * s)
        out[..., b] = factor * (y[..., a] * s + y[..., b] * c)
        mag[..., a] = mag[..., b] = factor * (np.abs(y[..., a]) + np.abs(y[..., b]))
    mag[..., 2 * half:] = np.abs(y[..., 2 * half:])
    return out, mag


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,hq,hkv,D,rot,T,axes,norm,packed,inplace", [
    ("fp16", 8, 8, 64, 64, 1, 1, True, False, False),
    ("bf16", 32, 8, 128, 128, 37, 3, True, True, False),
    ("fp16", 12, 4, 128, 64, 65, 1, True, True, True),
    ("bf16", 5, 5, 64, 34, 9, 2, True, False, True),       # pairs that do not fill 16-byte chunks
    ("fp16", 3, 1, 128, 2, 130, 1, False, True, False),
    ("bf16", 40, 40, 128, 96, 300, 1, True, False, False),
    ("fp16", 7, 1, 64, 46, 31, 3, True, True, True),
    ("bf16", 1, 1, 64, 62, 2100, 2, True, True, False),
    ("bf16", 17, 1, 128, 126, 3, 1, False, False, True),
])
def test_norm_rope(cuda_device, dtype, hq, hkv, D, rot, T, axes, norm, packed, inplace, interleaved):
    dt = W.DTYPES[dtype]
    rng = np.random.default_rng(T * 7 + rot)
    if packed:
        qkv = _randn((T, hq + 2 * hkv, D), 3, dt)
        q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    else:
        q, k = _randn((T, hq, D), 4, dt), _randn((T, hkv, D), 5, dt)
    q64, k64 = to_f64(q), to_f64(k)
    before = to_f64(qkv) if packed else None
    weights = [(1 + 0.3 * torch.randn(D, generator=_gen(i), device="cuda")).to(dt) if norm else None
               for i in range(2)]
    pos = rng.integers(0, 1 << 21, (axes, T)).astype(np.int32)
    pos[0, 0] = 0
    if T > 4:
        pos[0, 2] = -1
    pair_axes = [int(a) for a in rng.integers(0, axes, rot // 2)]
    freq = pkv.rope_frequencies(rot, 500000.0)
    q_out, k_out = (q, k) if inplace else (torch.full((T, hq, D), 7.0, dtype=dt, device="cuda"),
                                           torch.full((T, hkv, D), 7.0, dtype=dt, device="cuda"))
    kept = to_f64(q_out), to_f64(k_out)
    positions = torch.from_numpy(pos).cuda() if axes > 1 else torch.from_numpy(pos[0]).cuda()
    res = pkv.qk_norm_rope(q_out, k_out, q, k, positions, freq, q_weight=weights[0],
                           k_weight=weights[1], eps=1e-5, pair_axes=pair_axes if axes > 1 else None,
                           interleaved=interleaved, attn_factor=1.25)
    assert res[0] is q_out and res[1] is k_out
    real = pos[0] >= 0
    for out, x, w, old in zip((q_out, k_out), (q64, k64), weights, kept):
        w = None if w is None else to_f64(w)
        ref, mag = _norm_rope_ref(x, w, 1e-5, pos, pair_axes, freq.cpu().numpy(), interleaved, 1.25)
        got = to_f64(out)
        bound = torch.finfo(dt).eps / 2 * np.abs(ref) + 2.0 ** -20 * mag
        bound += 2.0 ** -25 if dt == torch.float16 else 0.0     # subnormal fp16: an absolute half step
        assert (np.abs(got - ref) <= bound)[real].all(), np.abs(got - ref)[real].max()
        assert np.array_equal(got[~real], old[~real])
    if packed:  # the rest of the projection's rows as it was
        now = to_f64(qkv)
        a = hq + hkv if inplace else 0
        assert np.array_equal(now[:, a:], before[:, a:])


def test_norm_rope_without_norm_is_rope_append(cuda_device):
    """The same bits as rope_kv_append, which turns k into the cache."""
    q, k, v = (_randn((50, n, 128), n, torch.bfloat16) for n in (8, 2, 2))
    pos = torch.randint(0, 1 << 20, (50,), generator=_gen(1), device="cuda", dtype=torch.int32)
    freq = pkv.rope_frequencies(128)
    kc = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(50, device="cuda")
    want = pkv.rope_kv_append(torch.empty_like(q), q, k, v, pos, freq, kc, kc.clone(), slots)
    got_q, got_k = pkv.qk_norm_rope(torch.empty_like(q), torch.empty_like(k), q, k, pos, freq)
    assert torch.equal(got_q, want)
    assert torch.equal(got_k, kc[slots // 16, :, slots % 16])


def test_norm_rope_refusals(cuda_device):
    q = _randn((3, 4, 64), 1, torch.bfloat16)
    pos = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    freq = pkv.rope_frequencies(8)
    out = torch.empty_like(q)
    with pytest.raises(ValueError, match="pair_axes"):
        pkv.qk_norm_rope(out, out, q, q, pos, freq)
    with pytest.raises(ValueError, match="axis"):
        pkv.qk_norm_rope(out, out, q, q, pos, freq, pair_axes=[0, 1, 2, 0])
    with pytest.raises(ValueError, match="axis"):
        pkv.qk_norm_rope(out, out, q, q, pos, freq, pair_axes=[0, 1, 0])
    with pytest.raises(ValueError):
        pkv.qk_norm_rope(out, out, q, q, pos, freq, pair_axes=[0, 1, -1, 0])
    with pytest.raises(ValueError, match="weight"):
        pkv.qk_norm_rope(out, out, q, q, pos[0], freq, q_weight=torch.ones(32, device="cuda").bfloat16())
    with pytest.raises(ValueError, match="token"):
        pkv.qk_norm_rope(out, out, q, q, pos[0, :2], freq)


# ---- attention ---------------------------------------------------------------------------------


class Case:
    """A pool whose unused rows and blocks hold NaN codes and NaN scales."""

    def __init__(self, seed, dtype, hq, hkv, D, B, lens, drafts=None, masks=None, spread=1.0):
        rng = np.random.default_rng(seed)
        self.dt, self.D = W.DTYPES[dtype], D
        self.lens = np.asarray(lens)
        S = len(lens)
        need = [-(-n // B) for n in lens]
        NB = sum(need) + 3
        perm = rng.permutation(NB)
        self.tables = np.full((S, max(need) + 2), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = perm[at:at + n]
            at += n
        self.caches = _empty_cache(NB, hkv, B, D, fill=0x7f)
        for s in self.caches[2:]:
            s.fill_(float("nan"))
        total = int(self.lens.sum())
        self.k, self.v = _randn((total, hkv, D), seed + 1, self.dt), _randn((total, hkv, D), seed + 2, self.dt)
        if spread != 1.0:  # V rows of very different sizes
            self.v *= (spread ** torch.randn((total, hkv, 1), generator=_gen(seed + 3), device="cuda")).to(self.dt)
        slots = np.concatenate([self.tables[s, np.arange(n) // B].astype(np.int64) * B + np.arange(n) % B
                                for s, n in enumerate(lens)] + [np.zeros(0, np.int64)])
        self.slots = torch.from_numpy(slots).cuda()
        if total:
            pkv.kv_append_fp8(self.k, self.v, *self.caches, self.slots)
        self.start = None
        rows = S
        if drafts is not None:
            self.start = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
            rows = int(self.start[-1])
            self.masks = np.asarray(masks, dtype=np.uint64).astype(np.int64) if masks is not None else None
            self.max_q = int(max(drafts))
        self.q = (2 * torch.randn((rows, hq, D), generator=_gen(seed + 7), device="cuda")).to(self.dt)
        self.scale = D ** -0.5
        self.max_ctx = int(max(lens))
        self.t_tables = torch.from_numpy(self.tables).cuda()
        self.t_lens = torch.from_numpy(self.lens.astype(np.int32)).cuda()

    def run(self, out=None, **kw):
        out = torch.full_like(self.q, 3.0) if out is None else out
        kw.setdefault("max_context_len", self.max_ctx)
        if self.start is None:
            return pkv.paged_attn_decode_fp8(out, self.q, *self.caches, self.t_tables, self.t_lens,
                                             self.scale, **kw)
        kw.setdefault("max_query_len", self.max_q)
        return pkv.paged_attn_tree_fp8(out, self.q, torch.from_numpy(self.start).cuda(),
                                       torch.from_numpy(self.masks).cuda(), *self.caches,
                                       self.t_tables, self.t_lens, self.scale, **kw)

    def reference(self):
        """(out, bound) in 64 bits on the GPU, from the codes in the caches."""
        values = torch.from_numpy(oracle.e4m3_values()).cuda()
        kc, vc, ks, vs = self.caches
        B, H = kc.shape[2], kc.shape[1]
        hq = self.q.shape[1]
        out = torch.zeros(self.q.shape, dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(out)
        eps = torch.finfo(self.dt).eps
        for s, n in enumerate(self.lens):
            n = int(n)
            lo, hi = (s, s + 1) if self.start is None else (int(self.start[s]), int(self.start[s + 1]))
            if n == 0 or hi == lo:
                continue
            at = self.t_tables[s, :-(-n // B)].long()

            def rows(c, sc):
                x = values[c.view(torch.uint8)[at].long()] * sc[at].double()
                return x.transpose(1, 2).reshape(-1, H, self.D)[:n].transpose(0, 1)

            k, v = rows(kc, ks), rows(vc, vs)                                  # [H, n, D]
            L = hi - lo
            q = self.q[lo:hi].double().view(L, H, hq // H, self.D).permute(1, 2, 0, 3)
            x = (q @ k[:, None].transpose(-1, -2)) * self.scale                # [H, G, L, n]
            a = ((q.abs() @ k[:, None].abs().transpose(-1, -2)) * self.scale)
            seen = torch.ones((L, n), dtype=torch.bool, device="cuda")
            if self.start is not None:
                for j in range(L):
                    m = int(self.masks[lo + j])
                    for i in range(L):
                        seen[j, n - L + i] = (m >> i) & 1 == 1
            x = torch.where(seen, x, -torch.inf)
            a = torch.where(seen, a, 0.0)
            p = torch.exp(x - x.amax(-1, keepdim=True))
            p = torch.where(seen, p / p.sum(-1, keepdim=True), 0.0)
            none = ~seen.any(-1)
            p[:, :, none] = 0.0
            # a row that is not seen must not count, NaN or not
            kept = torch.where(seen.any(0)[None, :, None], v, 0.0)
            o = torch.zeros((H, hq // H, L, self.D), dtype=torch.float64, device="cuda")
            size = torch.zeros_like(o)
            top = torch.zeros_like(o)
            for j in range(L):  # (per query: what one sees another may not)
                vj = torch.where(seen[j][None, :, None], kept, 0.0)
                o[:, :, j] = p[:, :, j] @ vj
                size[:, :, j] = p[:, :, j] @ vj.abs()
                top[:, :, j] = vj.abs().amax((1, 2))[:, None, None]
            dx = (self.D / 16 + 8) * 2.0 ** -23 * a.amax(-1, keepdim=True)
            b = eps / 2 * o.abs() + (2 * dx + 2.0 ** -17 + 2.0 ** -11) * size + n * 2.0 ** -23 * top
            if self.dt == torch.float16:
                b += 2.0 ** -25
            out[lo:hi] = o.permute(2, 0, 1, 3).reshape(L, hq, self.D)
            bound[lo:hi] = b.permute(2, 0, 1, 3).reshape(L, hq, self.D)
        return out, bound

    def check(self, got=None, **kw):
        got = self.run(**kw) if got is None else got
        ref, bound = self.reference()
        err = (got.double() - ref).abs()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        bad = ~(err <= bound * (1 + 1e-9)) & ~torch.isnan(ref)
        assert not bad.any(), (int(bad.sum()), float((err / bound.clamp(min=1e-30))[bad].max()))
        return got


DECODE = [
    # dtype, hq, hkv, D, B, lens, partition
    ("fp16", 8, 8, 64, 16, [1], 0),
    ("bf16", 8, 2, 128, 16, [1, 2, 15, 16, 17, 100], 0),
    ("fp16", 4, 1, 128, 8, [127, 128, 129, 0, 255, 256, 257], 0),
    ("bf16", 24, 3, 64, 32, [5, 0, 300, 1000, 7], 0),
    ("fp16", 40, 40, 128, 16, [33, 700, 512], 0),
    ("bf16", 32, 2, 64, 64, [640, 129, 1], 0),                # groups of 16
    ("fp16", 32, 1, 128, 128, [1300, 90], 0),                 # groups of 32
    ("bf16", 40, 1, 128, 16, [500, 131], 0),                  # groups of 40: two chunks
    ("fp16", 66, 1, 64, 16, [260], 0),                        # groups of 66: three chunks
    ("bf16", 33, 3, 128, 16, [4000, 17, 900], 0),             # groups of 11
    ("fp16", 7, 1, 64, 8, [3000], 128),
    ("bf16", 8, 1, 128, 16, [5000, 1, 129, 0, 128], 128),     # 40 partitions
    ("bf16", 12, 4, 128, 16, [2047, 2048, 2049], 512),
    ("fp16", 16, 4, 64, 16, [900, 1025], 1024),
]


@pytest.mark.parametrize("dtype,hq,hkv,D,B,lens,part", DECODE)
def test_decode(cuda_device, dtype, hq, hkv, D, B, lens, part):
    c = Case(hq * 31 + D, dtype, hq, hkv, D, B, lens)
    c.check(partition_size=part)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_decode_many_sequences(cuda_device, dtype):
    """More work items than SMs, of very different lengths."""
    lens = np.random.default_rng(3).integers(0, 700, 90).tolist()
    Case(11, dtype, 16, 4, 128, 16, lens).check()
    Case(12, dtype, 6, 3, 64, 8, lens).check()


def test_decode_loose_bound(cuda_device):
    c = Case(5, "bf16", 8, 2, 128, 16, [40, 300, 129])
    wide = torch.full((3, 4096), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.t_tables.shape[1]] = c.t_tables
    tight = c.check()
    c.t_tables = wide
    got = c.check(max_context_len=65536)
    assert (got - tight).abs().max() < 0.05


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
def test_decode_v_rows_of_any_size(cuda_device, dtype, D):
    """V rows 2^-8 .. 2^8 of one another, zero rows among them, and a position
    that takes almost all of the weight with a V of zero."""
    c = Case(9, dtype, 8, 2, D, 16, [700, 300, 65], spread=4.0)
    c.v[::7] = 0
    c.k[1] = 0
    q = c.q[0, ::4].float()                                     # KV head h's first query head
    c.k[1] = (q / q.norm(dim=-1, keepdim=True) * 40).to(c.dt)
    c.v[1] = 0
    pkv.kv_append_fp8(c.k, c.v, *c.caches, c.slots)
    c.check()
    c.check(partition_size=128)


def test_decode_nan_rows(cuda_device):
    """A NaN in K or V reaches its sequence and KV head, nothing else."""
    c = Case(4, "bf16", 8, 2, 128, 16, [200, 150, 90])
    c.k[5, 0, 3] = float("nan")
    c.v[210, 1, 7] = float("inf")
    pkv.kv_append_fp8(c.k, c.v, *c.caches, c.slots)
    got = c.run()
    nan = torch.isnan(got).all(-1)
    want = torch.zeros_like(nan)
    want[0, :4], want[1, 4:] = True, True
    assert torch.equal(nan, want) and torch.equal(torch.isnan(got).any(-1), want)


def test_decode_scales(cuda_device):
    for scale in (0.0, -0.125, 1.0):
        c = Case(21, "fp16", 4, 2, 64, 16, [130, 64, 3])
        c.scale = scale
        ref = torch.zeros(c.q.shape, dtype=torch.float64, device="cuda")
        c.check()


def test_decode_q_rows_of_any_size(cuda_device):
    """Query rows of zeros, of subnormals and of large elements beside small ones."""
    for dtype in ("fp16", "bf16"):
        c = Case(6, dtype, 8, 2, 64, 16, [300, 40])
        c.q[0, 0] = 0
        c.q[0, 1] = 2.0 ** -24
        c.q[0, 2, ::2] *= 2.0 ** -9
        c.q[0, 3, 5] = 60.0
        c.q[1, 4] *= 16
        c.check()


def test_decode_bad_tables_and_lengths(cuda_device):
    c = Case(13, "bf16", 8, 2, 128, 16, [100, 90, 80])
    good = c.run()
    c.t_tables[1, 2] = 1 << 20
    out = c.run()
    assert pkv.device_status(clear=True) == _lib.DEV_BAD_BLOCK_ID
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    c = Case(13, "bf16", 8, 2, 128, 16, [100, 90, 80])
    c.t_lens[1], c.t_lens[2] = -4, 1 << 30
    c.t_tables.clamp_(min=0)
    out = c.run()
    assert pkv.device_status(clear=True) == _lib.DEV_BAD_CONTEXT_LEN
    assert torch.equal(out[0], good[0]) and not out[1].any()


def test_workspace_may_hold_anything(cuda_device):
    c = Case(14, "fp16", 8, 2, 128, 16, [1000, 130, 0, 500])
    size = pkv.decode_fp8_workspace_size(4, 8, 2, 128, 1000, 128)
    ws = torch.full((size // 4 + 64,), float("nan"), device="cuda")
    got = c.check(partition_size=128, workspace=ws[:size // 4])
    assert torch.isnan(ws[size // 4:]).all()
    with pytest.raises(pkv.PagedKVError, match="WORKSPACE"):
        c.run(partition_size=128, workspace=ws[:size // 4 - 4])
    assert torch.equal(got, c.run(partition_size=128, workspace=ws[:size // 4]))


def _random_masks(rng, drafts):
    """Ancestors and self of random trees (several roots)."""
    masks = []
    for L in drafts:
        mine = []
        for j in range(L):
            parent = int(rng.integers(-1, j)) if j else -1
            mine.append((mine[parent] if parent >= 0 else 0) | 1 << j)
        masks += mine
    return masks


TREES = [
    # dtype, hq, hkv, D, B, lens, drafts, partition
    ("bf16", 8, 2, 128, 16, [50], [1], 0),
    ("fp16", 4, 4, 64, 16, [5, 17, 200], [5, 3, 8], 0),          # the whole context drafted in the first
    ("bf16", 32, 8, 64, 8, [129, 600, 31, 130], [2, 5, 1, 5], 0),
    ("fp16", 36, 12, 128, 32, [500, 1100], [64, 33], 0),         # groups of 3, several chunks
    ("bf16", 8, 1, 128, 16, [300, 64, 70], [17, 64, 0], 0),      # groups of 8; a sequence without drafts
    ("fp16", 5, 5, 128, 16, [128, 256, 160], [64, 40, 33], 0),   # drafts across a tile's border
    ("bf16", 16, 4, 64, 16, [1000, 700, 90], [16, 7, 16], 128),
    ("fp16", 14, 2, 128, 64, [400, 129], [10, 3], 256),          # groups of 7
    ("bf16", 40, 1, 128, 128, [700], [3], 0),                    # groups of 40
]


@pytest.mark.parametrize("dtype,hq,hkv,D,B,lens,drafts,part", TREES)
def test_tree(cuda_device, dtype, hq, hkv, D, B, lens, drafts, part):
    rng = np.random.default_rng(sum(lens))
    c = Case(hq + D, dtype, hq, hkv, D, B, lens, drafts, _random_masks(rng, drafts))
    c.check(partition_size=part)


def test_tree_masks_that_leave_nothing(cuda_device):
    """Queries that see no position (no context before the drafts), bits of
    drafts that are not there, and partitions in which a query sees nothing."""
    lens, drafts = [6, 200, 64, 140], [6, 4, 64, 30]
    rng = np.random.default_rng(1)
    masks = [0, 1, 0, 0b111000, 0xffffffffffffffff, 1 << 40,
             0, 0xf0, 0b1000, 1] + [int(m) for m in rng.integers(0, 1 << 63, 64)] + [0] * 30
    c = Case(3, "bf16", 8, 2, 128, 16, lens, drafts, masks)
    got = c.check()
    assert not got[0].any() and not got[2].any() and not got[5].any()
    c.check(partition_size=128)
    one = Case(3, "fp16", 4, 2, 64, 16, [64, 63], [64, 63], [0] * 127)
    assert not one.run().any()


def test_tree_nan_where_masked(cuda_device):
    """NaN and infinities in drafted rows reach the queries that see them."""
    lens, drafts = [140, 20], [12, 20]
    masks = [(1 << j) | 1 for j in range(12)] + [1 << j for j in range(20)]
    for D, dtype in ((128, "bf16"), (64, "fp16")):
        c = Case(8, dtype, 4, 2, D, 16, lens, drafts, masks)
        c.k[130, 0, 0], c.v[131, 0, 1] = float("inf"), float("nan")     # drafted tokens 2 and 3
        c.v[145, 1] = float("nan")                                     # drafted token 5 of the second
        pkv.kv_append_fp8(c.k, c.v, *c.caches, c.slots)
        # a NaN code that no append wrote, in the row of drafted token 7
        blk, off = int(c.tables[0, 135 // 16]), 135 % 16
        c.caches[1].view(torch.uint8)[blk, 0, off, 9] = 0xff
        got = c.run()
        nan = torch.isnan(got).all(-1)
        want = torch.zeros_like(nan)
        want[2, :2] = want[3, :2] = want[7, :2] = True
        want[12 + 5, 2:] = True
        assert torch.equal(torch.isnan(got).any(-1), want)
        want[7] = nan[7]     # (a single NaN code: its element is NaN, the rest of the row may be)
        assert torch.equal(nan, want)
        want[7, :2] = True
        clean = Case(8, dtype, 4, 2, D, 16, lens, drafts, masks).run()
        assert torch.equal(got[~want], clean[~want])


def test_tree_of_one_is_decode(cuda_device):
    lens = [1, 77, 128, 400, 129]
    a = Case(2, "bf16", 16, 4, 128, 16, lens)
    b = Case(2, "bf16", 16, 4, 128, 16, lens, [1] * 5, [1] * 5)
    assert torch.equal(a.q, b.q) and torch.equal(a.check(), b.check())


def test_tree_rows_behind_the_last_sequence(cuda_device):
    c = Case(2, "bf16", 8, 2, 64, 16, [40, 90], [3, 9], _random_masks(np.random.default_rng(0), [3, 9]))
    want = c.run()
    extra = 5
    c.q = torch.cat([c.q, torch.full((extra, 8, 64), float("nan"), dtype=c.dt, device="cuda")])
    c.masks = np.concatenate([c.masks, np.full(extra, -1)])
    out = c.run(torch.full_like(c.q, 3.0))
    assert torch.equal(out[:12], want) and (out[12:] == 3.0).all()


def test_tree_bad_counts(cuda_device):
    """More drafts than the bound, or than the context: flagged, nothing faults
    and the other sequences are right."""
    drafts = [3, 9, 4]
    c = Case(2, "bf16", 8, 2, 64, 16, [40, 90, 60], drafts, _random_masks(np.random.default_rng(0), drafts))
    want = c.run()
    out = c.run(max_query_len=4)
    assert pkv.device_status(clear=True) == _lib.DEV_BAD_CONTEXT_LEN
    assert torch.equal(out[:3], want[:3]) and torch.equal(out[12:], want[12:])
    c.t_lens[1] = 5
    out = c.run()
    assert pkv.device_status(clear=True) == _lib.DEV_BAD_CONTEXT_LEN
    assert torch.equal(out[:3], want[:3]) and torch.equal(out[12:], want[12:])
    c.start = np.array([0, 3, 1 << 20, 16], dtype=np.int32)      # not ascending
    c.run()
    assert pkv.device_status(clear=True) == _lib.DEV_BAD_CONTEXT_LEN


def test_same_bits_on_every_call(cuda_device):
    c = Case(17, "bf16", 32, 8, 128, 16, [900, 333, 2000, 5])
    outs = [c.run() for _ in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_captured_and_on_other_streams(cuda_device):
    """A captured step replayed with new inputs in place, and two streams at once."""
    c = Case(18, "bf16", 16, 4, 128, 16, [700, 131, 64])
    d = Case(19, "fp16", 8, 8, 64, 16, [500, 40], [7, 3], _random_masks(np.random.default_rng(4), [7, 3]))
    start, masks = torch.from_numpy(d.start).cuda(), torch.from_numpy(d.masks).cuda()
    wc = torch.empty(pkv.decode_fp8_workspace_size(3, 16, 4, 128, 700, 128), dtype=torch.uint8, device="cuda")
    oc, od = torch.empty_like(c.q), torch.empty_like(d.q)
    k, v, slots = c.k[:3].clone(), c.v[:3].clone(), c.slots[[699, 700 + 130, 700 + 131 + 63]].clone()

    def step():
        pkv.kv_append_fp8(k, v, *c.caches, slots)
        c.run(oc, partition_size=128, workspace=wc)
        pkv.paged_attn_tree_fp8(od, d.q, start, masks, *d.caches, d.t_tables, d.t_lens, d.scale,
                                d.max_ctx, d.max_q)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    k.copy_(_randn(k.shape, 77, c.dt))
    oc.zero_()
    od.zero_()
    graph.replay()
    torch.cuda.synchronize()
    c.check(oc)
    d.check(od)
    assert torch.equal(c.caches[2][c.slots[699] // 16, :, c.slots[699] % 16, 0],
                       torch.from_numpy(oracle.quantise(to_f64(k[0]))[1]).cuda().bfloat16())
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty_like(c.q), torch.empty_like(d.q)) for _ in streams]
    torch.cuda.synchronize()
    for st, (x, y) in zip(streams, outs):
        with torch.cuda.stream(st):
            for _ in range(5):
                c.run(x, partition_size=128)
                pkv.paged_attn_tree_fp8(y, d.q, start, masks, *d.caches, d.t_tables, d.t_lens,
                                        d.scale, d.max_ctx, d.max_q)
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x, oc) and torch.equal(y, od)


def test_a_run_over_an_8_bit_cache(cuda_device):
    """A prompt, a chunk over its prefix read back, a fork, drafted tokens
    checked in a tree, the accepted ones appended in order, and decode steps:
    the layer of a model that keeps its cache in 8 bits."""
    H, G, D, B, S = 2, 4, 64, 16, 2
    dt = torch.bfloat16
    alloc = pkv.BlockAllocator(num_blocks=24, block_size=B)
    caches = _empty_cache(24, H, B, D)
    freq = pkv.rope_frequencies(D)
    qw, kw = [(1 + 0.2 * torch.randn(D, generator=_gen(i), device="cuda")).to(dt) for i in (1, 2)]
    history = {s: [[], []] for s in (0, 1)}       # K and V rows in 16 bits, per position

    def layer(seed, positions):
        qkv = _randn((len(positions), (G + 2) * H, D), seed, dt)
        q, k, v = qkv[:, :G * H], qkv[:, G * H:G * H + H], qkv[:, -H:]
        pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
        pkv.qk_norm_rope(q, k, q, k, pos, freq, q_weight=qw, k_weight=kw)      # in place
        return q.contiguous(), k, v

    def remember(s, k, v):
        history[s][0] += list(to_f64(k))
        history[s][1] += list(to_f64(v))

    def reference(q, s, masks):
        """Queries q, the last of the sequence's positions, over its quantised rows."""
        rows = []
        for part in history[s]:
            codes, scales = oracle.quantise(np.stack(part))
            rows.append(oracle.e4m3_values()[codes] * scales[..., None])
        n = len(rows[0])
        k, v = (r.transpose(1, 0, 2)[None] for r in rows)                      # one block of n
        return oracle.tree_attention(to_f64(q), k, v, [[0]], [n], [0, len(q)], masks, D ** -0.5)[0]

    def near(got, ref, what):
        err = np.abs(to_f64(got) - ref)
        assert (err <= 2e-2 + 2e-2 * np.abs(ref)).all(), (what, err.max())

    # a prompt of 40, then a chunk of 13 over its prefix read back into 16 bits
    alloc.add_seq(0, 53)
    slots = torch.from_numpy(alloc.seq_slots(0, 0, 53)).cuda()
    _, k, v = layer(1, range(40))
    pkv.kv_append_fp8(k, v, *caches, slots[:40])
    remember(0, k, v)
    q, k, v = layer(2, range(40, 53))
    pkv.kv_append_fp8(k, v, *caches, slots[40:])
    remember(0, k, v)
    table = alloc.block_table([0], 4)
    blocks = table[0][table[0] >= 0]
    pairs = torch.tensor([[int(b), i] for i, b in enumerate(blocks)], device="cuda")
    wide = [torch.zeros((len(blocks), H, B, D), dtype=dt, device="cuda") for _ in range(2)]
    pkv.block_read_fp8(*wide, *caches, pairs)
    out = torch.empty_like(q)
    pkv.paged_attn_prefill(out, q, torch.tensor([0, 13], dtype=torch.int32, device="cuda"), *wide,
                           torch.arange(len(blocks), dtype=torch.int32, device="cuda")[None],
                           torch.tensor([53], dtype=torch.int32, device="cuda"), D ** -0.5, 53, 13)
    near(out, reference(q, 0, [(2 << j) - 1 for j in range(13)]), "chunk")
    # a fork that shares the prompt's blocks
    alloc.fork(0, 1)
    history[1] = [list(h) for h in history[0]]
    length = 53                                    # (the allocator's lengths run ahead: slots of
    for step in range(2):                          # rejected drafts are used again)
        # three drafted tokens per sequence: two guesses for the next, and one after the second
        masks, at = [0b001, 0b010, 0b110], length
        while alloc.seq_info(0)[0] < at + 3:
            _, pr = alloc.append_slots([0, 1])
            if len(pr):
                pr = torch.from_numpy(pr).cuda()
                pkv.block_copy(caches[0], caches[1], pr)
                pkv.block_copy(caches[2], caches[3], pr)
        slots = np.stack([alloc.seq_slots(s, at, 3) for s in range(S)], 1)     # [3, S]
        qs, kept = [], []
        for s in range(S):
            q, k, v = layer(10 * step + s + 5, [at, at, at + 1])
            pkv.kv_append_fp8(k, v, *caches, torch.from_numpy(slots[:, s].copy()).cuda())
            qs.append(q)
            kept.append((k.clone(), v.clone()))
        q = torch.cat(qs)
        lens = torch.full((S,), at + 3, dtype=torch.int32, device="cuda")
        tables = torch.from_numpy(alloc.block_table([0, 1], 8)).cuda()
        out = torch.empty_like(q)
        pkv.paged_attn_tree_fp8(out, q, torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda"),
                                torch.tensor(masks * 2, device="cuda"), *caches, tables, lens,
                                D ** -0.5, at + 3, 3)
        for s in range(S):
            old = [list(h) for h in history[s]]
            remember(s, *kept[s])
            near(out[3 * s:3 * s + 3], reference(qs[s], s, masks), f"tree {step} {s}")
            history[s] = old
            # tokens 1 and 2 are right: their rows again, at the first two places
            k, v = kept[s]
            pkv.kv_append_fp8(k[1:], v[1:], *caches, torch.from_numpy(slots[:2, s].copy()).cuda())
            remember(s, k[1:], v[1:])
        # a plain decode step, in the third place
        sl = slots[2].copy()
        q, k, v = layer(100 + step, [at + 2] * S)
        pkv.kv_append_fp8(k, v, *caches, torch.from_numpy(sl).cuda())
        tables = torch.from_numpy(alloc.block_table([0, 1], 8)).cuda()
        out = torch.empty_like(q)
        pkv.paged_attn_decode_fp8(out, q, *caches, tables, lens, D ** -0.5, at + 3)
        for s in range(S):
            remember(s, k[s:s + 1], v[s:s + 1])
            near(out[s:s + 1], reference(q[s:s + 1], s, [1]), f"decode {step} {s}")
        length = at + 3


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(cuda_device, seed):
    rng = np.random.default_rng(100 + seed)
    hkv = int(rng.choice([1, 2, 3, 5, 8]))
    group = int(rng.choice([1, 2, 3, 4, 6, 8, 16, 20]))
    D, B = int(rng.choice([64, 128])), int(rng.choice([8, 16, 32, 64, 128]))
    S = int(rng.integers(1, 9))
    lens = [int(np.exp(rng.uniform(0, np.log(1500)))) for _ in range(S)]
    part = int(rng.choice([0, 0, 128, 384]))
    dtype = str(rng.choice(["fp16", "bf16"]))
    Case(seed, dtype, hkv * group, hkv, D, B, lens).check(partition_size=part)
    drafts = [int(rng.integers(0, min(n, 24) + 1)) for n in lens]
    drafts[0] = max(drafts[0], 1)
    Case(seed + 50, dtype, hkv * group, hkv, D, B, lens, drafts, _random_masks(rng, drafts)).check(
        partition_size=part)
