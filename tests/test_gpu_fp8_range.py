"""Attention over a cache held in 8 bits where the types' ranges are used: query
elements far below the largest of their row, many weights far below the largest,
V rows whose sizes differ by any power of two.  Cases are those of test_gpu_fp8.

Tolerance.  As there, |err| <= eps / 2 |out| + (2 dx + 2^-17 + 2^-11) sum_t p_t |v_t|,
but each position's lost weight by itself, and the fp32 sums' roundings with the
length: of O^T, which takes up 32 positions at a time, at most 2^-23 each, and of the
weights, 128 of them side by side, 2^-24:
  (n / 32) 2^-23 + (n / 128) 2^-24 <= n 2^-27
of sum_t p_t |v_t|.  A weight times its V row's scale is rounded to fp16, whose own
half step is 2^-25, where the largest such product has come to 2^6 or more: 2^-31 of
it.  The scales that enter the product lie within 2^-6 and 2 of their reference, so
that a position loses at most 2^(7 - 31) of the largest weight, 2^-31 where all rows
have the same scale, and between, where they differ by 2^k, 2^(k + 1) <= 2^(2 k) times that:
  lost_t = min(p_t, 2^(min(7, 2 k) - 31) max_s p_s).
What is rounded last is the output with these errors in it: (1 + eps / 2) times them.
"""

import math

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_247_gb300 as pkv
from test_gpu_fp8 import Case, _clean_status, _gen, _random_masks  # noqa: F401 (an autouse fixture)

pytestmark = pytest.mark.gpu


def reference(c, held=0.0):
    """(out, bound) in 64 bits.  ``held``: what an element of a query row may be
    off by, of the row's largest (0 where the rows are held exactly)."""
    values = torch.from_numpy(oracle.e4m3_values()).cuda()
    kc, vc, ks, vs = c.caches
    B, H, hq = kc.shape[2], kc.shape[1], c.q.shape[1]
    out = torch.zeros(c.q.shape, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(out)
    for s, n in enumerate(int(n) for n in c.lens):
        lo, hi = (s, s + 1) if c.start is None else (int(c.start[s]), int(c.start[s + 1]))
        if n == 0 or hi == lo:
            continue
        at = c.t_tables[s, :-(-n // B)].long()

        def rows(x):
            return x.transpose(1, 2).reshape(-1, H, x.shape[-1])[:n].transpose(0, 1)

        k = rows(values[kc.view(torch.uint8)[at].long()] * ks[at].double())    # [H, n, D]
        scales = rows(vs[at].double())                                        # [H, n, 1]
        v = rows(values[vc.view(torch.uint8)[at].long()]) * scales
        L, G = hi - lo, hq // H
        q = c.q[lo:hi].double().view(L, H, G, c.D).permute(1, 2, 0, 3)         # [H, G, L, D]
        seen = torch.ones((L, n), dtype=torch.bool, device="cuda")
        if c.start is not None:
            for j in range(L):
                m = int(c.masks[lo + j])
                for i in range(L):
                    seen[j, n - L + i] = (m >> i) & 1 == 1
        kt = k[:, None].transpose(-1, -2)
        x = torch.where(seen, (q @ kt) * c.scale, -math.inf)
        a = (c.D / 16 + 8) * 2.0 ** -23 * (q.abs() @ kt.abs())
        a += held * q.abs().amax(-1, keepdim=True) * kt.abs().sum(-2, keepdim=True)
        dx = abs(c.scale) * torch.where(seen, a, 0.0).amax(-1, keepdim=True)
        p = torch.softmax(x, -1).nan_to_num(0.0)                              # (nothing seen: zeros)
        o, size = p @ v[:, None], p @ v[:, None].abs()
        e = torch.where((v != 0).any(-1), torch.log2(scales[..., 0]), math.nan)  # (rows of zeros lose nothing)
        e = e[~e.isnan()]
        k = float(e.max() - e.min()) if len(e) else 0.0
        lost = torch.minimum(p, 2.0 ** (min(7.0, 2 * k) - 31) * p.amax(-1, keepdim=True)) @ v[:, None].abs()
        half = torch.finfo(c.dt).eps / 2
        b = half * o.abs() + (1 + half) * ((2 * dx + 2.0 ** -17 + 2.0 ** -11 + n * 2.0 ** -27) * size + lost)
        b += 2.0 ** -25 if c.dt == torch.float16 else 2.0 ** -134              # half a subnormal step
        out[lo:hi] = o.permute(2, 0, 1, 3).reshape(L, hq, c.D)
        bound[lo:hi] = b.permute(2, 0, 1, 3).reshape(L, hq, c.D)
    return out, bound


def check(c, held=0.0, **kw):
    pkv.kv_append_fp8(c.k, c.v, *c.caches, c.slots)
    got = c.run(**kw).double()
    ref, bound = reference(c, held)
    worst = ((got - ref).abs() / bound).max()
    assert worst <= 1 + 1e-9, float(worst)
    return got


def case(dtype, rows, D, lens, drafts=None, masks=None, seed=1):
    """A case with one KV head and `rows` query rows of a sequence to an item."""
    return Case(seed, dtype, rows, 1, D, 16, lens, drafts, masks)


# ---- queries -----------------------------------------------------------------------------------


@pytest.mark.parametrize("rows,D", [(3, 64), (8, 128), (16, 64), (24, 128), (64, 64)])
@pytest.mark.parametrize("dtype,down,held", [
    ("bf16", 12, 0.0), ("bf16", 15, 0.0), ("bf16", 17, 0.0), ("fp16", 12, 0.0), ("fp16", 14, 0.0),
    ("bf16", 20, 2.0 ** -25), ("fp16", 17, 2.0 ** -25)])
def test_query_elements_far_below_the_largest(cuda_device, dtype, down, held, rows, D):
    """Logits that come from the small elements alone: K is zero where the query
    row is large, and all small elements of a row are the same, so that what one
    of them is off by adds up.  Three e4m3 parts, 16 apart, of a row scaled to a
    largest of more than 224 hold multiples of 2^-17: all eight bits of a bf16
    element from 2^-17 of the largest on, the eleven of an fp16 one from 2^-14."""
    c = case(dtype, rows, D, [40, 33])
    small = 1 + torch.randint(0, 128, (2, rows, 1), generator=_gen(3), device="cuda") / 128
    top = 1 + 127 / 128 * torch.rand((2, rows), generator=_gen(4), device="cuda")
    if dtype == "fp16":
        small += torch.randint(0, 8, (2, rows, 1), generator=_gen(5), device="cuda") / 1024
    c.q = (small * 2.0 ** (8 - down)).to(c.dt).expand(2, rows, D).contiguous()
    c.q[:, :, 5] = (top * 2.0 ** 8).to(c.dt)
    c.k = torch.randn((73, 1, D), generator=_gen(6), device="cuda") * 8 / D ** 0.5
    c.k[..., 5] = 0
    c.k = c.k.to(c.dt)
    c.scale = 2.0 ** (down - 8)
    check(c, held)


# ---- weights -----------------------------------------------------------------------------------


def heavy(c, n, at, gap):
    """Makes position `at` of sequence 0 outweigh the others by about 2^gap."""
    rows, D = c.q.shape[1], c.D
    c.q = (1 - torch.arange(rows, device="cuda") / (8 * rows))[None, :, None].expand(c.q.shape).to(c.dt).contiguous()
    c.k = 0.002 * torch.randn((n, 1, D), generator=_gen(8), device="cuda")
    c.k[at] = gap * math.log(2) / (D * c.scale)
    c.k = c.k.to(c.dt)


@pytest.mark.parametrize("rows,D", [(4, 64), (8, 128), (16, 128), (32, 64), (64, 128)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("gap", [24, 27])
def test_a_flat_tail_of_weights(cuda_device, dtype, gap, rows, D):
    """40,000 weights far below that of the first position, which alone they do
    not share a dimension with: each is small, their sum is the output there."""
    n = 40000
    c = case(dtype, rows, D, [n])
    heavy(c, n, 0, gap)
    c.v = 0.5 + 0.4 * torch.rand((n, 1, D), generator=_gen(9), device="cuda")
    c.v[..., 0] = 0
    c.v[0] = 0
    c.v[0, 0, 0] = 0.9
    c.v = c.v.to(c.dt)
    check(c, partition_size=-(-n // 128) * 128)


# ---- V rows ------------------------------------------------------------------------------------


@pytest.mark.parametrize("rows,D", [(4, 128), (12, 64), (32, 128), (64, 64)])
@pytest.mark.parametrize("at", [0, 20000, 32767])
@pytest.mark.parametrize("dtype,top", [("fp16", 1.0), ("fp16", 64.0), ("bf16", 400.0), ("fp16", 6e4),
                                       ("bf16", 1e6), ("bf16", 2.0 ** 100)])
def test_one_large_element_of_v(cuda_device, dtype, top, at, rows, D):
    """One position of great weight has a V row with a single large element, the
    other positions' weights add up to as much: every other dimension is theirs."""
    n = 32768
    c = case(dtype, rows, D, [n])
    heavy(c, n, at, 15)
    c.v = 0.5 + 0.6 * (torch.rand((n, 1, D), generator=_gen(2), device="cuda") - 0.5)
    c.v[at, 0, 0] = top
    c.v = c.v.to(c.dt)
    check(c, partition_size=n)


SIZES = [("fp16", -14, 12), ("bf16", -14, 12), ("bf16", -60, 55), ("bf16", -120, -30), ("bf16", 20, 115)]


@pytest.mark.parametrize("rows,D", [(1, 128), (8, 64), (16, 128), (27, 64), (64, 128)])
@pytest.mark.parametrize("dtype,lo,hi", SIZES)
def test_v_rows_of_every_size(cuda_device, dtype, lo, hi, rows, D):
    """V rows of any two sizes, zero rows among them, each row in an eighth of the
    dimensions, so that every dimension sums rows of other sizes."""
    lens = [700, 130, 1, 257]
    n = sum(lens)
    c = case(dtype, rows, D, lens, seed=rows)
    e = torch.randint(lo, hi + 1, (n, 1, 1), generator=_gen(5), device="cuda").double()
    own = (torch.arange(D, device="cuda") % 8)[None, None] == torch.randint(0, 8, (n, 1, 1), generator=_gen(6),
                                                                           device="cuda")
    v = torch.randn((n, 1, D), generator=_gen(7), device="cuda", dtype=torch.float64) * torch.exp2(e) * own
    v[::9] = 0
    c.v = v.to(c.dt)
    check(c)
    check(c, partition_size=128)


@pytest.mark.parametrize("dtype,lo,hi", SIZES)
def test_v_rows_of_every_size_under_trees(cuda_device, dtype, lo, hi):
    lens, drafts = [300, 64, 129, 40], [16, 64, 9, 3]
    c = Case(3, dtype, 4, 2, 64, 16, lens, drafts, _random_masks(np.random.default_rng(2), drafts))
    e = torch.randint(lo, hi + 1, (sum(lens), 2, 1), generator=_gen(5), device="cuda").double()
    own = torch.rand((sum(lens), 2, 64), generator=_gen(8), device="cuda") < 0.2
    c.v = (torch.randn((sum(lens), 2, 64), generator=_gen(7), device="cuda", dtype=torch.float64) * torch.exp2(e)
           * own).to(c.dt)
    check(c)
    check(c, partition_size=128)


@pytest.mark.parametrize("rows,D", [(4, 128), (16, 64), (48, 128)])
@pytest.mark.parametrize("size", [-126, -100, -70, -62, 60, 75, 110])
def test_v_rows_of_one_size_beside_zeros(cuda_device, size, rows, D):
    """Half of the positions hold zeros, the others rows of one size."""
    c = case("bf16", rows, D, [300, 128, 5])
    c.v = torch.randn((433, 1, D), generator=_gen(4), device="cuda", dtype=torch.float64) * 2.0 ** size
    c.v[::2] = 0
    c.v = c.v.to(c.dt)
    check(c)
    check(c, partition_size=128)


def test_tiles_of_zeros_before_and_after(cuda_device):
    """Whole tiles of zero rows at either end, and a cache of nothing else."""
    c = case("bf16", 8, 128, [640, 384, 256])
    c.v[:256] = 0
    c.v[640 + 128:1024] = 0
    c.v[1024:] = 0
    got = check(c)
    assert not got[2].any()
    check(c, partition_size=128)


def test_partitions_of_the_largest_values(cuda_device):
    """Partial outputs near the end of bf16's range, joined without passing it."""
    c = case("bf16", 8, 64, [1500])
    c.v = (torch.randn((1500, 1, 64), generator=_gen(4), device="cuda", dtype=torch.float64) * 2.0 ** 124).to(c.dt)
    c.k *= 0.01
    got = check(c, partition_size=128)
    assert torch.isfinite(got).all()


def test_a_huge_row_that_some_queries_do_not_see(cuda_device):
    """A drafted V row far above the rest: queries that do not see it get what
    the rest gives, those that do get theirs."""
    for D, rows, up in ((64, 4, 90), (128, 2, 110)):
        lens, drafts = [200, 60], [12, 5]
        masks = [(1 << j) | 1 for j in range(12)] + [1 << j for j in range(5)]
        c = Case(4, "bf16", rows, 1, D, 16, lens, drafts, masks)
        c.v = c.v.double()
        c.v[188 + 6] *= 2.0 ** up
        c.v[200 + 57] *= 2.0 ** up
        c.v = c.v.to(c.dt)
        check(c)
        check(c, partition_size=128)


def test_a_scale_of_zero_gives_the_mean(cuda_device):
    """Logits that are all zero: every output is the mean of the V rows."""
    c = Case(21, "fp16", 4, 2, 64, 16, [130, 64, 3])
    c.scale = 0.0
    got = check(c)
    values = torch.from_numpy(oracle.e4m3_values()).cuda()
    at = c.slots[:130]
    v = values[c.caches[1].view(torch.uint8)[at // 16, :, at % 16].long()] * c.caches[3][at // 16, :, at % 16].double()
    mean, size = v.mean(0), v.abs().mean(0)
    for h in range(4):
        assert ((got[0, h] - mean[h // 2]).abs() <= 2.0 ** -10 * size[h // 2] + 2.0 ** -25).all()
