"""Attention over a cache held in 8 bits where the types' ranges are used: query
elements far below the largest of their row, many weights far below the largest.
Cases are those of test_gpu_fp8.

Tolerance.  As there, |err| <= eps / 2 |out| + (2 dx + 2^-17 + 2^-11) sum_t p_t |v_t|,
but each position's lost weight by itself, and the fp32 sums' roundings with the
length: of O^T, which takes up 32 positions at a time, at most 2^-23 each, and of the
weights, 128 of them side by side, 2^-24:
  (n / 32) 2^-23 + (n / 128) 2^-24 <= n 2^-27
of sum_t p_t |v_t|.  A weight times its V row's scale is rounded to fp16 where the
largest such product stands at 2^6 or more: its own half step is 2^-25, so that a
position loses at most 2^-31 of the largest product over its own scale:
  lost_t = min(p_t, 2^-31 max_s p_s 2^e_s / 2^e_t).
"""

import math

import pytest
import torch

import oracle
import paged_kv_cache_247_gb300 as pkv
from test_gpu_fp8 import Case, _clean_status, _gen  # noqa: F401 (an autouse fixture)

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
        e2 = scales[:, None].transpose(-1, -2)                                # [H, 1, 1, n]
        most = (p * e2).amax(-1, keepdim=True) / e2
        lost = torch.minimum(p, 2.0 ** -31 * most) @ v[:, None].abs()
        b = torch.finfo(c.dt).eps / 2 * o.abs() + (2 * dx + 2.0 ** -17 + 2.0 ** -11 + n * 2.0 ** -27) * size + lost
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
