"""Head norms over the whole range of bf16, where the squares of a row's elements pass
that of fp32.  Reference and tolerance are those of test_gpu_fp8."""

import numpy as np
import pytest
import torch

import paged_kv_cache_247_gb300 as pkv
from _gpu_util import to_f64
from test_gpu_fp8 import _clean_status, _gen, _norm_rope_ref  # noqa: F401 (an autouse fixture)

pytestmark = pytest.mark.gpu


def _check(x, weight, eps, rot, interleaved):
    """x as q, its first heads as k: every row within the tolerance of its own."""
    T, H, D = x.shape
    dt = x.dtype
    q, k = x, x[:, :max(H // 4, 1)].contiguous()
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 37
    freq = pkv.rope_frequencies(rot, 10000.0)
    q_out, k_out = pkv.qk_norm_rope(torch.empty_like(q), torch.empty_like(k), q, k, pos, freq, q_weight=weight,
                                    k_weight=weight, eps=eps, interleaved=interleaved)
    eps = float(np.float32(eps))
    for got, rows in ((q_out, q), (k_out, k)):
        ref, mag = _norm_rope_ref(to_f64(rows), to_f64(weight), eps, pos.cpu().numpy()[None], [0] * (rot // 2),
                                  freq.cpu().numpy(), interleaved, 1.0)
        err = np.abs(to_f64(got) - ref)
        bound = torch.finfo(dt).eps / 2 * np.abs(ref) + 2.0 ** -20 * mag + 2.0 ** -134
        assert (err <= bound).all(), float((err / bound).max())
    return q_out, k_out


@pytest.mark.parametrize("interleaved,rot", [(False, 64), (False, 34), (True, 64)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-36, 1e-6, 1e-3])
def test_rows_of_any_size(cuda_device, eps, D, interleaved, rot):
    """Rows from 2^-120 to 2^120, neighbours of very different sizes in one warp.
    (Where eps is above the squares, the outputs are small, not one.)"""
    gen = _gen(D)
    x = torch.randn((41, 9, D), generator=gen, device="cuda", dtype=torch.float64)
    e = torch.randint(-120, 121, (41, 9, 1), generator=gen, device="cuda").double()
    x = (x * torch.exp2(e)).bfloat16()
    w = (1 + 0.3 * torch.randn(D, generator=gen, device="cuda")).bfloat16()
    _check(x, w, eps, rot, interleaved)


def test_a_row_alone_gives_the_same_bits(cuda_device):
    """What its neighbours hold does not change a row."""
    x = torch.randn((8, 8, 128), generator=_gen(1), device="cuda").bfloat16()
    w = torch.ones(128, device="cuda").bfloat16()
    clean, _ = _check(x, w, 1e-6, 128, False)
    y = x.clone()
    y[:, 1::2] *= 2.0 ** 100
    mixed, _ = _check(y, w, 1e-6, 128, False)
    assert torch.equal(mixed[:, ::2], clean[:, ::2])


def test_infinities_nan_and_zeros(cuda_device):
    """As the formula says: an infinity leaves NaN in its place and zeros beside it,
    a NaN NaN everywhere in its row, a row of zeros zeros (NaN where eps is 0)."""
    x = torch.randn((3, 4, 64), generator=_gen(2), device="cuda").bfloat16()
    x[0, 0, 5], x[1, 1, 7], x[2] = float("inf"), float("nan"), 0.0
    w = torch.ones(64, device="cuda").bfloat16()
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    freq = pkv.rope_frequencies(64)
    out, _ = pkv.qk_norm_rope(torch.empty_like(x), torch.empty_like(x), x, x, pos, freq, q_weight=w, k_weight=w)
    nan = torch.isnan(out)
    assert nan[0, 0, 5] and nan[1, 1].all() and not out[2].any()
    assert (out[0, 0, :5] == 0).all() and not nan[0, 1:].any() and not nan[1, 0].any()
    out, _ = pkv.qk_norm_rope(torch.empty_like(x), torch.empty_like(x), x, x, pos, freq, q_weight=w, k_weight=w, eps=0.0)
    assert torch.isnan(out[2]).all()
