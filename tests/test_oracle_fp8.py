"""Pins of the oracle's 8-bit rows and tree attention to facts that do not come
from it: torch's own e4m3, powers of two, causal attention and row order."""

import math

import numpy as np
import pytest
import torch

import oracle


def test_values_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    ours = oracle.e4m3_values()
    assert np.array_equal(ours, codes, equal_nan=True)
    assert np.nanmax(ours) == 448.0


@pytest.mark.parametrize("seed", range(3))
def test_codes_are_nearest(seed):
    x = torch.randn(40, 64, generator=torch.Generator().manual_seed(seed)).bfloat16()
    codes, scales = oracle.quantise(x.double().numpy())
    m, e = np.frexp(scales)
    assert (m == 0.5).all()                                  # powers of two
    top = x.abs().amax(-1).double().numpy()
    assert (top <= 448 * scales).all() and (top > 224 * scales).all()
    again = (x.float() / torch.from_numpy(scales).float()[:, None]).to(torch.float8_e4m3fn)
    assert np.array_equal(codes, again.view(torch.uint8).numpy())


def test_rows_at_the_borders():
    rows = np.zeros((6, 64))
    rows[1, 0] = 448.0
    rows[2, 0] = np.nextafter(448.0, 449.0)
    rows[3, 0] = -2.0 ** -133
    rows[4, 3] = math.nan
    rows[5, 9] = -math.inf
    codes, scales = oracle.quantise(rows)
    assert scales[0] == 2.0 ** -126 and not codes[0].any()
    assert scales[1] == 1.0 and codes[1, 0] == 126
    assert scales[2] == 2.0 and codes[2, 0] == 118
    assert scales[3] == 2.0 ** -126 and codes[3, 0] == 0x84    # -2^-7 of the scale: a subnormal code
    assert math.isnan(scales[4]) and math.isnan(scales[5]) and not codes[4:].any()


def test_read_back_and_appended_again():
    x = np.random.default_rng(5).standard_normal((50, 64))
    codes, scales = oracle.quantise(x)
    values = oracle.e4m3_values()[codes] * scales[:, None]
    codes2, scales2 = oracle.quantise(values)
    assert np.array_equal(oracle.e4m3_values()[codes2] * scales2[:, None], values)


def test_norm_has_unit_size():
    x = np.random.default_rng(1).standard_normal((7, 3, 64)) * 9
    y = oracle.norm(x, np.ones(64), 0.0)
    assert np.allclose((y * y).mean(-1), 1.0)


def test_chain_is_causal_attention():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 6, 2, 8, 64))
    tables, lens = np.array([[3, 0, 5], [1, 2, 4]]), np.array([20, 9])
    start = np.array([0, 5, 7])
    q = rng.standard_normal((7, 4, 64))
    masks = [(2 << j) - 1 for j in range(5)] + [(2 << j) - 1 for j in range(2)]
    got, size, logit = oracle.tree_attention(q, k, v, tables, lens, start, masks, 0.1)
    ref = oracle.paged_prefill_attention(q, k, v, tables, lens, start, 0.1)
    assert np.allclose(got, ref, atol=1e-13)
    assert (size >= np.abs(got) - 1e-13).all() and (logit > 0).all()


def test_masks_choose_what_is_seen():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 2, 1, 8, 64))
    q = rng.standard_normal((3, 1, 64))
    args = (np.array([[1, 0]]), np.array([3]), np.array([0, 3]))
    got, _, _ = oracle.tree_attention(q, k, v, *args, [0, 1, 0b100], 1.0)
    assert not got[0].any()                                   # sees nothing
    assert np.allclose(got[1, 0], v[1, 0, 0]) and np.allclose(got[2, 0], v[1, 0, 2])
