"""Pins of the oracle's eviction functions to facts that do not come from it."""

import math

import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_rotation_and_depends_on_distance(interleaved):
    rng = np.random.default_rng(0)
    freq = 100.0 ** (-np.arange(4) / 4)
    x = rng.standard_normal((2, 1, 10))
    y = oracle.rope(x, [3, 8], freq, interleaved)
    assert np.array_equal(y[..., 8:], x[..., 8:])             # past the rotated dimensions
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    z = oracle.rope(x, [103, 108], freq, interleaved)
    assert np.isclose(y[0, 0] @ y[1, 0], z[0, 0] @ z[1, 0])   # only the distance counts
    assert np.array_equal(oracle.rope(x, [0, -1], freq, interleaved), x)
    one = np.zeros((1, 1, 4))
    one[0, 0, 0] = 1.0
    turned = oracle.rope(one, [1], [math.pi / 2, 0.0], interleaved, factor=2.0)[0, 0]
    want = [0, 2, 0, 0] if interleaved else [0, 0, 2, 0]
    assert np.allclose(turned, want)


def test_attention_weights_sum_to_the_queries():
    rng = np.random.default_rng(1)
    k = rng.standard_normal((5, 2, 4, 8))
    q = rng.standard_normal((6, 4, 8))
    w = oracle.attention_weights(q, k, [3, 0, 4], 9, 0.3)
    assert w.shape == (2, 9) and np.allclose(w.sum(1), 6 * 2)
    assert np.allclose(oracle.attention_weights(q, k, [3, 0, 4], 9, 0.3, window=2).sum(1), 2 * 2)
    # equal logits: query at position p spreads 1 / (p + 1) over what it sees
    u = oracle.attention_weights(np.zeros((3, 2, 8)), k, [1, 2], 3, 1.0)
    assert np.allclose(u, [[1 + 1 / 2 + 1 / 3, 1 / 2 + 1 / 3, 1 / 3]] * 2)


def test_select_and_compact():
    w = [0.0, 5.0, 1.0, 5.0, math.nan, -0.0, 5.0, 2.0, 0.0]
    assert oracle.evict_select(w, 9, 9, 2, 1) == list(range(9))
    assert oracle.evict_select(w, 9, 4, 1, 1) == [0, 1, 3, 8]      # ties: the lowest positions
    assert oracle.evict_select(w, 9, 8, 0, 0) == [0, 1, 2, 3, 5, 6, 7, 8]  # NaN goes first
    assert oracle.evict_select(w, 9, 3, 3, 0) == [6, 7, 8]
    assert oracle.evict_select(w, 9, 3, 0, 3) == [0, 1, 2]
    cache = np.arange(12.0).reshape(3, 1, 4, 1)
    table = np.array([[2, 0]])
    keep = np.array([[[1, 4, 6]]])
    out = oracle.compact(cache, table, table, keep, [7])
    assert out[2, 0, :, 0].tolist() == [9.0, 0.0, 2.0, 11.0]
    assert np.array_equal(out[:2], cache[:2])
    moved = oracle.compact(cache, table, np.array([[1]]), keep, [7])
    assert moved[1, 0, :, 0].tolist() == [9.0, 0.0, 2.0, 7.0] and np.array_equal(moved[2], cache[2])
    ww = oracle.compact_weights(np.arange(9.0).reshape(1, 1, 9), keep, [7])
    assert ww[0, 0].tolist() == [1, 4, 6, 0, 0, 0, 0, 7, 8]
