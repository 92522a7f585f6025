"""How the library splits contexts over an 8-bit cache, on a machine without a GPU (or
on one with 152 SMs), read off the workspace sizes."""

import pytest

import paged_kv_cache_247_gb300 as pkv

SMS = 152


def parts_of(seqs, kv_heads, rows, dim, ctx):
    size = pkv.decode_fp8_workspace_size(seqs, kv_heads * rows, kv_heads, dim, ctx)
    per_part = seqs * kv_heads * rows * (dim + 2) * 4
    assert size % per_part == 0
    return max(size // per_part, 1)


def model_us(units, rows, dim, tiles, parts):
    """The call's time as the library reckons it."""
    slots = (1 if rows > 32 else 2) * SMS
    whole, rest = divmod(units * parts, slots)
    rounds = whole + (max(rest / slots, 0.8) if rest else 0.0)
    us = 1.5 * (-(-tiles // parts) + 2) * rounds
    if parts > 1:
        us += 7 + parts * (0.2 + units * min(rows, 64) * dim * 8 / 6.8e6)
    return us


@pytest.mark.parametrize("seqs,kv_heads,rows,dim,ctx", [
    (1, 1, 1, 128, 1), (1, 1, 1, 128, 129), (1, 1, 4, 64, 16384), (1, 1, 64, 128, 1 << 20), (1, 8, 4, 128, 32768),
    (2, 1, 33, 64, 5000), (3, 5, 7, 128, 1 << 17), (4, 8, 64, 64, 8192), (13, 1, 16, 128, 99999),
    (19, 8, 12, 128, 4096), (32, 8, 16, 128, 4096), (64, 8, 4, 128, 8192), (152, 4, 1, 64, 70000), (1, 1, 2, 128, 1 << 29)])
def test_the_split_is_the_models_best(lib, seqs, kv_heads, rows, dim, ctx):
    """Within 1 % of the best of all splits of up to three rounds of items."""
    units, tiles = seqs * kv_heads, -(-ctx // 128)
    slots = (1 if rows > 32 else 2) * SMS
    distinct = {-(-tiles // -(-tiles // p)) for p in range(1, min(tiles, 3 * slots // units + 1) + 1)}
    best = min(model_us(units, rows, dim, tiles, p) for p in distinct)
    parts = parts_of(seqs, kv_heads, rows, dim, ctx)
    assert parts in distinct
    assert model_us(units, rows, dim, tiles, parts) <= 1.01 * best


@pytest.mark.parametrize("seqs,heads,rows,dim,ctx", [(4, 8, 20, 64, 600), (4, 8, 1, 64, 200), (1, 8, 4, 128, 1024)])
def test_short_contexts_stay_whole(lib, seqs, heads, rows, dim, ctx):
    """A split costs more on the host than it gains: four chains of drafts over up to
    600 positions took 28 us a call, whole 13."""
    assert parts_of(seqs, heads, rows, dim, ctx) == 1


@pytest.mark.parametrize("rows,ctx,most", [(1, 16384, 50), (4, 16384, 50), (4, 65536, 90)])
def test_one_sequence_of_one_head(lib, rows, ctx, most):
    """Where partitions cost their joining alone: 128 of one tile took 28.7 us, 26 of
    five 16.4; 171 of three 38.9, 57 of nine 24.6."""
    assert 10 <= parts_of(1, 1, rows, 128, ctx) <= most
