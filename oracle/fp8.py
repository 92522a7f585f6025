"""A cache held in 8 bits, in fp64 and plain loops (oracle, test infrastructure).

"Only 20.4% of your KV cache held actual tokens", section "Why the KV cache is
the thing that limits your batch": the cache's bytes bound the batch.  The
pages give no 8-bit format; these are the plain definitions of the calls that
use one:

* ``e4m3_values`` — the 256 values of e4m3: a sign, four exponent bits with
  bias 7, three bits of fraction, NaN where all seven bits are set;
* ``quantise`` — the scale 2^e of a row and its codes, each the nearest value
  (the even code of two as near);
* ``norm`` — a head row divided by its root mean square, times a weight;
* ``tree_attention`` — attention of drafted tokens with a mask among them.
"""

import math

import numpy as np

from .attention import gather_sequence_kv


def e4m3_values():
    out = []
    for code in range(256):
        sign, e, f = (-1.0 if code & 0x80 else 1.0), (code >> 3) & 15, code & 7
        if e == 15 and f == 7:
            out.append(math.nan)
        elif e == 0:
            out.append(sign * f * 2.0 ** -9)
        else:
            out.append(sign * (1 + f / 8) * 2.0 ** (e - 7))
    return np.array(out)


def row_scale(row):
    """The smallest 2^e, e >= -126, with every |element| <= 448 * 2^e."""
    top = max(abs(float(x)) for x in row)
    e = -126
    while top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def quantise(x):
    """Codes (uint8, shape of ``x``) and scales (x.shape[:-1]) of rows."""
    x = np.asarray(x, dtype=np.float64)
    flat = x.reshape(-1, x.shape[-1])
    codes = np.zeros(flat.shape, dtype=np.uint8)
    scales = np.zeros(len(flat))
    positive = e4m3_values()[:127]
    for i, row in enumerate(flat):
        if not np.isfinite(row).all():
            scales[i] = math.nan
            continue
        scales[i] = row_scale(row)
        y = np.abs(row) / scales[i]
        above = np.minimum(np.searchsorted(positive, y), 126)  # first value >= y
        below = np.maximum(above - 1, 0)
        to_above, to_below = positive[above] - y, y - positive[below]
        up = (to_above < to_below) | ((to_above == to_below) & (above % 2 == 0))
        codes[i] = np.where(up, above, below) | np.where(np.signbit(row), 128, 0)
    return codes.reshape(x.shape), scales.reshape(x.shape[:-1])


def norm(x, weight, eps):
    x = np.asarray(x, dtype=np.float64)
    return x * weight / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def tree_attention(q, k_cache, v_cache, block_tables, context_lens, query_start, masks, scale):
    """``q`` [T, Hq, D] over fp64 caches: query j of sequence s sees every
    position before the sequence's drafted ones (its last L_s), and drafted
    position i where bit i of its mask is set; zeros if it sees nothing.  Also
    returns sum_t p_t |v_t| and max_t |scale| sum |q_d k_d| per output (the
    magnitudes that rounding errors scale with)."""
    q = np.asarray(q, dtype=np.float64)
    out = np.zeros_like(q)
    size, logit = np.zeros_like(q), np.zeros_like(q)
    group = q.shape[1] // k_cache.shape[1]
    for s, ctx in enumerate(context_lens):
        ctx, row0 = int(ctx), int(query_start[s])
        count = int(query_start[s + 1]) - row0
        k, v = gather_sequence_kv(k_cache, v_cache, block_tables[s], ctx)
        for j in range(count):
            bits = int(masks[row0 + j])
            seen = np.array([t < ctx - count or (bits >> (t - (ctx - count))) & 1 for t in range(ctx)],
                            dtype=bool)
            if not seen.any():
                continue
            for h in range(q.shape[1]):
                kk, vv = k[seen, h // group], v[seen, h // group]
                x = scale * (kk @ q[row0 + j, h])
                p = np.exp(x - x.max())
                p /= p.sum()
                out[row0 + j, h] = p @ vv
                size[row0 + j, h] = p @ np.abs(vv)
                logit[row0 + j, h] = abs(scale) * (np.abs(kk) @ np.abs(q[row0 + j, h])).max()
    return out, size, logit
