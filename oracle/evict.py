"""A cache smaller than the history, in fp64 and plain loops (oracle, test
infrastructure).

"The KV cache is a systems problem", section "Eviction and reuse can move costs
elsewhere": a sequence may drop cached positions and go on.  The pages give no
algorithm; these are the plain definitions of the calls that do it:

* ``rope`` — each pair of a head row turned by position * frequency;
* ``attention_weights`` — how much softmax weight each held position receives
  from given queries, per KV head (summed over the group's query heads);
* ``evict_select`` — the first ``sinks``, the last ``recent`` and the heaviest
  of the others, ties to the lowest position, in ascending order;
* ``compact`` — row i of the compacted sequence is row ``keep[i]``.
"""

import math

import numpy as np

from .attention import gather_sequence_kv


def rope(x, positions, inv_freq, interleaved, factor=1.0):
    """``x`` [T, H, D] with the first 2 * len(inv_freq) dimensions of every
    row turned; rows of negative positions unchanged."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    for t, pos in enumerate(positions):
        if pos < 0:
            continue
        for i, f in enumerate(inv_freq):
            c, s = math.cos(float(pos) * float(f)), math.sin(float(pos) * float(f))
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            u, v = x[t, :, a].copy(), x[t, :, b].copy()
            x[t, :, a] = factor * (u * c - v * s)
            x[t, :, b] = factor * (u * s + v * c)
    return x


def attention_weights(q, k_cache, block_table_row, context_len, scale, window=0):
    """Weights [Hkv, context_len] that the positions of one sequence receive
    from the queries ``q`` [L, Hq, D], its last L positions (causal); only the
    last ``window`` of them count (0: all)."""
    q = np.asarray(q, dtype=np.float64)
    n_q, num_q_heads, _ = q.shape
    k_seq, _ = gather_sequence_kv(k_cache, k_cache, block_table_row, context_len)
    num_kv_heads = k_cache.shape[1]
    group = num_q_heads // num_kv_heads
    out = np.zeros((num_kv_heads, context_len))
    first = max(0, n_q - window) if window else 0
    for j in range(first, n_q):
        pos = context_len - n_q + j
        for h in range(num_q_heads):
            logits = scale * (k_seq[:pos + 1, h // group] @ q[j, h])
            e = np.exp(logits - logits.max())
            out[h // group, :pos + 1] += e / e.sum()
    return out


def evict_select(weights, n, budget, recent, sinks):
    """Kept positions (ascending list) of one row of ``n`` weights."""
    if n <= budget:
        return list(range(n))
    middle = range(sinks, n - recent)

    def rank(i):
        w = float(weights[i])
        return (1, 0.0, i) if math.isnan(w) else (0, -w, i)

    chosen = sorted(middle, key=rank)[:budget - sinks - recent]
    return list(range(sinks)) + sorted(chosen) + list(range(n - recent, n))


def compact(cache, src_tables, dst_tables, keep, lens):
    """The cache after moving position keep[s][h][i] of every sequence and
    head to position i (any array [NB, Hkv, B, ...])."""
    old, new = np.asarray(cache), np.array(cache)
    B = old.shape[2]
    S, H, budget = keep.shape
    for s in range(S):
        for h in range(H):
            for i in range(min(int(lens[s]), budget)):
                k = int(keep[s, h, i])
                new[dst_tables[s, i // B], h, i % B] = old[src_tables[s, k // B], h, k % B]
    return new


def compact_weights(weights, keep, lens):
    """Rows of weights [S, H, W] moved likewise; what a sequence held behind
    its kept positions becomes 0."""
    old, new = np.asarray(weights), np.array(weights)
    S, H, budget = keep.shape
    for s in range(S):
        n = int(lens[s])
        m = min(n, budget)
        new[s, :, :n] = 0
        for h in range(H):
            new[s, h, :m] = old[s, h, keep[s, h, :m]]
    return new
