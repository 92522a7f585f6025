"""The cache-eviction operators as a program uses them: the cases that are measured, their
inputs, the plain form of each operator in elementary torch operations, and its value in 64 bits.

The operators keep a sequence going in a paged cache smaller than its history: rotary positions
applied while new rows are appended, attention that also accumulates how much weight each cached
position received (one decode step, or a chunk of a prompt), the choice of the positions to keep,
and the compaction of the cache to them.
"""

import math
import random

import torch

own = False  # true: run() calls the framework's operators

_DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---- cases ---------------------------------------------------------------------------------------


def listed():
    return [
        # a small batch's decode step of a grouped-head layer: latency only
        {"name": "rope_step_8", "op": "rope", "tokens": 8, "heads": 32, "kv_heads": 8, "dim": 64,
         "block": 16, "dtype": "bf16", "rot": 64, "interleaved": False, "packed": True, "far": 4096},
        # one decode step of 64 sequences, 40 single heads of 128
        {"name": "rope_step_64_mha", "op": "rope", "tokens": 64, "heads": 40, "kv_heads": 40, "dim": 128,
         "block": 16, "dtype": "fp16", "rot": 128, "interleaved": True, "packed": False, "far": 2048},
        # prompt chunks of 8 x 2,048 tokens far into long contexts, half of each head rotated
        {"name": "rope_prompt_16k", "op": "rope", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "block": 16, "dtype": "bf16", "rot": 64, "interleaved": False, "packed": True, "far": 1000000},
        # a handful of short conversations on a small model: latency only
        {"name": "decode_4_short", "op": "decode", "seqs": 4, "heads": 8, "kv_heads": 8, "dim": 64,
         "block": 16, "dtype": "fp16", "lo": 1, "hi": 200, "decay": 1.0, "slack": 3, "shape": 1},
        # 64 requests of lengths around 500 over 40 single heads
        {"name": "decode_64_mha", "op": "decode", "seqs": 64, "heads": 40, "kv_heads": 40, "dim": 128,
         "block": 16, "dtype": "fp16", "lo": 16, "hi": 2048, "decay": 1.0, "slack": 0, "shape": 2},
        # 64 long conversations over grouped heads, decaying weights
        {"name": "decode_64x8k", "op": "decode", "seqs": 64, "heads": 32, "kv_heads": 8, "dim": 128,
         "block": 16, "dtype": "bf16", "lo": 8192, "hi": 8192, "decay": 0.98, "slack": 64, "shape": 3},
        # whole short prompts, of which the last 32 queries decide what is kept
        {"name": "prefill_16_prompts", "op": "prefill", "seqs": 16, "heads": 40, "kv_heads": 40, "dim": 128,
         "block": 16, "dtype": "fp16", "lo": 100, "hi": 700, "chunk": 700, "window": 32, "decay": 1.0,
         "shape": 4},
        # second half of 4k prompts in chunks of 2k, every query counted
        {"name": "prefill_8x2k_of_4k", "op": "prefill", "seqs": 8, "heads": 32, "kv_heads": 8, "dim": 128,
         "block": 16, "dtype": "bf16", "lo": 4096, "hi": 4096, "chunk": 2048, "window": 0, "decay": 1.0,
         "shape": 5},
        # 64 sequences that outgrew 8k together, cut to 2k
        {"name": "select_64x8k", "op": "select", "seqs": 64, "kv_heads": 8, "lo": 6000, "hi": 8192,
         "budget": 2048, "recent": 256, "sinks": 4, "slack": 0, "shape": 6},
        # one very long document, cut to a quarter
        {"name": "select_1x128k", "op": "select", "seqs": 1, "kv_heads": 8, "lo": 131072, "hi": 131072,
         "budget": 32768, "recent": 1024, "sinks": 4, "slack": 0, "shape": 7},
        # a lone sequence of a small model cut in half: latency
        {"name": "compact_1x1k", "op": "compact", "seqs": 1, "kv_heads": 8, "dim": 64, "block": 16,
         "dtype": "fp16", "lo": 1000, "hi": 1000, "budget": 500, "recent": 64, "slack": 0, "fresh": False,
         "shape": 8},
        # the 64 sequences of above, in place
        {"name": "compact_64x8k", "op": "compact", "seqs": 64, "kv_heads": 8, "dim": 128, "block": 16,
         "dtype": "bf16", "lo": 6000, "hi": 8192, "budget": 2048, "recent": 256, "slack": 0, "fresh": False,
         "shape": 6},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "decode", "prefill", "select", "compact"])
    dim, block = rng.choice([64, 128]), rng.choice([8, 16, 32, 64, 128])
    dtype = rng.choice(["fp16", "bf16"])
    kv = rng.choice([1, 2, 4, 5, 8, 12, 40])
    shape = rng.randrange(1 << 20)
    if op == "rope":
        heads = kv * rng.choice([1, 2, 3, 4, 7, 8])
        while heads > 64:
            heads -= kv
        return {"op": op, "tokens": _log_int(rng, 1, 16384 * 48 // (heads + 2 * kv) if heads + 2 * kv > 48 else 16384),
                "heads": heads, "kv_heads": kv, "dim": dim, "block": block, "dtype": dtype,
                "rot": rng.choice([dim, dim // 2, 32, 2 * rng.randrange(1, dim // 2 + 1)]),
                "interleaved": rng.random() < 0.5, "packed": rng.random() < 0.5,
                "far": _log_int(rng, 1 << 8, 1 << 21)}
    if op == "decode":
        group = rng.choice([1, 2, 3, 4, 7, 8, 16, 32])
        hi = _log_int(rng, 1, 32768)
        most = 64 * 8192 * 8 * 128 // (hi * kv * dim * max(1, group // 4))  # K/V elements, and the plain form's logits
        seqs = _log_int(rng, 1, max(1, min(256, most)))
        return {"op": op, "seqs": seqs, "heads": kv * group, "kv_heads": kv, "dim": dim, "block": block,
                "dtype": dtype, "lo": rng.choice([1, hi, max(1, hi // 3)]), "hi": hi,
                "decay": rng.choice([1.0, 0.9, 0.0]), "slack": rng.randrange(0, 40), "shape": shape}
    if op == "prefill":
        group = rng.choice([1, 2, 3, 4, 8])
        hi = _log_int(rng, 16, 8192)
        chunk = _log_int(rng, 1, hi)
        most = 8 * 32 * 2048 * 4096 // (hi * chunk * kv * group)
        while most < 1:
            chunk = max(1, chunk // 2)
            most = 8 * 32 * 2048 * 4096 // (hi * chunk * kv * group)
        return {"op": op, "seqs": _log_int(rng, 1, min(32, most)), "heads": kv * group, "kv_heads": kv,
                "dim": dim, "block": block, "dtype": dtype, "lo": rng.choice([max(1, hi // 7), hi]), "hi": hi,
                "chunk": chunk, "window": rng.choice([0, 0, 1, 16, 100]), "decay": rng.choice([1.0, 0.5, 0.0]),
                "shape": shape}
    hi = _log_int(rng, 64, 131072) if op == "select" else _log_int(rng, 2, 32768)
    budget = _log_int(rng, 8, hi // 2) if op == "select" else _log_int(rng, 1, hi)
    most = 64 * 8192 * 8 // (hi * kv) if op == "select" else 64 * 8192 * 8 * 128 // (hi * kv * dim)
    case = {"op": op, "seqs": _log_int(rng, 1, max(1, min(128, most))), "kv_heads": kv,
            "lo": rng.choice([1, hi, max(1, hi // 2)]), "hi": hi, "budget": budget,
            "recent": rng.randrange(0, budget // 2 + 1), "slack": rng.randrange(0, 40), "shape": shape}
    if op == "select":
        case["sinks"] = rng.randrange(0, budget // 4 + 1)
    else:
        case.update(dim=dim, block=block, dtype=dtype, fresh=rng.random() < 0.3)
    return case


def _lens(case):
    """Context lengths, spread over their logarithm; a case's lengths do not depend on its inputs' seed."""
    rng = random.Random(case["shape"])
    if case["lo"] == case["hi"]:
        return [case["hi"]] * case["seqs"]
    return [case["hi"]] + [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["seqs"] - 1)]


def _chunks(case):
    """Queries of each sequence: the whole context where it is shorter than the chunk."""
    return [min(n, case["chunk"]) for n in _lens(case)]


def work(case):
    e, op = 2, case["op"]
    if op == "rope":
        t, hq, h, d, r = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["rot"]
        return {"bytes": 2 * t * (hq + 2 * h) * d * e + 12 * t + 4 * r, "flops": 3 * r * (hq + h) * t}
    lens, h = _lens(case), case["kv_heads"]
    n = sum(lens)
    if op == "decode":
        d, hq, s = case["dim"], case["heads"], case["seqs"]
        return {"bytes": n * h * (2 * d * e + (8 if case["decay"] else 4)) + 2 * s * hq * d * e +
                4 * sum(-(-x // case["block"]) for x in lens), "flops": 4 * n * hq * d}
    if op == "prefill":
        d, hq = case["dim"], case["heads"]
        q = _chunks(case)
        pairs = sum(l * x - l * (l - 1) // 2 for l, x in zip(q, lens))
        return {"bytes": n * h * (2 * d * e + (8 if case["decay"] else 4)) + 2 * sum(q) * hq * d * e,
                "flops": 4 * pairs * hq * d}
    kept = sum(min(x, case["budget"]) for x in lens)
    if op == "select":
        over = sum(x for x in lens if x > case["budget"])
        return {"bytes": h * (4 * over + 4 * case["seqs"] * case["budget"]), "flops": 0}
    return {"bytes": h * kept * (4 * case["dim"] * e + 4 + 8) + h * 4 * (n - kept), "flops": 0}


# ---- inputs --------------------------------------------------------------------------------------


def _tables(case, lens, gen, copies=1):
    """Block tables over one pool in random order; with copies = 2, tables of other blocks too."""
    b = case["block"]
    per = torch.tensor([-(-x // b) for x in lens], device="cuda")
    width, total = int(max(-(-x // b) for x in lens)), int(sum(-(-x // b) for x in lens))
    pool = copies * total + total // 8 + 1
    perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    first = torch.cumsum(per, 0) - per
    col = torch.arange(width, device="cuda")
    at = first[:, None] + col
    held = col < per[:, None]
    out = [torch.where(held, perm[torch.where(held, at + c * total, 0)], -1).to(torch.int32) for c in range(copies)]
    return pool, out


def _cache(case, pool, gen):
    shape = (pool, case["kv_heads"], case["block"], case["dim"])
    dt = _DTYPES[case["dtype"]]
    return [torch.randn(shape, generator=gen, device="cuda", dtype=dt) for _ in range(2)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op == "rope":
        t, hq, h, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        dt, b = _DTYPES[case["dtype"]], case["block"]
        if case["packed"]:  # the projection's output, one row per token
            qkv = torch.randn((t, hq + 2 * h, d), generator=gen, device="cuda", dtype=dt)
            st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
        else:
            st["q"], st["k"], st["v"] = [torch.randn((t, n, d), generator=gen, device="cuda", dtype=dt)
                                         for n in (hq, h, h)]
        pool = -(-t // b) + 8
        st["k_cache"] = torch.zeros((pool, h, b, d), dtype=dt, device="cuda")
        st["v_cache"] = torch.zeros_like(st["k_cache"])
        st["slots"] = torch.randperm(pool * b, generator=gen, device="cuda")[:t]
        st["positions"] = torch.randint(0, case["far"], (t,), generator=gen, device="cuda", dtype=torch.int32)
        st["inv_freq"] = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        st["q_out"] = torch.empty((t, hq, d), dtype=dt, device="cuda")
        return st
    lens = _lens(case)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["max_ctx"] = max(lens)
    cap = max(lens) + case.get("slack", 0)
    # accumulated weights: heavy-tailed, some positions never attended to
    w = torch.exp(2.0 * torch.randn((case["seqs"], case["kv_heads"], cap), generator=gen, device="cuda") - 4.0)
    st["weights"] = torch.where(torch.rand(w.shape, generator=gen, device="cuda") < 0.02, 0.0, w)
    if op in ("decode", "prefill"):
        dt = _DTYPES[case["dtype"]]
        pool, (st["tables"],) = _tables(case, lens, gen)
        st["k_cache"], st["v_cache"] = _cache(case, pool, gen)
        st["scale"] = case["dim"] ** -0.5
        rows = case["seqs"]
        if op == "prefill":
            q = _chunks(case)
            st["start"] = torch.tensor([0] + q, device="cuda").cumsum(0).to(torch.int32)
            st["max_q"], rows = max(q), sum(q)
        # queries that attend unevenly: logits of standard deviation 2
        st["q"] = 2.0 * torch.randn((rows, case["heads"], case["dim"]), generator=gen, device="cuda", dtype=dt)
        st["out"] = torch.empty_like(st["q"])
        return st
    st["keep"] = torch.empty((case["seqs"], case["kv_heads"], case["budget"]), dtype=torch.int32, device="cuda")
    if op == "select":
        return st
    pool, tables = _tables(case, lens, gen, 2 if case["fresh"] else 1)
    st["tables"], st["to"] = tables[0], tables[-1]
    st["k_cache"], st["v_cache"] = _cache(case, pool, gen)
    st["keep"].copy_(_choose(st["weights"], st["lens"], case["budget"], case["recent"], 0))
    return st


# ---- the operators, plain or the framework's ------------------------------------------------------


def _gather(cache, tables):
    """[S, H, tokens, D] in 32 bits, through the tables."""
    x = cache[tables.clamp(min=0).long()].float()
    s, n, h, b, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(s, h, n * b, d)


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _rope(st):
    c = st["case"]
    angle = st["positions"].double()[:, None] * st["inv_freq"]  # 64 bits: positions are far
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = _rotate(st["q"], cos, sin, c["rot"], c["interleaved"]).to(st["q"].dtype)
    k = _rotate(st["k"], cos, sin, c["rot"], c["interleaved"]).to(st["k"].dtype)
    blk, off = st["slots"] // c["block"], st["slots"] % c["block"]
    st["k_cache"][blk, :, off] = k
    st["v_cache"][blk, :, off] = st["v"]
    st["q_out"].copy_(q)


def _accumulate(st, seen, p):
    """weights := decay * weights + p at the positions a sequence holds."""
    w = st["weights"]
    n = min(w.shape[2], p.shape[2])
    old = w[:, :, :n]
    w[:, :, :n] = torch.where(seen[:, None, :n], st["case"]["decay"] * old + p[:, :, :n], old)


def _decode(st):
    q, lens = st["q"], st["lens"]
    s, hq, d = q.shape
    k, v = _gather(st["k_cache"], st["tables"]), _gather(st["v_cache"], st["tables"])
    h = k.shape[1]
    seen = torch.arange(k.shape[2], device=q.device) < lens[:, None]
    x = (q.float().view(s, h, hq // h, d) @ k.transpose(-1, -2)) * st["scale"]
    x = torch.where(seen[:, None, None], x, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    p = e / e.sum(-1, keepdim=True)
    st["out"].copy_((p @ v).view(s, hq, d))
    _accumulate(st, seen, p.sum(2))


def _prefill(st):
    c, q, lens, start = st["case"], st["q"], st["lens"].long(), st["start"].long()
    t, hq, d = q.shape
    k, v = _gather(st["k_cache"], st["tables"]), _gather(st["v_cache"], st["tables"])
    s, h, n, _ = k.shape
    count = start[1:] - start[:-1]
    j = torch.arange(st["max_q"], device=q.device)
    there = j < count[:, None]
    rows = torch.where(there, start[:-1, None] + j, 0)
    qp = q[rows].float().view(s, st["max_q"], h, hq // h, d).permute(0, 2, 3, 1, 4)
    x = (qp @ k[:, :, None].transpose(-1, -2)) * st["scale"]
    key = torch.arange(n, device=q.device)
    last = torch.where(there, (lens - count)[:, None] + j, 0)  # a row that is none sees position 0
    seen = key <= last[:, :, None]
    x = torch.where(seen[:, None, None], x, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    x /= x.sum(-1, keepdim=True)
    o = (x @ v[:, :, None]).permute(0, 3, 1, 2, 4).reshape(s, st["max_q"], hq, d)
    row = torch.arange(t, device=q.device)
    of = torch.searchsorted(start, row, right=True) - 1
    st["out"].copy_(o[of, row - start[of]])
    counts = there & (j >= count[:, None] - (c["window"] or st["max_q"]))
    _accumulate(st, key < lens[:, None], (x * counts[:, None, None, :, None]).sum((2, 3)))


def _choose(weights, lens, budget, recent, sinks):
    n = weights.shape[2]
    key = torch.arange(n, device=weights.device)
    held = (key < lens[:, None])[:, None]
    always = ((key < sinks) | (key >= lens[:, None] - recent))[:, None]
    rank = torch.where(held, torch.where(always, math.inf, weights), -math.inf)
    order = torch.argsort(rank, dim=-1, descending=True, stable=True)[..., :budget]
    order = torch.where(order < lens[:, None, None], order, n).sort(-1).values
    keep = torch.where(order < n, order, -1)
    if budget > n:
        keep = torch.nn.functional.pad(keep, (0, budget - n), value=-1)
    return keep.to(torch.int32)


def _compact(st):
    c, w = st["case"], st["weights"]
    lens, b = st["lens"].long(), c["block"]
    n = lens.clamp(max=c["budget"])
    i = torch.minimum(torch.arange(c["budget"], device=w.device), n[:, None] - 1)  # past the end: the last row again
    keep = st["keep"].long().gather(2, i[:, None].expand(st["keep"].shape))
    frm = st["tables"].long().gather(1, (keep // b).flatten(1)).view(keep.shape)
    to = st["to"].long().gather(1, i // b)[:, None].expand(keep.shape)
    head = torch.arange(c["kv_heads"], device=w.device)[:, None]
    off = (i % b)[:, None].expand(keep.shape)
    st["k_cache"][to, head, off] = st["k_cache"][frm, head, keep % b]
    st["v_cache"][to, head, off] = st["v_cache"][frm, head, keep % b]
    key = torch.arange(w.shape[2], device=w.device)
    m = min(c["budget"], w.shape[2])
    new = torch.where((key >= n[:, None]) & (key < lens[:, None]), 0.0, 1.0)[:, None] * w
    new[..., :m] = torch.where((key[:m] < n[:, None])[:, None], w.gather(2, keep)[..., :m], new[..., :m])
    w.copy_(new)


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        import paged_kv_cache_247_gb300 as pkv
        if op == "rope":
            pkv.rope_kv_append(st["q_out"], st["q"], st["k"], st["v"], st["positions"], st["inv_freq"],
                               st["k_cache"], st["v_cache"], st["slots"], interleaved=c["interleaved"])
        elif op == "decode":
            pkv.paged_attn_decode_weights(st["out"], st["weights"], st["q"], st["k_cache"], st["v_cache"],
                                          st["tables"], st["lens"], st["scale"], st["max_ctx"], decay=c["decay"])
        elif op == "prefill":
            pkv.paged_attn_prefill_weights(st["out"], st["weights"], st["q"], st["start"], st["k_cache"],
                                           st["v_cache"], st["tables"], st["lens"], st["scale"], st["max_ctx"],
                                           st["max_q"], window=c["window"], decay=c["decay"])
        elif op == "select":
            pkv.kv_evict_select(st["keep"], st["weights"], st["lens"], st["max_ctx"], recent=c["recent"],
                                sinks=c["sinks"])
        else:
            pkv.kv_compact(st["k_cache"], st["v_cache"], st["tables"], st["keep"], st["lens"],
                           weights=st["weights"], dst_tables=st["to"])
    elif op == "rope":
        _rope(st)
    elif op == "decode":
        _decode(st)
    elif op == "prefill":
        _prefill(st)
    elif op == "select":
        st["keep"].copy_(_choose(st["weights"], st["lens"], c["budget"], c["recent"], c["sinks"]))
    else:
        _compact(st)
    if op == "rope":
        return {"q_out": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    if op in ("decode", "prefill"):
        return {"out": st["out"], "weights": st["weights"]}
    if op == "select":
        return {"keep": st["keep"]}
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"], "weights": st["weights"]}


# ---- the same in 64 bits, sequence by sequence -----------------------------------------------------


def _rows(cache, table, n):
    """K or V of one sequence's n positions, [n, H, D] in 64 bits."""
    b = cache.shape[2]
    x = cache[table[:-(-n // b)].long()].double()
    return x.transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])[:n]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        r = case["rot"]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           st["positions"].double()[:, None] * st["inv_freq"])[:, None]
        res = {}
        for name in ("q", "k"):
            x = st[name].double().clone()
            first = x[..., 0:r:2] if case["interleaved"] else x[..., :r // 2]
            second = x[..., 1:r:2] if case["interleaved"] else x[..., r // 2:r]
            z = torch.complex(first.clone(), second.clone()) * turn
            first.copy_(z.real)
            second.copy_(z.imag)
            res[name] = x
        caches = []
        for x, cache in ((res["k"], st["k_cache"]), (st["v"].double(), st["v_cache"])):
            flat = cache.double().transpose(1, 2).reshape(-1, case["kv_heads"], case["dim"]).clone()
            flat[st["slots"]] = x
            caches.append(flat.view(-1, case["block"], case["kv_heads"], case["dim"]).transpose(1, 2))
        return {"q_out": res["q"], "k_cache": caches[0], "v_cache": caches[1]}
    lens = _lens(case)
    weights = st["weights"].double()
    if op == "select":  # whole numbers: one row at a time, by repeated comparison of (weight, position)
        keep = torch.full_like(st["keep"], -1)
        for s, n in enumerate(lens):
            m = min(n, case["budget"])
            lo, hi = min(case["sinks"], n), max(n - case["recent"], 0)
            for h in range(case["kv_heads"]):
                pos = torch.arange(n, device="cuda")
                if n > m:
                    w = weights[s, h, lo:hi]
                    w, at = torch.sort(-w, stable=True)
                    pos = torch.cat((pos[:lo], torch.sort(at[:m - lo - (n - hi)] + lo).values, pos[hi:]))
                keep[s, h, :m] = pos.int()
        return {"keep": keep}
    if op == "compact":
        k, v = st["k_cache"].double(), st["v_cache"].double()
        b = case["block"]
        for s, n in enumerate(lens):
            m = min(n, case["budget"])
            at = torch.arange(m, device="cuda")
            for h in range(case["kv_heads"]):
                src = st["keep"][s, h, :m].long()
                for new, old in ((k, st["k_cache"]), (v, st["v_cache"])):
                    new[st["to"][s].long()[at // b], h, at % b] = old[st["tables"][s].long()[src // b], h, src % b].double()
                kept = weights[s, h, src]
                weights[s, h, :n] = 0
                weights[s, h, :m] = kept
        return {"k_cache": k, "v_cache": v, "weights": weights}
    h, hq = case["kv_heads"], case["heads"]
    queries = _chunks(case) if op == "prefill" else [1] * len(lens)
    if sum(l * n for l, n in zip(queries, lens)) * hq * case["dim"] > 4e12:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for s, (l, n) in enumerate(zip(queries, lens)):
        k, v = _rows(st["k_cache"], st["tables"][s], n), _rows(st["v_cache"], st["tables"][s], n)
        hidden = torch.arange(n, device="cuda") > torch.arange(n - l, n, device="cuda")[:, None]
        counted = l if not case.get("window") else min(l, case["window"])
        for i in range(h):
            q = st["q"][row:row + l, i * (hq // h):(i + 1) * (hq // h)].double()
            p = torch.softmax((torch.einsum("lgd,nd->gln", q, k[:, i]) * st["scale"]).masked_fill(hidden, -math.inf), -1)
            out[row:row + l, i * (hq // h):(i + 1) * (hq // h)] = torch.einsum("gln,nd->lgd", p, v[:, i])
            weights[s, i, :n] = case["decay"] * weights[s, i, :n] + p[:, l - counted:].sum((0, 1))
        row += l
    return {"out": out, "weights": weights}
