"""The operators of a paged cache held in 8 bits, as a program uses them: the cases that are
measured, their inputs, the plain form of each operator in elementary torch operations, and its
value in 64 bits.

A cache row (one token, one KV head) is held as e4m3 codes and one scale, the smallest power of
two 2^e (e >= -126) for which no element of the row is above 448 * 2^e.  A layer's step normalises
and turns the heads of q and k (qk_norm_rope), quantises k and v into their slots
(kv_append_fp8) and attends over the cache with one query per sequence (paged_attn_decode_fp8) or
with a tree of drafted tokens (paged_attn_tree_fp8).  Prompt chunks read cached blocks back into
16 bits (block_read_fp8) for the attention that takes those.
"""

import math
import random

import torch

own = False  # true: run() calls the framework's operators

_DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
_E4M3 = torch.float8_e4m3fn


# ---- cases ---------------------------------------------------------------------------------------


def listed():
    return [
        # a decode step of 64 sequences, grouped heads, slices of the joint projection: latency only
        {"name": "append_step_64", "op": "append", "tokens": 64, "kv_heads": 8, "dim": 128, "block": 16,
         "dtype": "bf16", "packed": True, "padding": 0.0},
        # prompt chunks of 8 x 2,048 tokens
        {"name": "append_prompt_16k", "op": "append", "tokens": 16384, "kv_heads": 8, "dim": 128, "block": 16,
         "dtype": "bf16", "packed": True, "padding": 0.0},
        # the cached prefix of one short prompt on a small model: latency only
        {"name": "read_1x600", "op": "read", "blocks": 38, "kv_heads": 8, "dim": 64, "block": 16, "dtype": "fp16"},
        # the cached prefixes of 8 prompts of 4,096 tokens
        {"name": "read_8x4k", "op": "read", "blocks": 2048, "kv_heads": 8, "dim": 128, "block": 16,
         "dtype": "bf16"},
        # a decode step of 64 sequences: latency
        {"name": "norm_rope_step_64", "op": "norm_rope", "tokens": 64, "heads": 32, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "rot": 128, "interleaved": False, "axes": 1, "norm": True, "packed": True,
         "far": 8192},
        # 16k tokens of images: time, height and width turn a part of the pairs each
        {"name": "norm_rope_image_16k", "op": "norm_rope", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "rot": 128, "interleaved": False, "axes": 3, "norm": True, "packed": True,
         "far": 4096},
        # a handful of short conversations on a small model: latency only
        {"name": "decode_4_short", "op": "decode", "seqs": 4, "heads": 8, "kv_heads": 8, "dim": 64,
         "block": 16, "dtype": "fp16", "lo": 1, "hi": 200, "shape": 1},
        # 64 requests of lengths around 500 over 40 single heads
        {"name": "decode_64_mha", "op": "decode", "seqs": 64, "heads": 40, "kv_heads": 40, "dim": 128,
         "block": 16, "dtype": "fp16", "lo": 16, "hi": 2048, "shape": 2},
        # 64 long conversations over grouped heads
        {"name": "decode_64x8k", "op": "decode", "seqs": 64, "heads": 32, "kv_heads": 8, "dim": 128,
         "block": 16, "dtype": "bf16", "lo": 8192, "hi": 8192, "shape": 3},
        # four short conversations, a chain of at most five drafted tokens each: latency
        {"name": "tree_4_chains", "op": "tree", "seqs": 4, "heads": 32, "kv_heads": 8, "dim": 64, "block": 16,
         "dtype": "bf16", "lo": 20, "hi": 600, "drafts": 5, "branch": 1, "shape": 4},
        # 8 sequences of odd lengths with the widest trees, groups of three heads
        {"name": "tree_8_wide", "op": "tree", "seqs": 8, "heads": 36, "kv_heads": 12, "dim": 128, "block": 32,
         "dtype": "fp16", "lo": 500, "hi": 2000, "drafts": 64, "branch": 4, "shape": 5},
        # 32 conversations of 4k, trees of 16 drafted tokens
        {"name": "tree_32x4k", "op": "tree", "seqs": 32, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16,
         "dtype": "bf16", "lo": 4096, "hi": 4096, "drafts": 16, "branch": 3, "shape": 6},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "norm_rope", "decode", "decode", "tree", "tree"])
    dim, block = rng.choice([64, 128]), rng.choice([8, 16, 32, 64, 128])
    dtype = rng.choice(["fp16", "bf16"])
    kv = rng.choice([1, 2, 4, 5, 8, 12, 40])
    shape = rng.randrange(1 << 20)
    if op == "append":
        return {"op": op, "tokens": _log_int(rng, 1, min(16384, 16384 * 8 // kv)), "kv_heads": kv, "dim": dim,
                "block": block, "dtype": dtype, "packed": rng.random() < 0.5, "padding": rng.choice([0.0, 0.1])}
    if op == "read":
        return {"op": op, "blocks": _log_int(rng, 1, 32768 * 8 // (kv * block)), "kv_heads": kv, "dim": dim,
                "block": block, "dtype": dtype}
    if op == "norm_rope":
        heads = kv * rng.choice([1, 2, 3, 4, 7, 8])
        while heads > 64:
            heads -= kv
        return {"op": op, "tokens": _log_int(rng, 1, min(16384, 16384 * 40 // (heads + kv))), "heads": heads,
                "kv_heads": kv, "dim": dim, "dtype": dtype,
                "rot": rng.choice([dim, dim // 2, 32, 2 * rng.randrange(1, dim // 2 + 1)]),
                "interleaved": rng.random() < 0.5, "axes": rng.choice([1, 1, 2, 3]), "norm": rng.random() < 0.8,
                "packed": rng.random() < 0.5, "far": _log_int(rng, 1 << 8, 1 << 21)}
    case = {"op": op, "seqs": 0, "heads": 0, "kv_heads": kv, "dim": dim, "block": block, "dtype": dtype}
    if op == "decode":
        group = rng.choice([1, 2, 3, 4, 7, 8, 16, 32, 40])
        hi = _log_int(rng, 1, 32768)
        most = 64 * 8192 * 8 * 128 // (hi * kv * dim * max(1, group // 4))  # codes of K, and the plain form's logits
        case.update(lo=rng.choice([1, hi, max(1, hi // 3)]), hi=hi)
    else:
        group = rng.choice([1, 2, 3, 4, 7, 8])
        hi = _log_int(rng, 2, 16384)
        drafts = min(hi, rng.choice([1, 2, 3, 5, 8, 16, 17, 33, 64]))
        most = 32 * 4096 * 8 * 128 * 4 * 16 // (hi * kv * dim * max(16, group * drafts))
        while most < 1:
            hi //= 2
            drafts = min(hi, drafts)
            most = 32 * 4096 * 8 * 128 * 4 * 16 // (hi * kv * dim * max(16, group * drafts))
        case.update(lo=rng.choice([1, hi, max(1, hi // 3)]), hi=hi, drafts=drafts, branch=rng.choice([1, 2, 4]))
    case.update(seqs=_log_int(rng, 1, max(1, min(128, most))), heads=kv * group, shape=shape)
    return case


def _lens(case):
    """Context lengths, spread over their logarithm; a case's lengths do not depend on its inputs' seed."""
    rng = random.Random(case["shape"])
    if case["lo"] == case["hi"]:
        return [case["hi"]] * case["seqs"]
    return [case["hi"]] + [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["seqs"] - 1)]


def _drafts(case):
    """Drafted tokens of each sequence: the last of its context."""
    rng = random.Random(case["shape"] + 1)
    return [min(n, case["drafts"] if i == 0 else rng.randint((case["drafts"] + 1) // 2, case["drafts"]))
            for i, n in enumerate(_lens(case))]


def work(case):
    op, h, d = case["op"], case.get("kv_heads"), case["dim"]
    if op == "append":  # 16-bit rows in; codes and a scale out
        return {"bytes": case["tokens"] * (2 * h * (3 * d + 2) + 8), "flops": 0}
    if op == "read":
        return {"bytes": case["blocks"] * (2 * h * case["block"] * (3 * d + 2) + 16), "flops": 0}
    if op == "norm_rope":
        t, hq = case["tokens"], case["heads"]
        return {"bytes": t * (hq + h) * d * 4 + 4 * t * case["axes"] + 4 * case["rot"] + 4 * d,
                "flops": t * (hq + h) * (4 * d + 3 * case["rot"])}
    lens, hq = _lens(case), case["heads"]
    n = sum(lens)
    rows = sum(_drafts(case)) if op == "tree" else case["seqs"]
    tables = 4 * sum(-(-x // case["block"]) for x in lens)
    pairs = sum(l * x for l, x in zip(_drafts(case), lens)) if op == "tree" else n
    return {"bytes": n * h * 2 * (d + 2) + 4 * rows * hq * d + tables + (8 * rows if op == "tree" else 0),
            "flops": 4 * pairs * hq * d}


# ---- inputs --------------------------------------------------------------------------------------


def _tables(case, lens, gen):
    """Block tables over one pool in random order."""
    b = case["block"]
    per = torch.tensor([-(-x // b) for x in lens], device="cuda")
    width, total = int(max(-(-x // b) for x in lens)), int(sum(-(-x // b) for x in lens))
    pool = total + total // 8 + 1
    perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    first = torch.cumsum(per, 0) - per
    col = torch.arange(width, device="cuda")
    held = col < per[:, None]
    return pool, torch.where(held, perm[torch.where(held, first[:, None] + col, 0)], -1).to(torch.int32)


def _rows_like(shape, gen, dt):
    """Rows as projections give them: some larger than others, each with a heavy element now and then."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=dt)
    x *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=gen, device="cuda")).to(dt)
    return x


def _cache(case, pool, gen):
    """A pool that holds quantised rows everywhere: (codes, scales) of K and of V."""
    shape = (pool, case["kv_heads"], case["block"], case["dim"])
    k, ks = _quantise(_rows_like(shape, gen, _DTYPES[case["dtype"]]))
    v, vs = _quantise(_rows_like(shape, gen, _DTYPES[case["dtype"]]))
    return k, v, ks, vs


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], _DTYPES[case["dtype"]]
    st = {"case": case}
    if op == "append":
        t, h, d, b = case["tokens"], case["kv_heads"], case["dim"], case["block"]
        if case["packed"]:  # the projection's output, one row per token, with as many heads of q
            qkv = _rows_like((t, 3 * h, d), gen, dt)
            st["k"], st["v"] = qkv[:, h:2 * h], qkv[:, 2 * h:]
        else:
            st["k"], st["v"] = _rows_like((t, h, d), gen, dt), _rows_like((t, h, d), gen, dt)
        pool = -(-t // b) + 8
        slots = torch.randperm(pool * b, generator=gen, device="cuda")[:t]
        padding = torch.rand((t,), generator=gen, device="cuda") < case["padding"]
        st["slots"] = torch.where(padding, -1, slots)
        st["k_cache"] = torch.zeros((pool, h, b, d), dtype=_E4M3, device="cuda")
        st["v_cache"] = torch.zeros_like(st["k_cache"])
        st["k_scales"] = torch.zeros((pool, h, b, 1), dtype=torch.bfloat16, device="cuda")
        st["v_scales"] = torch.zeros_like(st["k_scales"])
        return st
    if op == "read":
        n, h, d, b = case["blocks"], case["kv_heads"], case["dim"], case["block"]
        pool = n + n // 8 + 1
        st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"] = _cache(case, pool, gen)
        src = torch.randperm(pool, generator=gen, device="cuda")[:n]
        st["pairs"] = torch.stack((src, torch.arange(n, device="cuda")), 1).contiguous()
        st["k_out"] = torch.zeros((n, h, b, d), dtype=dt, device="cuda")
        st["v_out"] = torch.zeros_like(st["k_out"])
        return st
    if op == "norm_rope":
        t, hq, h, d, a = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["axes"]
        if case["packed"]:
            qkv = _rows_like((t, hq + 2 * h, d), gen, dt)
            st["q"], st["k"] = qkv[:, :hq], qkv[:, hq:hq + h]
        else:
            st["q"], st["k"] = _rows_like((t, hq, d), gen, dt), _rows_like((t, h, d), gen, dt)
        st["q_out"] = torch.empty((t, hq, d), dtype=dt, device="cuda")
        st["k_out"] = torch.empty((t, h, d), dtype=dt, device="cuda")
        st["q_weight"] = st["k_weight"] = None
        if case["norm"]:
            st["q_weight"], st["k_weight"] = [
                (1.0 + 0.2 * torch.randn((d,), generator=gen, device="cuda")).to(dt) for _ in range(2)]
        st["positions"] = torch.randint(0, case["far"], (a, t), generator=gen, device="cuda", dtype=torch.int32)
        pairs = case["rot"] // 2
        st["axes"] = None if a == 1 else [i * a // pairs for i in range(pairs)]  # a section of the pairs each
        if a == 1:
            st["positions"] = st["positions"][0]
        st["inv_freq"] = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        return st
    lens = _lens(case)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["max_ctx"] = max(lens)
    pool, st["tables"] = _tables(case, lens, gen)
    st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"] = _cache(case, pool, gen)
    st["scale"] = case["dim"] ** -0.5
    rows = case["seqs"]
    if op == "tree":
        count = _drafts(case)
        rows, st["max_q"] = sum(count), max(count)
        st["start"] = torch.tensor([0] + count, device="cuda").cumsum(0).to(torch.int32)
        # drafted token j grows from one of the `branch` before it; it sees its ancestors and itself
        grid = torch.zeros((case["seqs"], st["max_q"]), dtype=torch.int64, device="cuda")
        for j in range(st["max_q"]):
            back = torch.randint(1, case["branch"] + 1, (case["seqs"],), generator=gen, device="cuda")
            parent = grid.gather(1, (j - back).clamp(min=0)[:, None])[:, 0]
            bit = (1 << j) if j < 63 else -(1 << 63)
            grid[:, j] = torch.where(back <= j, parent, 0) | bit
        there = torch.arange(st["max_q"], device="cuda") < torch.tensor(count, device="cuda")[:, None]
        st["masks"] = grid[there]
    # queries that attend unevenly: logits of standard deviation around 2
    st["q"] = 2.0 * torch.randn((rows, case["heads"], case["dim"]), generator=gen, device="cuda", dtype=dt)
    st["out"] = torch.empty_like(st["q"])
    return st


# ---- the operators, plain or the framework's ------------------------------------------------------


def _quantise(x):
    """Codes and scales of rows: exact, powers of two apart from the one rounding to e4m3."""
    x = x.float()
    top = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1), and 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(top > 0, e, -126).clamp(min=-126)
    scale = torch.ldexp(torch.ones_like(top), e)
    return (x / scale).to(_E4M3), scale.to(torch.bfloat16)


def _append(st):
    b = st["case"]["block"]
    t = torch.nonzero(st["slots"] >= 0)[:, 0]
    blk, off = st["slots"][t] // b, st["slots"][t] % b
    k, ks = _quantise(st["k"][t])
    v, vs = _quantise(st["v"][t])
    st["k_cache"].view(torch.uint8)[blk, :, off] = k.view(torch.uint8)
    st["v_cache"].view(torch.uint8)[blk, :, off] = v.view(torch.uint8)
    st["k_scales"][blk, :, off] = ks
    st["v_scales"][blk, :, off] = vs


def _read(st):
    src, dst = st["pairs"][:, 0], st["pairs"][:, 1]
    k = st["k_cache"].view(torch.uint8)[src].view(_E4M3).float() * st["k_scales"][src].float()
    v = st["v_cache"].view(torch.uint8)[src].view(_E4M3).float() * st["v_scales"][src].float()
    st["k_out"][dst] = k.to(st["k_out"].dtype)
    st["v_out"][dst] = v.to(st["v_out"].dtype)


def _norm_rotate(x, weight, eps, cos, sin, rot, interleaved):
    x = x.float()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _norm_rope(st):
    c = st["case"]
    pos = st["positions"].double()  # 64 bits: positions are far
    if c["axes"] > 1:
        pos = pos[st["axes"]].t()  # the position that turns each pair, [tokens, pairs]
    else:
        pos = pos[:, None]
    angle = pos * st["inv_freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    st["q_out"].copy_(_norm_rotate(st["q"], st["q_weight"], 1e-6, cos, sin, c["rot"], c["interleaved"]))
    st["k_out"].copy_(_norm_rotate(st["k"], st["k_weight"], 1e-6, cos, sin, c["rot"], c["interleaved"]))


def _gather(cache, scales, tables):
    """[S, H, tokens, D] in 32 bits, through the tables."""
    at = tables.clamp(min=0).long()
    x = cache.view(torch.uint8)[at].view(_E4M3).float() * scales[at].float()
    s, n, h, b, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(s, h, n * b, d)


def _softmax(x):
    x = torch.exp(x - x.amax(-1, keepdim=True))
    return x / x.sum(-1, keepdim=True)


def _decode(st):
    q, lens = st["q"], st["lens"]
    s, hq, d = q.shape
    k = _gather(st["k_cache"], st["k_scales"], st["tables"])
    v = _gather(st["v_cache"], st["v_scales"], st["tables"])
    h = k.shape[1]
    seen = torch.arange(k.shape[2], device=q.device) < lens[:, None]
    x = (q.float().view(s, h, hq // h, d) @ k.transpose(-1, -2)) * st["scale"]
    p = _softmax(torch.where(seen[:, None, None], x, -math.inf))
    st["out"].copy_((p @ v).view(s, hq, d))


def _tree(st):
    q, lens, start = st["q"], st["lens"].long(), st["start"].long()
    t, hq, d = q.shape
    k = _gather(st["k_cache"], st["k_scales"], st["tables"])
    v = _gather(st["v_cache"], st["v_scales"], st["tables"])
    s, h, n, _ = k.shape
    count = start[1:] - start[:-1]
    j = torch.arange(st["max_q"], device=q.device)
    there = j < count[:, None]
    rows = torch.where(there, start[:-1, None] + j, 0)
    qp = q[rows].float().view(s, st["max_q"], h, hq // h, d).permute(0, 2, 3, 1, 4)
    x = (qp @ k[:, :, None].transpose(-1, -2)) * st["scale"]
    at = torch.arange(n, device=q.device) - (lens - count)[:, None]  # below 0: the context before the drafts
    bits = (st["masks"][rows][:, :, None] >> at.clamp(0, 63)[:, None]) & 1
    drafted = (bits == 1) & (at < count[:, None])[:, None]
    seen = (at < 0)[:, None] | drafted | ((at == 0)[:, None] & ~there[:, :, None])  # (a row that is none sees one)
    p = _softmax(torch.where(seen[:, None, None], x, -math.inf))
    o = (p @ v[:, :, None]).permute(0, 3, 1, 2, 4).reshape(s, st["max_q"], hq, d)
    st["out"].copy_(o[there])


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        import paged_kv_cache_247_gb300 as pkv
        if op == "append":
            pkv.kv_append_fp8(st["k"], st["v"], st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"],
                              st["slots"])
        elif op == "read":
            pkv.block_read_fp8(st["k_out"], st["v_out"], st["k_cache"], st["v_cache"], st["k_scales"],
                               st["v_scales"], st["pairs"])
        elif op == "norm_rope":
            pkv.qk_norm_rope(st["q_out"], st["k_out"], st["q"], st["k"], st["positions"], st["inv_freq"],
                             q_weight=st["q_weight"], k_weight=st["k_weight"], eps=1e-6, pair_axes=st["axes"],
                             interleaved=c["interleaved"])
        elif op == "decode":
            pkv.paged_attn_decode_fp8(st["out"], st["q"], st["k_cache"], st["v_cache"], st["k_scales"],
                                      st["v_scales"], st["tables"], st["lens"], st["scale"], st["max_ctx"])
        else:
            pkv.paged_attn_tree_fp8(st["out"], st["q"], st["start"], st["masks"], st["k_cache"], st["v_cache"],
                                    st["k_scales"], st["v_scales"], st["tables"], st["lens"], st["scale"],
                                    st["max_ctx"], st["max_q"])
    elif op == "append":
        _append(st)
    elif op == "read":
        _read(st)
    elif op == "norm_rope":
        _norm_rope(st)
    elif op == "decode":
        _decode(st)
    else:
        _tree(st)
    if op == "append":
        return {n: st[n] for n in ("k_cache", "v_cache", "k_scales", "v_scales")}
    if op == "read":
        return {"k_out": st["k_out"], "v_out": st["v_out"]}
    if op == "norm_rope":
        return {"q_out": st["q_out"], "k_out": st["k_out"]}
    return {"out": st["out"]}


# ---- the same in 64 bits --------------------------------------------------------------------------


def _round_e4m3(y):
    """The nearest value of e4m3 (ties to even) to |y| <= 448, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _scales_of(x):
    """The smallest power of two (from 2^-126) that brings a row to at most 448."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -126)))
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)  # (log2 may be off by a rounding)
    e = torch.where((top <= 448 * torch.exp2(e - 1)) & (e > -126), e - 1, e)
    return torch.exp2(e)


def _positions_of(cache, scales, table, n):
    """One sequence's n positions, [n, H, D] in 64 bits."""
    at = table[:-(-n // cache.shape[2])].long()
    x = cache.view(torch.uint8)[at].view(_E4M3).double() * scales[at].double()
    return x.transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])[:n]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "append":
        res = {}
        for name in ("k", "v"):
            x = st[name].double()
            scale = _scales_of(x)
            there = st["slots"] >= 0
            for part, value in (("cache", _round_e4m3(x / scale)), ("scales", scale)):
                held = st[f"{name}_{part}"].double().transpose(1, 2)  # [pool, block, H, ...]
                shape = held.shape
                flat = held.reshape(-1, *shape[2:]).clone()
                flat[st["slots"][there]] = value[there]
                res[f"{name}_{part}"] = flat.view(shape).transpose(1, 2)
        return res
    if op == "read":
        res = {}
        for name in ("k", "v"):
            x = st[f"{name}_out"].double()
            for lo in range(0, case["blocks"], 4096):
                src, dst = st["pairs"][lo:lo + 4096].t()
                x[dst] = st[f"{name}_cache"].double()[src] * st[f"{name}_scales"].double()[src]
            res[f"{name}_out"] = x
        return res
    if op == "norm_rope":
        r, d = case["rot"], case["dim"]
        pos = st["positions"].double()
        pos = pos[:, None].expand(-1, r // 2) if case["axes"] == 1 else torch.stack([pos[a] for a in st["axes"]], 1)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos * st["inv_freq"])[:, None]
        res = {}
        for name in ("q", "k"):
            x = st[name].double()
            if st[f"{name}_weight"] is not None:
                x = x * st[f"{name}_weight"].double() * (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / d +
                                                         1e-6) ** -0.5
            x = x.clone()
            first = x[..., 0:r:2] if case["interleaved"] else x[..., :r // 2]
            second = x[..., 1:r:2] if case["interleaved"] else x[..., r // 2:r]
            z = torch.complex(first.clone(), second.clone()) * turn
            first.copy_(z.real)
            second.copy_(z.imag)
            res[f"{name}_out"] = x
        return res
    lens, h, hq = _lens(case), case["kv_heads"], case["heads"]
    queries = _drafts(case) if op == "tree" else [1] * len(lens)
    if sum(l * n for l, n in zip(queries, lens)) * hq * case["dim"] > 2e12 or len(lens) * h > 20000:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for s, (l, n) in enumerate(zip(queries, lens)):
        k = _positions_of(st["k_cache"], st["k_scales"], st["tables"][s], n)
        v = _positions_of(st["v_cache"], st["v_scales"], st["tables"][s], n)
        hidden = torch.zeros((l, n), dtype=torch.bool, device="cuda")
        if op == "tree":
            sees = [[(m >> i) & 1 == 0 for i in range(l)] for m in st["masks"][row:row + l].tolist()]
            hidden[:, n - l:] = torch.tensor(sees, device="cuda")
        q = st["q"][row:row + l].double().view(l, h, hq // h, case["dim"])
        x = torch.einsum("lhgd,nhd->hgln", q, k) * st["scale"]
        p = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
        out[row:row + l] = torch.einsum("hgln,nhd->lhgd", p, v).reshape(l, hq, case["dim"])
        row += l
    return {"out": out}
