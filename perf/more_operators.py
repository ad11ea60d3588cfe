"""Attention over prompts packed one after the other, and the cache in 8 bits that their keys
and values go into, as they are measured: cases, inputs, plain forms, 64-bit definitions.

* ``prompts`` / ``prompts_bwd``: attention of packed sequences of different lengths, grouped
  heads, with or without keys cached before the first query, and its gradients.
* ``append8``: new keys and values into a paged cache of 8 bits a value, with a scale for each
  block of 16 tokens and head, and what those blocks hold afterwards.
* ``decode8``: attention of each request's newest tokens over its 8-bit cache.

With ``own`` false ``run`` computes them from elementary torch operations; with ``own``
true it makes the calls of ``exact_io_aware_26_gb300``.

A block of the cache (``block_bytes(d)`` bytes) holds 16 tokens of one head:
    int8   keys    [16][d]                 at d = 128 the halves of odd tokens' rows change places
    int8   values  [d / 4][4][4][4]        channel c of token j at [c / 4][j / 4][c % 4][j % 4]
    float  scale of the keys, scale of the values: 0 or powers of two
    uint16 tokens with a NaN key, tokens with a NaN value (bit j: token j); 4 bytes of 0
A code times its scale is the value.  Tokens that join a block may raise its scale; the
codes that were there are then rounded to the new one.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 16        # tokens of a cache block
SATURATE = 16384  # quantised values saturate here
LEAST = -64       # least exponent of a scale that is not 0
MOST_PAIRS = 12 * 16384 * 16384 // 6 * 32 * 128  # (query, key) pairs x heads x channels of the largest case


def listed():
    return [
        # serving: three short prompts, where latency counts
        dict(name="prompts_short", op="prompts", R=3, Hq=32, Hk=8, d=128, dtype="f16", least=1, most=32, prefix=0,
             causal=True, lens=1),
        # training: four sequences of up to 2048 tokens in place of a padded batch
        dict(name="prompts_n2048", op="prompts", R=4, Hq=12, Hk=12, d=64, dtype="bf16", least=1024, most=2048, prefix=0,
             causal=True, lens=2),
        # serving: prompts of very different lengths, four query heads per key head
        dict(name="prompts_n16384", op="prompts", R=12, Hq=32, Hk=8, d=128, dtype="bf16", least=1, most=16384, prefix=0,
             causal=True, lens=3),
        # serving: pieces of up to 512 rows of prompts whose first part, up to 8192 tokens, is cached
        dict(name="prompts_prefix", op="prompts", R=8, Hq=16, Hk=2, d=128, dtype="bf16", least=1, most=512, prefix=8192,
             causal=True, lens=4),
        # training, backward: the sequences of up to 2048 tokens
        dict(name="prompts_bwd_n2048", op="prompts_bwd", R=4, Hq=12, Hk=12, d=64, dtype="bf16", least=1024, most=2048,
             prefix=0, causal=True, lens=2),
        # training, backward: long and short documents, four query heads per key head
        dict(name="prompts_bwd_n8192", op="prompts_bwd", R=12, Hq=32, Hk=8, d=128, dtype="bf16", least=1, most=8192,
             prefix=0, causal=True, lens=5),
        # serving: the newest token of 256 requests into the cache, into blocks that hold others
        dict(name="append8_tokens", op="append8", R=256, H=8, d=128, dtype="bf16", page=64, least=1, most=1, held=200,
             lens=6),
        # serving: a trading day as one prompt
        dict(name="append8_day", op="append8", R=1, H=12, d=64, dtype="bf16", page=64, least=23400, most=23400, held=0,
             lens=7),
        # serving: the next token after a trading day, a key head for each query head
        dict(name="decode8_day", op="decode8", R=1, Hq=12, Hk=12, d=64, dtype="bf16", page=64, least=23400, most=23400,
             q_len=1, window=0, lens=1),
        # serving: a few short contexts, where latency counts
        dict(name="decode8_n2048", op="decode8", R=4, Hq=12, Hk=12, d=64, dtype="f16", page=16, least=1, most=2048,
             q_len=1, window=0, lens=2),
        # serving: a full batch of ragged long contexts, four query heads per key head
        dict(name="decode8_n16384", op="decode8", R=64, Hq=32, Hk=8, d=128, dtype="bf16", page=64, least=512, most=16384,
             q_len=1, window=0, lens=3),
        # serving: up to four draft tokens checked at once, in a window of the context
        dict(name="decode8_drafts", op="decode8", R=16, Hq=16, Hk=2, d=128, dtype="bf16", page=32, least=1, most=8192,
             q_len=4, window=4096, lens=4),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompts", "prompts", "prompts_bwd", "prompts_bwd", "append8", "decode8", "decode8"])
    d, hk = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8, 12])
    dtype, page = rng.choice(["bf16", "f16"]), rng.choice([16, 32, 64, 128])
    if op in ("prompts", "prompts_bwd"):
        hq = hk * rng.choice([1, 1, 2, 4, 5, 8])
        budget = MOST_PAIRS // (2 if op == "prompts" else 8) // (hq * d)  # pairs
        R, prefix = _log(rng, 1, 64), rng.choice([0, 0, _log(rng, 1, 8192)])
        most = _log(rng, 1, 16384)
        while R > 1 and R * most * (most + prefix) > budget:
            R = (R + 1) // 2
        while most > 1 and R * most * (most + prefix) > budget:
            most = most * 3 // 4
        return dict(op=op, R=R, Hq=hq, Hk=hk, d=d, dtype=dtype, least=rng.randint(0, most), most=most, prefix=prefix,
                    causal=rng.random() < 0.85, lens=rng.randrange(1 << 20))
    if op == "append8":
        most = _log(rng, 1, 24000)
        R = _log(rng, 1, max(1, min(300, 24000 // most)))
        return dict(op=op, R=R, H=hk, d=d, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), page=page,
                    least=rng.randint(1, most), most=most, held=rng.choice([0, _log(rng, 1, 500)]), lens=rng.randrange(1 << 20))
    most = _log(rng, 1, 30000)
    R = _log(rng, 1, max(1, min(300, 64 * 16384 * 8 * 128 // (2 * hk * d * most))))
    q_len = rng.choice([1, 1, 1, 2, 5, 8])
    return dict(op="decode8", R=R, Hq=hk * rng.choice([1, 2, 4, 5, 8]), Hk=hk, d=d, dtype=dtype, page=page,
                least=rng.randint(0, most), most=most, q_len=q_len, window=rng.choice([0, 0, rng.randint(1, most)]),
                lens=rng.randrange(1 << 20))


# ---------------------------------------------------------------- inputs


def _lengths(case):
    """Lengths of each request, part of the case and not of the seed: (queries, keys) of
    prompts, (new tokens, held tokens) of append8, (cached tokens, new ones) of decode8."""
    r, R = random.Random(case["lens"]), range(case["R"])
    first = [r.randint(case["least"], case["most"]) for _ in R]
    if case["op"] == "append8":
        return first, [r.randint(0, case["held"]) for _ in R]
    if case["op"] == "decode8":
        return first, [r.randint(1, case["q_len"]) for _ in R]
    if max(first) == 0:
        first[0] = 1
    return first, [n + r.randint(0, case["prefix"]) for n in first]


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def block_bytes(d):
    """Bytes of one cache block: 16 tokens' key codes, value codes, scales and marks."""
    return 2 * BLOCK * d + 16


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dev, d = case["op"], "cuda", case["d"]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    s, dt = dict(case), DTYPES[case["dtype"]]
    if op in ("prompts", "prompts_bwd"):
        new, keys = _lengths(case)
        s["new"], s["keys"] = new, keys
        s["cu_q"], s["cu_k"] = ints(_starts(new)), ints(_starts(keys))
        s["scale"] = 1.0 / math.sqrt(d)
        s["q"] = normal(sum(new), case["Hq"], d, dtype=dt)
        packed = normal(sum(keys), 2 * case["Hk"], d, dtype=dt)  # one projection: keys, values
        s["k"], s["v"] = packed[:, :case["Hk"]], packed[:, case["Hk"]:]
        if op == "prompts_bwd":
            s["do"] = normal(sum(new), case["Hq"], d, dtype=dt)
            s["o"], s["lse"] = _prompts_plain(s)
    elif op == "append8":
        H, page = case["H"], case["page"]
        new, held = _lengths(case)
        pages_of = [(h + n + page - 1) // page for n, h in zip(new, held)]
        pages = sum(pages_of) + 3
        order = torch.randperm(pages, generator=g, device=dev)
        first = _starts(pages_of)

        def slots(r, a, b):  # of tokens a .. b - 1 of request r
            t = torch.arange(a, b, device=dev)
            return order[first[r] + t // page] * page + t % page

        s["slots"] = torch.cat([slots(r, h, h + n) for r, (n, h) in enumerate(zip(new, held))]).to(torch.int32)
        # what the blocks that get new tokens hold afterwards
        s["back"] = torch.cat([slots(r, h // BLOCK * BLOCK, h + n) for r, (n, h) in enumerate(zip(new, held))]).to(torch.int32)
        packed = normal(sum(new), 2 * H, d, dtype=dt)
        s["k"], s["v"] = packed[:, :H], packed[:, H:]
        s["cache"] = _full_cache(pages, H, page, d, lambda *shape: 0.5 * normal(*shape))
    else:
        R, Hq, Hk, page = (case[k] for k in ("R", "Hq", "Hk", "page"))
        kv, new = _lengths(case)
        have = [(n + page - 1) // page for n in kv]
        pages, width = sum(have) + 1, max(max(have), 1)
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        table = torch.full((R, width), -1, dtype=torch.int32)
        for r, (at, h) in enumerate(zip(_starts(have), have)):
            table[r, :h] = torch.arange(at, at + h, dtype=torch.int32)
        table = table.to(dev)
        s["block_table"] = torch.where(table >= 0, order[table.clamp(min=0).long()], -1).to(torch.int32)
        s["kv_lens"], s["cu_q"] = ints(kv), ints(_starts(new))
        s["q"] = normal(sum(new), Hq, d, dtype=dt)
        s["scale"] = 1.0 / math.sqrt(d)
        s["cache"] = _full_cache(pages, Hk, page, d, normal)
    return s


# ---------------------------------------------------------------- the cache's format


def _full_cache(pages, H, page, d, values):
    """A cache whose every token holds a value."""
    cache = torch.zeros(pages, H, page // BLOCK, block_bytes(d), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (H * page * d))
    for a in range(0, pages, step):
        part = cache[a:a + step]
        sides = [values(part.shape[0], H, page // BLOCK, BLOCK, d) for _ in (0, 1)]
        scales = [_scale_for(x.abs().amax((-1, -2))) for x in sides]
        codes = [_codes_for(x, sc[..., None, None]) for x, sc in zip(sides, scales)]
        part.copy_(_block(codes[0], codes[1], scales[0], scales[1]))
    return cache


def _scale_for(most):
    """The least power of two that brings magnitudes of up to ``most`` to 127; 0 for 0."""
    m, e = torch.frexp(most.float())
    e = torch.where(m <= 127 / 128, e - 7, e - 6).clamp(min=LEAST)
    return torch.where(most > 0, ((e + 127) << 23).to(torch.int32).view(torch.float32), 0.0)  # 2^e


def _codes_for(x, scale):
    return torch.where(scale > 0, torch.round(x / torch.where(scale > 0, scale, 1.0)), 0.0).to(torch.int8)


def _turn(keys):
    """Key rows [.., 16, d] with the halves of odd tokens in each other's place (its own inverse)."""
    if keys.shape[-1] < 128:
        return keys
    out = keys.clone()
    out[..., 1::2, :] = keys[..., 1::2, :].roll(keys.shape[-1] // 2, -1)
    return out


def _block(k, v, ks, vs):
    """Block bytes of codes [.., 16, d] and scales [..]."""
    d, lead = k.shape[-1], k.shape[:-2]
    vt = v.unflatten(-2, (4, 4)).unflatten(-1, (d // 4, 4)).movedim(-2, -4).transpose(-1, -2)  # [.., c / 4, j / 4, c % 4, j % 4]
    tail = torch.stack([ks, vs, torch.zeros_like(ks), torch.zeros_like(ks)], -1).view(torch.uint8)
    return torch.cat([_turn(k).reshape(*lead, -1).view(torch.uint8), vt.reshape(*lead, -1).contiguous().view(torch.uint8), tail], -1)


def _unblock(blocks):
    """(key codes, value codes) [.., 16, d] int8 and (key scales, value scales) [..] of block bytes."""
    n = (blocks.shape[-1] - 16) // 2
    d, lead = n // BLOCK, blocks.shape[:-1]
    k = _turn(blocks[..., :n].contiguous().view(torch.int8).reshape(*lead, BLOCK, d))
    v = blocks[..., n:2 * n].contiguous().view(torch.int8).reshape(*lead, d // 4, 4, 4, 4)  # c / 4, j / 4, c % 4, j % 4
    v = v.transpose(-1, -2).movedim(-4, -2).reshape(*lead, BLOCK, d)
    tail = blocks[..., 2 * n:2 * n + 8].contiguous().view(torch.float32)
    return k, v, tail[..., 0], tail[..., 1]


# ---------------------------------------------------------------- the passes


def run(s):
    return {"prompts": _prompts, "prompts_bwd": _prompts_bwd, "append8": _append8, "decode8": _decode8}[s["op"]](s)


def _pieces(s):
    """(rows a : b of q, first key, keys, position of row a among them) of each sequence, at most
    2^29 pairs of all heads at a time."""
    at_q, at_k = _starts(s["new"]), _starts(s["keys"])
    for r, (n, m) in enumerate(zip(s["new"], s["keys"])):
        step = max(1, (1 << 29) // max(1, s["Hq"] * m))
        for a in range(0, n, step):
            b = min(n, a + step)
            seen = min(m, m - n + b) if s["causal"] else m
            yield at_q[r] + a, at_q[r] + b, at_k[r], max(seen, 0), m - n + a


def _scores(s, a, b, k0, m, pos):
    """Scaled scores [Hk, G * (b - a), m] of rows a : b, hidden ones -inf."""
    Hk, d = s["Hk"], s["d"]
    q = s["q"][a:b].float().unflatten(1, (Hk, -1)).permute(1, 2, 0, 3).flatten(1, 2)
    x = torch.matmul(q, s["k"][k0:k0 + m].float().permute(1, 2, 0)) * s["scale"]
    if s["causal"]:
        last = pos + torch.arange(b - a, device="cuda").repeat(s["Hq"] // Hk)
        x.masked_fill_(torch.arange(m, device="cuda") > last[:, None], -math.inf)
    return x


def _rows(x, n):
    """[Hk, G * n, c] as [n, Hq, c]."""
    return x.unflatten(1, (-1, n)).permute(2, 0, 1, 3).flatten(1, 2)


def _prompts_plain(s):
    o = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    for a, b, k0, m, pos in _pieces(s):
        if m == 0:
            o[a:b], lse[a:b] = 0, -math.inf
            continue
        x = _scores(s, a, b, k0, m, pos)
        top = x.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        p = x.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        y = torch.matmul(p, s["v"][k0:k0 + m].float().transpose(0, 1)) / torch.where(total > 0, total, 1.0)
        o[a:b] = _rows(y, b - a).to(o.dtype)
        lse[a:b] = _rows(top + torch.log(total), b - a)[..., 0]
    return o, lse


def _prompts(s):
    if own:
        import exact_io_aware_26_gb300 as fa
        return fa.attention_fwd_packed(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=s["causal"], scale=s["scale"])
    return _prompts_plain(s)


def _prompts_bwd(s):
    if own:
        import exact_io_aware_26_gb300 as fa
        return fa.attention_bwd_packed(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["cu_q"], s["cu_k"],
                                       causal=s["causal"], scale=s["scale"])
    Hk = s["Hk"]
    dq = torch.zeros_like(s["q"])
    dk, dv = (torch.zeros(s["k"].shape, dtype=torch.float32, device="cuda") for _ in (0, 1))
    for a, b, k0, m, pos in _pieces(s):
        if m == 0:
            continue

        def heads(x):  # rows a : b as [Hk, G * (b - a), c]
            return x[a:b].float().unflatten(1, (Hk, -1)).permute(1, 2, 0, 3).flatten(1, 2)

        lse, do = heads(s["lse"][..., None]), heads(s["do"])
        p = _scores(s, a, b, k0, m, pos).sub_(torch.where(lse == -math.inf, math.inf, lse)).exp_()
        dv[k0:k0 + m] += torch.matmul(p.transpose(1, 2), do).transpose(0, 1)
        ds = torch.matmul(do, s["v"][k0:k0 + m].float().permute(1, 2, 0))
        ds = ds.sub_((do * heads(s["o"])).sum(-1, keepdim=True)).mul_(p)
        del p
        dq[a:b] = _rows(torch.matmul(ds, s["k"][k0:k0 + m].float().transpose(0, 1)) * s["scale"], b - a).to(dq.dtype)
        dk[k0:k0 + m] += torch.matmul(ds.transpose(1, 2), heads(s["q"])).transpose(0, 1) * s["scale"]
    return dq, dk.to(s["k"].dtype), dv.to(s["v"].dtype)


def _append8(s):
    if own:
        import exact_io_aware_26_gb300 as fa
        fa.kv8_append(s["k"], s["v"], s["slots"], s["cache"])
        return fa.kv8_gather(s["cache"], s["back"], s["d"], dtype=DTYPES[s["dtype"]])
    page, dt = s["page"], DTYPES[s["dtype"]]
    slot = s["slots"].long()
    blocks = s["cache"].transpose(1, 2).flatten(0, 1)  # [pages * blocks of a page, H, bytes]: a copy
    blk, at = slot // BLOCK, slot % BLOCK
    k, v, *old = _unblock(blocks)
    fresh = torch.zeros(blocks.shape[0], dtype=torch.bool, device="cuda")
    fresh[blk[at == 0]] = True  # nothing that was there counts
    sides, scales = [], []
    for codes, scale, x in zip((k, v), old, (s["k"], s["v"])):
        x = x.float().clamp(-SATURATE, SATURATE)
        most = torch.zeros(scale.shape, device="cuda").index_reduce_(0, blk, x.abs().amax(-1), "amax")
        before = torch.where(fresh[:, None], 0.0, scale)
        after = torch.maximum(before, _scale_for(most))
        grown = (after > before) & (before > 0)
        kept = torch.round(codes.float() * torch.where(grown, before / torch.where(grown, after, 1.0), 1.0)[..., None, None])
        kept[blk, :, at] = _codes_for(x, after[blk][..., None]).float()
        touched = torch.zeros_like(fresh)
        touched[blk] = True
        sides.append(torch.where(touched[:, None, None, None], kept, codes.float()).to(torch.int8))
        scales.append(torch.where(touched[:, None], after, scale))
    blocks = _block(sides[0], sides[1], scales[0], scales[1])
    s["cache"].copy_(blocks.unflatten(0, (-1, page // BLOCK)).transpose(1, 2))
    back = s["back"].long()
    return tuple((c[back // BLOCK, :, back % BLOCK].float() * sc[back // BLOCK][..., None]).to(dt) for c, sc in zip(sides, scales))


def _decode8(s):
    if own:
        import exact_io_aware_26_gb300 as fa
        return fa.kv8_attention(s["q"], s["cache"], s["block_table"], s["kv_lens"], cu_q=s["cu_q"], max_q_len=s["q_len"],
                                scale=s["scale"], window=s["window"])
    q, d, Hk = s["q"], s["d"], s["Hk"]
    T, Hq, _ = q.shape
    blocks = s["cache"][s["block_table"].long().clamp(min=0)]  # [R, pages, Hk, blocks, bytes]
    k, v, ks, vs = _unblock(blocks)
    del blocks

    def whole(codes, scale):  # a request's keys or values, [R, Hk, 1, tokens, d]
        return (codes.float() * scale[..., None, None]).transpose(1, 2).flatten(2, 4)[:, :, None]

    # each request's new tokens, padded to the longest: [R, Hk, G, q_len, d]
    start, n = s["cu_q"][:-1].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    i = torch.arange(s["q_len"], device="cuda")
    mine = q[(start[:, None] + i).clamp(max=T - 1)].float().unflatten(2, (Hk, Hq // Hk)).permute(0, 2, 3, 1, 4)
    x = torch.matmul(mine, whole(k, ks).transpose(-1, -2)) * s["scale"]
    key = torch.arange(x.shape[-1], device="cuda")
    pos = (s["kv_lens"].long() - n)[:, None] + i
    sees = (key <= pos[..., None]) & (key < s["kv_lens"][:, None, None])
    if s["window"]:
        sees = sees & (key > pos[..., None] - s["window"])
    x = x.masked_fill(~sees[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, whole(v, vs)) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total)).squeeze(-1)
    # back to the tokens
    t = torch.arange(T, device="cuda")
    r = torch.searchsorted(s["cu_q"][1:].contiguous().long(), t, right=True)
    at = t - start[r]
    return o.permute(0, 3, 1, 2, 4)[r, at].flatten(1, 2).to(q.dtype), lse.permute(0, 3, 1, 2)[r, at].flatten(1, 2)


# ---------------------------------------------------------------- what a pass cannot do without


def _seen(n, m, causal):
    """Pairs that n queries over m keys see, the last query at the last key."""
    if not causal:
        return n * m
    full = min(n, m)  # rows that see a key
    return full * (m - full) + full * (full + 1) // 2


def work(case):
    op, d = case["op"], case["d"]
    first, second = _lengths(case)
    if op in ("prompts", "prompts_bwd"):
        pairs = sum(_seen(n, m, case["causal"]) for n, m in zip(first, second))
        q, kv = sum(first) * case["Hq"], sum(second) * case["Hk"]
        if op == "prompts":
            return {"bytes": 4 * q * d + 4 * kv * d + 4 * q, "flops": 4 * pairs * case["Hq"] * d}
        return {"bytes": 8 * q * d + 8 * kv * d + 4 * q, "flops": 10 * pairs * case["Hq"] * d}
    if op == "append8":
        e = 4 if case["dtype"] == "f32" else 2
        rows = sum(first) * case["H"]
        back = sum(n + h % BLOCK for n, h in zip(first, second)) * case["H"]
        return {"bytes": rows * 2 * d * (e + 1) + back * 2 * d * (e + 1), "flops": 8 * rows * d}
    read = pairs = 0
    for n, m in zip(first, second):
        low = max(0, n - m - case["window"] + 1) if case["window"] else 0
        read += n - low
        for i in range(m):
            p = n - m + i
            pairs += max(0, p + 1 - (max(0, p - case["window"] + 1) if case["window"] else 0))
    T = sum(second)
    return {"bytes": read * case["Hk"] * block_bytes(d) // BLOCK + T * case["Hq"] * (4 * d + 4),
            "flops": 4 * pairs * case["Hq"] * d}


# ---------------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    op = case["op"]
    if op != "append8" and work(case)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    if op == "append8":
        return _exact_append8(case, s)
    if op == "decode8":
        return _exact_decode8(case, s)
    G = case["Hq"] // case["Hk"]
    q = s["q"].double()
    o, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), *(torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda") for _ in (0, 1))
    at_q = at_k = 0
    for n, m in zip(s["new"], s["keys"]):
        for a in range(0, n, 1024):
            b = min(n, a + 1024)
            end = min(m, m - n + b) if case["causal"] else m
            if end <= 0:
                continue
            unseen = torch.ones(b - a, end, dtype=torch.bool, device="cuda").triu(m - n + a + 1) if case["causal"] else None
            rows, cols = slice(at_q + a, at_q + b), slice(at_k, at_k + end)
            for h in range(case["Hq"]):
                K, V = s["k"][cols, h // G].double(), s["v"][cols, h // G].double()
                x = q[rows, h] @ K.T * s["scale"]
                if unseen is not None:
                    x[unseen] = -math.inf
                if op == "prompts":
                    lse[rows, h] = torch.logsumexp(x, -1)
                    o[rows, h] = torch.nan_to_num(torch.softmax(x, -1), nan=0.0) @ V
                    continue
                known = s["lse"][rows, h].double()[:, None]
                w = torch.where(known > -math.inf, torch.exp(x - known), 0.0)
                do = s["do"][rows, h].double()
                dv[cols, h // G] += w.T @ do
                ds = w * (do @ V.T - (do * s["o"][rows, h].double()).sum(-1, keepdim=True)) * s["scale"]
                dq[rows, h] += ds @ K
                dk[cols, h // G] += ds.T @ q[rows, h]
        at_q += n
        at_k += m
    return (o, lse) if op == "prompts" else (dq, dk, dv)


def _value_of(raw, d, side, token):
    """Codes (64 bits) of one token of blocks [.., bytes], [.., d], from the layout's addresses."""
    c = torch.arange(d, device="cuda")
    if side == 0:
        where = token * d + (c if token % 2 == 0 or d < 128 else (c + d // 2) % d)
    else:
        where = BLOCK * d + c // 4 * 64 + token // 4 * 16 + c % 4 * 4 + token % 4
    byte = raw[..., where].double()
    return torch.where(byte >= 128, byte - 256, byte)


def _scale_of(raw, d, side):
    return raw[..., 2 * BLOCK * d + 4 * side:2 * BLOCK * d + 4 * side + 4].contiguous().view(torch.float32)[..., 0].double()


def _power(e):
    """2^e, exactly, in 64 bits."""
    return ((e.clamp(-1000, 1000).long() + 1023) << 52).view(torch.float64)


def _exact_append8(case, s):
    d, page = case["d"], case["page"]
    new, held = _lengths(case)
    found = ([], [])
    at = 0
    for n, h in zip(new, held):
        for b in range(h // BLOCK, (h + n - 1) // BLOCK + 1):
            lo, hi = max(h, b * BLOCK), min(h + n, (b + 1) * BLOCK)  # its new tokens
            slot = int(s["slots"][at + lo - h])
            raw = s["cache"][slot // page, :, slot % page // BLOCK]
            for side, x in enumerate((s["k"], s["v"])):
                x = x[at + lo - h:at + hi - h].double().clamp(-SATURATE, SATURATE)
                most = x.abs().amax((0, 2))
                e = torch.round(torch.log2(most / 127))  # or one more: the least with most <= 127 * 2^e
                e = torch.where(most > 127 * _power(e), e + 1, e).clamp(min=LEAST)
                need = torch.where(most > 0, _power(e), 0.0)
                before = torch.zeros_like(need) if lo == b * BLOCK else _scale_of(raw, d, side)
                scale = torch.maximum(before, need)
                safe = torch.where(scale > 0, scale, 1.0)
                for j in range(b * BLOCK, lo):
                    found[side].append(torch.round(_value_of(raw, d, side, j % BLOCK) * (before / safe)[:, None]) * scale[:, None])
                found[side].extend(torch.round(x / safe[:, None]) * scale[:, None])
        at += n
    return tuple(torch.stack(f) for f in found)


def _exact_decode8(case, s):
    q, d, page, G = s["q"].double(), case["d"], case["page"], case["Hq"] // case["Hk"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    kv, new = _lengths(case)
    at = 0
    for r, (n, m) in enumerate(zip(kv, new)):
        if n:
            raw = s["cache"][s["block_table"][r, :(n + page - 1) // page].long()].transpose(0, 1).flatten(1, 2)  # [Hk, blocks, bytes]
            K, V = (torch.stack([_value_of(raw, d, side, j) for j in range(BLOCK)], 2).mul_(_scale_of(raw, d, side)[..., None, None])
                    .flatten(1, 2)[:, :n] for side in (0, 1))
            for i in range(m):
                p = n - m + i
                first = max(0, p - case["window"] + 1) if case["window"] else 0
                if p < 0:
                    continue
                for h in range(case["Hk"]):
                    x = q[at + i, h * G:(h + 1) * G] @ K[h, first:p + 1].T * s["scale"]
                    lse[at + i, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                    out[at + i, h * G:(h + 1) * G] = torch.softmax(x, -1) @ V[h, first:p + 1]
        at += m
    return out, lse
