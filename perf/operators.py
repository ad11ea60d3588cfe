"""The operators around the attention kernels, as they are measured: their cases, their
inputs, their plain forms and their 64-bit definitions.

* ``norm_rope`` / ``norm_rope_bwd``: RMS norms of the query and key heads and the rotation
  by position, from the packed projection to the layout the attention reads, and back.
* ``plan``: block tables and slot maps of a paged cache, from request lengths.
* ``append``: new keys and values quantised to 4 bits into their slots of the cache (and
  read back from there, as the values the codes stand for).
* ``decode``: attention of each request's newest tokens over its 4-bit cache.

With ``own`` false ``run`` computes them from elementary torch operations; with ``own``
true it makes the calls of ``exact_io_aware_26_gb300``.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
GROUP = 32        # channels that share one (scale, base) pair
SATURATE = 16384  # quantised values saturate here
BLOCK = 16        # tokens of a cache block


def listed():
    return [
        # training: the packed projection of a trading day (23,400 steps, 12 heads)
        dict(name="norm_rope_day", op="norm_rope", B=1, N=23400, Hq=12, Hk=12, d=64, rot=64, dtype="bf16",
             interleaved=False, heads_first=True, far=0),
        # serving: sixteen single tokens at far positions, four query heads per key head
        dict(name="norm_rope_tokens", op="norm_rope", B=1, N=16, Hq=32, Hk=8, d=128, rot=128, dtype="f16",
             interleaved=False, heads_first=False, far=900000),
        # training, backward: the batch of 12-head sequences
        dict(name="norm_rope_bwd_n2048", op="norm_rope_bwd", B=4, N=2048, Hq=12, Hk=12, d=64, rot=64, dtype="bf16",
             interleaved=False, heads_first=True, far=0),
        # training, backward: the long 16-head sequences
        dict(name="norm_rope_bwd_n16384", op="norm_rope_bwd", B=2, N=16384, Hq=16, Hk=16, d=128, rot=128, dtype="bf16",
             interleaved=False, heads_first=True, far=0),
        # serving: one new token for each of 256 requests, some of which have ended
        dict(name="plan_tokens", op="plan", R=256, T=256, most=16384, page=64, width=260, pages=40000, ended=0.05),
        # serving: a step that takes in prompts
        dict(name="plan_prompts", op="plan", R=96, T=65536, most=16384, page=16, width=2100, pages=200000, ended=0.1),
        # serving: the newest token of 256 requests into the cache
        dict(name="append_tokens", op="append", T=256, H=8, d=128, dtype="bf16", page=64, pages=600),
        # serving: a trading day as one prompt
        dict(name="append_day", op="append", T=23400, H=12, d=64, dtype="bf16", page=64, pages=500),
        # serving: the next token after a trading day, a key head for each query head
        dict(name="decode_day", op="decode", R=1, Hq=12, Hk=12, d=64, dtype="bf16", page=64, least=23400, most=23400,
             q_len=1, window=0, lens=1),
        # serving: a few short contexts, where latency counts
        dict(name="decode_n2048", op="decode", R=4, Hq=12, Hk=12, d=64, dtype="f16", page=16, least=1, most=2048,
             q_len=1, window=0, lens=2),
        # serving: a full batch of ragged long contexts, four query heads per key head
        dict(name="decode_n16384", op="decode", R=64, Hq=32, Hk=8, d=128, dtype="bf16", page=64, least=512, most=16384,
             q_len=1, window=0, lens=3),
        # serving: up to four draft tokens checked at once, in a window of the context
        dict(name="decode_drafts", op="decode", R=16, Hq=16, Hk=2, d=128, dtype="bf16", page=32, least=1, most=8192,
             q_len=4, window=4096, lens=4),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "plan", "append", "decode", "decode"])
    if op in ("norm_rope", "norm_rope_bwd"):
        d = rng.choice([64, 128])
        hk = rng.choice([1, 2, 3, 4, 8, 12, 16])
        hq = hk * rng.choice([1, 1, 2, 4, 5])
        most = max(1, 2 * 16384 * 32 * 128 // ((hq + hk) * d))
        n = _log(rng, 1, min(most, 40000))
        return dict(op=op, B=rng.randint(1, max(1, min(4, most // n))), N=n, Hq=hq, Hk=hk, d=d,
                    rot=rng.choice([d, d, d // 2, 2 * rng.randint(0, d // 2)]), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    interleaved=rng.random() < 0.3, heads_first=rng.random() < 0.6, far=rng.choice([0, 0, _log(rng, 1000, 1000000)]))
    if op == "plan":
        R, page = _log(rng, 1, 1000), rng.choice([16, 32, 64, 128])
        most = _log(rng, 64, 16384)
        T = _log(rng, R, max(R, 65536))
        return dict(op=op, R=R, T=T, most=most, page=page, width=(most + T) // page + 2,
                    pages=R * (most // page + 1) + T // page + R + rng.randint(1, 1000), ended=rng.choice([0.0, 0.1, 0.5]))
    if op == "append":
        d, H = rng.choice([64, 128]), rng.choice([1, 2, 3, 8, 12])
        T, page = _log(rng, 1, 24000), rng.choice([16, 32, 64, 128])
        return dict(op=op, T=T, H=H, d=d, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), page=page,
                    pages=2 * (T // page + 1) + rng.randint(0, 50))
    hk = rng.choice([1, 2, 3, 4, 8, 12])
    d, most = rng.choice([64, 128]), _log(rng, 1, 30000)
    R = _log(rng, 1, max(1, min(300, 64 * 16384 * 8 * 128 // (2 * hk * d * most))))
    q_len = rng.choice([1, 1, 1, 2, 5, 8])
    return dict(op="decode", R=R, Hq=hk * rng.choice([1, 2, 4, 5, 8]), Hk=hk, d=d, dtype=rng.choice(["bf16", "f16"]),
                page=rng.choice([16, 32, 64, 128]), least=rng.randint(0, most), most=most, q_len=q_len,
                window=rng.choice([0, 0, rng.randint(1, most)]), lens=rng.randrange(1 << 20))


# ---------------------------------------------------------------- inputs


def _lengths(case):
    """(cached tokens, new tokens) of each request of a decode case: part of the case, not of the seed."""
    r = random.Random(case["lens"])
    kv = [r.randint(case["least"], case["most"]) for _ in range(case["R"])]
    return kv, [r.randint(1, case["q_len"]) for _ in range(case["R"])]


def block_bytes(d):
    """Bytes of one cache block: 16 tokens' key codes, key pairs, value codes, value pairs."""
    return 2 * (BLOCK * d // 2 + BLOCK * (d // GROUP) * 4)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dev = case["op"], "cuda"

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev).to(dtype)

    s = dict(case)
    if op in ("norm_rope", "norm_rope_bwd"):
        B, N, Hq, Hk, d, rot, dt = (case[k] for k in ("B", "N", "Hq", "Hk", "d", "rot", "dtype"))
        packed = normal(B, N, Hq + 2 * Hk, d, dtype=DTYPES[dt])  # one projection: queries, keys, values
        s["q"], s["k"] = packed[:, :, :Hq], packed[:, :, Hq:Hq + Hk]
        s["wq"], s["wk"] = ((1 + 0.1 * normal(d)).to(DTYPES[dt]) for _ in range(2))
        s["eps"] = 1e-6
        # the turns (2^-64 each) that a position adds to each pair's angle
        turns = [int(round(10000.0 ** (-2.0 * i / max(rot, 1)) / (2 * math.pi) * 2 ** 64)) for i in range(rot // 2)]
        s["freqs"] = torch.tensor(turns, dtype=torch.int64, device=dev)
        s["positions"] = None
        if case["far"]:
            s["positions"] = torch.randint(0, case["far"], (B, N), generator=g, device=dev).to(torch.int32)
        if op == "norm_rope_bwd":
            shape = (lambda h: (B, h, N, d)) if case["heads_first"] else (lambda h: (B, N, h, d))
            s["dyq"], s["dyk"] = normal(*shape(Hq), dtype=DTYPES[dt]), normal(*shape(Hk), dtype=DTYPES[dt])
    elif op == "plan":
        R, T, page, width, pages = (case[k] for k in ("R", "T", "page", "width", "pages"))
        seq = torch.randint(0, case["most"] + 1, (R,), generator=g, device=dev)
        # as many new tokens as fit the step, shared out among the requests
        share = torch.rand(R, generator=g, device=dev).double() ** 3 if T > R else torch.full((R,), 0.5, device=dev).double()
        new = torch.clamp((share / share.sum() * (T - R)).long() + 1, max=page * (width - 1) - case["most"])
        s["new_lens"] = torch.where(torch.rand(R, generator=g, device=dev) < case["ended"], -1, new).to(torch.int32)
        s["seq_lens"] = seq.to(torch.int32)
        have = (seq + page - 1) // page
        off = torch.cumsum(have, 0) - have
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        i = torch.arange(width, device=dev)
        at = (off[:, None] + i).clamp(max=pages - 1)
        s["block_table"] = torch.where(i < have[:, None], order[at], -1).to(torch.int32)
        used = have.sum()
        s["free_pages"] = torch.roll(order, -int(used))
        s["free_count"] = (pages - used).to(torch.int32).reshape(1)
    elif op == "append":
        T, H, d, page, pages, dt = (case[k] for k in ("T", "H", "d", "page", "pages", "dtype"))
        packed = normal(T, 2 * H, d, dtype=DTYPES[dt])
        s["k"], s["v"] = packed[:, :H], packed[:, H:]
        s["cache"] = torch.zeros(pages, H, page // BLOCK, block_bytes(d), dtype=torch.uint8, device=dev)
        s["slots"] = torch.randperm(pages * page, generator=g, device=dev)[:T].to(torch.int32)
    else:
        R, Hq, Hk, d, page, dt = (case[k] for k in ("R", "Hq", "Hk", "d", "page", "dtype"))
        kv, new = _lengths(case)
        have = [(n + page - 1) // page for n in kv]
        pages, width = sum(have) + 1, max(max(have), 1)
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        at, table = 0, torch.full((R, width), -1, dtype=torch.int32)
        for r, h in enumerate(have):
            table[r, :h] = torch.arange(at, at + h, dtype=torch.int32)
            at += h
        table = table.to(dev)
        s["block_table"] = torch.where(table >= 0, order[table.clamp(min=0).long()], -1).to(torch.int32)
        s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
        s["cu_q"] = torch.tensor([sum(new[:r]) for r in range(R + 1)], dtype=torch.int32, device=dev)
        s["q"] = normal(sum(new), Hq, d, dtype=DTYPES[dt])
        s["scale"] = 1.0 / math.sqrt(d)
        s["cache"] = torch.empty(pages, Hk, page // BLOCK, block_bytes(d), dtype=torch.uint8, device=dev)
        step = max(1, (1 << 27) // (Hk * page * d))
        for a in range(0, pages, step):
            part = s["cache"][a:a + step]
            for half in (0, 1):
                codes, pairs = _quantise(normal(part.shape[0], Hk, page // BLOCK, BLOCK, d))
                _codes(part, d)[half].copy_(codes)
                _pairs(part, d)[half].copy_(pairs)
    return s


# ---------------------------------------------------------------- the cache's format


def _codes(cache, d):
    """Views of the key and value codes, [pages, heads, blocks, 16, d/2] bytes."""
    n = BLOCK * d // 2
    half = cache.shape[-1] // 2
    return [cache[..., a:a + n].unflatten(-1, (BLOCK, d // 2)) for a in (0, half)]


def _pairs(cache, d):
    """Views of the key and value (scale, base) pairs, [pages, heads, blocks, 16, groups * 4] bytes."""
    n, w = BLOCK * d // 2, d // GROUP * 4
    half = cache.shape[-1] // 2
    return [cache[..., a + n:a + half].unflatten(-1, (BLOCK, w)) for a in (0, half)]


def _quantise(x):
    """Code bytes [..., d/2] and pair bytes [..., d/32 * 4] of x [..., d]."""
    x = x.float().clamp(-SATURATE, SATURATE).unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = ((hi - lo) * 16 / 15).half()
    base = (lo - scale.float()).half()
    s, b = scale.float(), base.float()
    code = torch.where(s > 0, torch.round((x - b) * 16 / torch.where(s > 0, s, 1.0) - 16).clamp(0, 15), 0.0)
    code = code.flatten(-2).to(torch.uint8)
    pairs = torch.cat([scale, base], -1).contiguous().flatten(-2).view(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), pairs


def _values(codes, pairs):
    """The fp16 values that code and pair bytes stand for, [..., d]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (-1, GROUP)).float()
    p = pairs.contiguous().view(torch.float16).unflatten(-1, (-1, 2)).float()
    return (p[..., 1:] + p[..., :1] * (1 + c / 16)).half().flatten(-2)


# ---------------------------------------------------------------- the passes


def run(s):
    return {"norm_rope": _norm_rope, "norm_rope_bwd": _norm_rope_bwd, "plan": _plan, "append": _append,
            "decode": _decode}[s["op"]](s)


def _angles(s):
    """cos and sin of each token's angles, [B, N, 1, rot/2], formed in 64 bits."""
    B, N = s["q"].shape[:2]
    pos = torch.arange(N, device="cuda").expand(B, N) if s["positions"] is None else s["positions"]
    a = pos.double()[..., None, None] * (s["freqs"].double() * (2 * math.pi / 2.0 ** 64))
    return a.cos().float(), a.sin().float()


def _pairs_of(y, rot, interleaved):
    """The first and second elements of the rotated pairs of y."""
    return (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])


def _rotate(y, cos, sin, rot, interleaved):
    a, b = _pairs_of(y, rot, interleaved)
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.cat([torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1), y[..., rot:]], -1)


def _norm_rope(s):
    if own:
        import exact_io_aware_26_gb300 as fa
        return fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["freqs"], positions=s["positions"], eps=s["eps"],
                               interleaved=s["interleaved"], heads_first=s["heads_first"])
    cos, sin = _angles(s)

    def one(x, w):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w.float()
        y = _rotate(y, cos, sin, s["rot"], s["interleaved"]).to(x.dtype)
        return y.transpose(1, 2).contiguous() if s["heads_first"] else y

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _norm_rope_bwd(s):
    if own:
        import exact_io_aware_26_gb300 as fa
        return fa.qk_norm_rope_bwd(s["q"], s["k"], s["dyq"], s["dyk"], s["wq"], s["wk"], s["freqs"],
                                   positions=s["positions"], eps=s["eps"], interleaved=s["interleaved"],
                                   heads_first=s["heads_first"])
    cos, sin = _angles(s)

    def one(x, dy, w):
        dy = dy.transpose(1, 2) if s["heads_first"] else dy
        dz = _rotate(dy.float(), cos, -sin, s["rot"], s["interleaved"])
        r = torch.rsqrt((x.float() ** 2).mean(-1, keepdim=True) + s["eps"])
        n = x.float() * r
        dn = dz * w.float()
        dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
        return dx.to(x.dtype), (dz * n).double().sum((0, 1, 2)).float()

    dq, dwq = one(s["q"], s["dyq"], s["wq"])
    dk, dwk = one(s["k"], s["dyk"], s["wk"])
    return dq, dk, dwq, dwk


def _plan(s):
    page, T = s["page"], s["T"]
    if own:
        import exact_io_aware_26_gb300 as fa
        out = fa.paged_plan(s["seq_lens"], s["new_lens"], s["block_table"], s["free_pages"], s["free_count"], page, T)
        return {**out, "block_table": s["block_table"], "free_pages": s["free_pages"]}
    table, stack = s["block_table"], s["free_pages"]
    width, pages = table.shape[1], stack.shape[0]
    seq, ended = s["seq_lens"].long(), s["new_lens"] < 0
    new, top = s["new_lens"].long().clamp(min=0), s["free_count"].long()
    have = (seq + page - 1) // page
    cu = torch.cumsum(new, 0)
    # pages of ended requests go onto the stack of free pages, in order
    freed = torch.where(ended, have.clamp(max=width), 0)
    freed_off = torch.cumsum(freed, 0) - freed
    i = torch.arange(width, device="cuda")
    to = torch.where(i < freed[:, None], top + freed_off[:, None] + i, pages)
    pool = torch.cat([stack, stack[:1]])
    pool = pool.scatter(0, to.clamp(max=pages).flatten(), table.flatten())
    there = top + freed.sum()
    # pages that the new tokens need come off its end, all of a request's or none
    after = (seq + new + page - 1) // page
    fits = ~ended & (after <= width) & (cu <= T)
    need = torch.where(fits, after - have, 0)
    upto = torch.cumsum(need, 0)
    served = fits & ((need == 0) | (upto <= there))
    taken = torch.where(served, upto, 0).amax()
    need_off = upto - need
    from_pool = there - 1 - (need_off[:, None] + i - have[:, None])
    fresh = served[:, None] & (i >= have[:, None]) & (i < after[:, None])
    table.copy_(torch.where(fresh, pool[from_pool.clamp(0, pages)], table))
    left = there - taken
    j = torch.arange(pages, device="cuda")
    stack.copy_(torch.where((j >= top) & (j < left), pool[:pages], stack))
    kv = torch.where(ended, 0, seq + torch.where(served, new, 0))
    # the step's tokens
    t = torch.arange(T, device="cuda")
    r = torch.searchsorted(cu, t, right=True)
    real, r = r < seq.shape[0], r.clamp(max=seq.shape[0] - 1)
    pos = seq[r] + t - (cu - new)[r]
    slot = table[r, (pos // page).clamp(0, width - 1)].long() * page + pos % page
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    return {"kv_lens": kv.int(), "cu_q": torch.cat([zero, cu]).clamp(max=T).int(), "positions": torch.where(real, pos, 0).int(),
            "slots": torch.where(real & served[r], slot, -1).int(),
            "counts": torch.stack([left[0], cu[-1], (upto[-1] - there[0]).clamp(min=0)]).int(),
            "block_table": table, "free_pages": stack}


def _append(s):
    if own:
        import exact_io_aware_26_gb300 as fa
        fa.kv4_append(s["k"], s["v"], s["slots"], s["cache"])
        return fa.kv4_gather(s["cache"], s["slots"], s["d"], dtype=DTYPES[s["dtype"]])
    d, slot = s["d"], s["slots"].long()
    at = (slot // s["page"], slice(None), slot % s["page"] // BLOCK, slot % BLOCK)
    codes, pairs = _codes(s["cache"], d), _pairs(s["cache"], d)
    codes[0][at], pairs[0][at] = _quantise(s["k"])
    codes[1][at], pairs[1][at] = _quantise(s["v"])
    return tuple(_values(codes[h][at], pairs[h][at]).to(DTYPES[s["dtype"]]) for h in (0, 1))


def _decode(s):
    if own:
        import exact_io_aware_26_gb300 as fa
        return fa.kv4_attention(s["q"], s["cache"], s["block_table"], s["kv_lens"], cu_q=s["cu_q"], max_q_len=s["q_len"],
                                scale=s["scale"], window=s["window"])
    q, cache, d, page = s["q"], s["cache"], s["d"], s["page"]
    T, Hq, _ = q.shape
    R, Hk = s["kv_lens"].shape[0], s["Hk"]
    mine = cache[s["block_table"].long().clamp(min=0)]  # [R, pages, Hk, blocks, bytes]

    def whole(half):  # a request's keys or values, [R, Hk, 1, tokens, d]
        x = _values(_codes(mine, d)[half], _pairs(mine, d)[half])
        return x.transpose(1, 2).flatten(2, 4)[:, :, None].float()

    # each request's new tokens, padded to the longest: [R, Hk, G, q_len, d]
    start, n = s["cu_q"][:-1].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    i = torch.arange(s["q_len"], device="cuda")
    mineq = q[(start[:, None] + i).clamp(max=T - 1)].float().unflatten(2, (Hk, Hq // Hk)).permute(0, 2, 3, 1, 4)
    x = torch.matmul(mineq, whole(0).transpose(-1, -2)) * s["scale"]
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
    o = torch.matmul(p, whole(1)) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total)).squeeze(-1)
    # back to the tokens
    t = torch.arange(T, device="cuda")
    r = torch.searchsorted(s["cu_q"][1:].contiguous().long(), t, right=True)
    at = t - start[r]
    return o.permute(0, 3, 1, 2, 4)[r, at].flatten(1, 2).to(q.dtype), lse.permute(0, 3, 1, 2)[r, at].flatten(1, 2)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    if op in ("norm_rope", "norm_rope_bwd"):
        e = 4 if case["dtype"] == "f32" else 2
        n = case["B"] * case["N"] * (case["Hq"] + case["Hk"]) * case["d"]
        return {"bytes": n * e * (2 if op == "norm_rope" else 3), "flops": n * (9 if op == "norm_rope" else 18)}
    if op == "plan":
        return {"bytes": 8 * case["T"] + 20 * case["R"] + 4 * (case["T"] // case["page"]), "flops": 10 * case["T"]}
    if op == "append":
        e = 4 if case["dtype"] == "f32" else 2
        rows = case["T"] * case["H"]
        cells = block_bytes(case["d"]) // BLOCK
        return {"bytes": rows * (4 * case["d"] * e + 2 * cells) + 8 * case["T"], "flops": rows * case["d"] * 16}
    kv, new = _lengths(case)
    read = pairs = 0
    for n, m in zip(kv, new):
        first = max(0, n - m - case["window"] + 1) if case["window"] else 0
        read += n - first
        for i in range(m):
            p = n - m + i
            pairs += max(0, p + 1 - (max(0, p - case["window"] + 1) if case["window"] else 0))
    T = sum(new)
    return {"bytes": read * case["Hk"] * block_bytes(case["d"]) // BLOCK + T * case["Hq"] * (4 * case["d"] + 4),
            "flops": 4 * pairs * case["Hq"] * case["d"]}


# ---------------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    op, s = case["op"], prepare(case, seed)
    if op == "plan":
        return None
    if op == "append":
        # the value of a code is what the format makes of it: (16 + code) / 16 steps of the scale above the base
        def round_trip(x):
            x = torch.clamp(x.double(), -SATURATE, SATURATE).reshape(*x.shape[:-1], -1, GROUP)
            lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            scale = ((hi - lo) * 16 / 15).float().half().double()
            base = (lo - scale).float().half().double()
            code = torch.nan_to_num(torch.round(16 * (x - base) / scale - 16)).clamp(0, 15)
            return (base + scale * (16 + code) / 16).half().double().flatten(-2)
        return round_trip(s["k"]), round_trip(s["v"])
    if op == "decode":
        q, d, page, G = s["q"].double(), case["d"], case["page"], case["Hq"] // case["Hk"]
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        kv, new = _lengths(case)
        at = 0
        for r, (n, m) in enumerate(zip(kv, new)):
            if n:
                own_pages = s["cache"][s["block_table"][r, :(n + page - 1) // page].long()]
                half = own_pages.shape[-1] // 2

                def side(a):
                    raw = own_pages[..., a:a + half].transpose(0, 1).reshape(case["Hk"], -1, half)
                    codes = raw[..., :BLOCK * d // 2].reshape(case["Hk"], -1, d // 2).int()
                    pair = raw[..., BLOCK * d // 2:].contiguous().view(torch.float16).reshape(case["Hk"], -1, d // GROUP, 2).double()
                    code = torch.empty(*codes.shape[:-1], d, dtype=torch.float64, device="cuda")
                    code[..., 0::2], code[..., 1::2] = codes % 16, codes // 16
                    scale, base = (pair[..., j].repeat_interleave(GROUP, -1) for j in (0, 1))
                    return (base + scale * (16 + code) / 16).half().double()[:, :n]

                K, V = side(0), side(half)
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
    B, N = s["q"].shape[:2]
    rot = case["rot"]
    pos = torch.arange(N, device="cuda").repeat(B, 1) if s["positions"] is None else s["positions"]
    exponent = torch.arange(rot // 2, device="cuda").double() * (2.0 / max(rot, 1))
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[:, :, None, None] * 10000.0 ** -exponent)
    if case["interleaved"]:
        first = torch.arange(0, rot, 2, device="cuda")
        second = first + 1
    else:
        first = torch.arange(rot // 2, device="cuda")
        second = first + rot // 2

    def turned(y, by):
        z = torch.complex(y[..., first], y[..., second]) * by
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    found = []
    for x, w, dy in ((s["q"], s["wq"], s.get("dyq")), (s["k"], s["wk"], s.get("dyk"))):
        x, w = x.double(), w.double()
        norm = torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + s["eps"])
        if op == "norm_rope":
            y = turned(x / norm * w, turn)
            found.append(y.transpose(1, 2) if case["heads_first"] else y)
        else:
            dz = turned((dy.transpose(1, 2) if case["heads_first"] else dy).double(), turn.conj())
            dn = dz * w
            found.append((dn / norm - x * (dn * x).sum(-1, keepdim=True) / (case["d"] * norm ** 3), (dz * x / norm).sum((0, 1, 2))))
    return tuple(found) if op == "norm_rope" else (found[0][0], found[1][0], found[0][1], found[1][1])
