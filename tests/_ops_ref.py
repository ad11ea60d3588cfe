"""Plain 64-bit implementations of the operators around the attention, from their
formulas (include/fa.h), for the tests.  numpy only; nothing of the package."""
from __future__ import annotations

import math

import numpy as np

GROUP, BLOCK, SATURATE = 32, 16, 16384.0


# ---------------------------------------------------------------- norms and rotation

def _partners(d, rot, interleaved):
    """For every channel its pair, or -1, and whether it is the pair's second element."""
    pair, second = np.full(d, -1), np.zeros(d, bool)
    for c in range(rot):
        pair[c] = c // 2 if interleaved else c % (rot // 2)
        second[c] = c % 2 == 1 if interleaved else c >= rot // 2
    return pair, second


def rotate(y, pos, turns, interleaved, back=False):
    """y [B, N, H, d] rotated by pos [B, N]; turns: uint64 phase steps (2^-64 turns)."""
    B, N, H, d = y.shape
    rot = 2 * len(turns)
    pair, second = _partners(d, rot, interleaved)
    # exact phases in whole numbers, then the angle
    phase = np.array([[[(int(p) * int(t)) % 2 ** 64 for t in turns] for p in row] for row in pos], dtype=object)
    angle = (phase.reshape(B, N, -1).astype(np.float64) if rot else np.zeros((B, N, 0))) * (2 * math.pi / 2.0 ** 64)
    if back:
        angle = -angle
    out = y.copy()
    for c in range(d):
        if pair[c] < 0:
            continue
        a = [k for k in range(rot) if pair[k] == pair[c]]
        u, v = y[..., a[0]], y[..., a[1]]
        cos, sin = np.cos(angle[..., pair[c]])[..., None], np.sin(angle[..., pair[c]])[..., None]
        out[..., c] = u * sin + v * cos if second[c] else u * cos - v * sin
    return out


def norm_rope(x, w, pos, turns, eps, interleaved):
    """(y, n): the result and the normed values before the rotation."""
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return rotate(n, pos, turns, interleaved), n


def norm_rope_bwd(x, dy, w, pos, turns, eps, interleaved):
    """(dx, dw) and the magnitudes that bound their rounding errors."""
    dz = rotate(dy, pos, turns, interleaved, back=True)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = x * r
    dn = dz * w
    dx = r * (dn - h * (dn * h).mean(-1, keepdims=True))
    size = np.abs(rotate(np.abs(dy), pos, np.zeros_like(turns), interleaved))
    rot = 2 * len(turns)
    pair, _ = _partners(x.shape[-1], rot, interleaved)
    for c in range(rot):  # |dz| <= |dy_a| + |dy_b|
        a = [k for k in range(rot) if pair[k] == pair[c]]
        size[..., c] = np.abs(dy[..., a[0]]) + np.abs(dy[..., a[1]])
    gn = size * np.abs(w)
    return dx, (dz * h).sum((0, 1, 2)), r * (gn + np.abs(h) * (gn * np.abs(h)).mean(-1, keepdims=True)), (size * np.abs(h)).sum((0, 1, 2))


# ---------------------------------------------------------------- the 4-bit cache

def block_bytes(d):
    return 2 * (BLOCK * d // 2 + BLOCK * (d // GROUP) * 4)


def quantise(x):
    """(codes [..., d], scale, base [..., d / 32] fp16) of fp32 x [..., d]: the documented
    steps, each one fp32 operation."""
    f = np.float32
    g = x.astype(f).reshape(*x.shape[:-1], -1, GROUP)
    nan = np.isnan(g).any(-1)
    g = np.clip(np.where(np.isnan(g), f(0), g), f(-SATURATE), f(SATURATE))
    lo, hi = g.min(-1), g.max(-1)
    scale = ((hi - lo) * f(16) / f(15)).astype(np.float16)
    base = (lo - scale.astype(f)).astype(np.float16)
    s, b = scale.astype(f)[..., None], base.astype(f)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.rint((g - b) * f(16) / s - f(16))
    code = np.where(s > 0, np.clip(np.nan_to_num(code), 0, 15), 0).astype(np.uint8)
    scale, base = np.where(nan, np.float16(np.nan), scale), np.where(nan, np.float16(np.nan), base)
    code[nan] = 0
    return code.reshape(x.shape), scale, base


def values(codes, scale, base):
    """fp16(base + scale (1 + c / 16)), as fp64."""
    c = codes.reshape(*codes.shape[:-1], -1, GROUP).astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):  # slots that were never written may hold anything
        v = base.astype(np.float64)[..., None] + scale.astype(np.float64)[..., None] * (1 + c / 16)
        return v.astype(np.float16).astype(np.float64).reshape(codes.shape)


def pack(codes, scale, base):
    """Code bytes and pair bytes of one half of a block: [..., 16, d] -> [..., half]."""
    cb = (codes[..., 0::2] | (codes[..., 1::2] << 4)).reshape(*codes.shape[:-2], -1)
    pb = np.stack([scale, base], -1).astype(np.float16)
    pb = np.ascontiguousarray(pb).view(np.uint8).reshape(*codes.shape[:-2], -1)
    return np.concatenate([cb, pb], -1)


def unpack(raw, d):
    """The fp64 values of half blocks [..., half] -> [..., 16, d]."""
    n = BLOCK * d // 2
    cb = raw[..., :n].reshape(*raw.shape[:-1], BLOCK, d // 2)
    codes = np.empty((*cb.shape[:-1], d), np.uint8)
    codes[..., 0::2], codes[..., 1::2] = cb & 15, cb >> 4
    pairs = np.ascontiguousarray(raw[..., n:]).view(np.float16).reshape(*raw.shape[:-1], BLOCK, d // GROUP, 2)
    return values(codes, pairs[..., 0], pairs[..., 1])


def cache_of(k, v, page_size):
    """A cache of consecutive pages holding k, v [T, H, d] at slots 0 .. T - 1 (zeros after)."""
    T, H, d = k.shape
    pages = max(1, -(-T // page_size))
    out = np.zeros((pages, H, page_size // BLOCK, block_bytes(d)), np.uint8)
    for half, x in enumerate((k, v)):
        full = np.zeros((pages * page_size, H, d), np.float32)
        full[:T] = x
        c, s, b = quantise(full)
        s[T:], b[T:] = 0, 0
        blk = lambda a: a.reshape(pages, page_size // BLOCK, BLOCK, H, -1).transpose(0, 3, 1, 2, 4)
        out[..., half * block_bytes(d) // 2:(half + 1) * block_bytes(d) // 2] = pack(blk(c), blk(s), blk(b))
    return out


def slot_values(cache, slots, d):
    """(k, v) fp64 [T, H, d] of the slots."""
    page_size = cache.shape[2] * BLOCK
    half = cache.shape[3] // 2
    k, v = unpack(cache[..., :half], d), unpack(cache[..., half:], d)  # [pages, H, blocks, 16, d]
    at = (slots // page_size, slice(None), slots % page_size // BLOCK, slots % BLOCK)
    return k[at], v[at]


def attention(q, cache, table, kv_lens, cu_q, scale, window, d):
    """(o, lse, size, slack): the result, and per row sum p |v| / l and the bounds' score term."""
    T, Hq, _ = q.shape
    page_size, Hk = cache.shape[2] * BLOCK, cache.shape[1]
    G = Hq // Hk
    o, lse = np.zeros((T, Hq, d)), np.full((T, Hq), -np.inf)
    size, slack = np.zeros((T, Hq, d)), np.zeros((T, Hq))
    half = cache.shape[3] // 2
    every = [unpack(cache[..., a:a + half], d) for a in (0, half)]
    for r, n in enumerate(kv_lens):
        q0, q1 = cu_q[r], cu_q[r + 1]
        if n <= 0 or q1 <= q0:
            continue
        j = np.arange(n)
        k, v = (x[table[r][j // page_size], :, j % page_size // BLOCK, j % BLOCK] for x in every)
        for i in range(q1 - q0):
            p = n - (q1 - q0) + i
            first = max(0, p - window + 1) if window else 0
            if p < 0:
                continue
            for h in range(Hq):
                kk, vv = k[first:p + 1, h // G], v[first:p + 1, h // G]
                s = kk @ q[q0 + i, h] * scale
                m = s.max()
                w = np.exp(s - m)
                l = w.sum()
                o[q0 + i, h], lse[q0 + i, h] = w @ vv / l, m + math.log(l)
                size[q0 + i, h] = w @ np.abs(vv) / l + len(s) * 2.0 ** -14 * np.abs(vv).max() / l
                slack[q0 + i, h] = (np.abs(kk) @ np.abs(q[q0 + i, h])).max() * scale
    return o, lse, size, slack


# ---------------------------------------------------------------- block tables

def plan(seq, new, table, stack, count, page, T):
    """(kv_lens, cu_q, positions, slots, counts, table, stack), by hand."""
    table, stack = [list(r) for r in table], list(stack)
    width, R = len(table[0]), len(seq)
    pool = stack[:count]
    kv, cu, pos, slots = [], [0], [], []
    pages_of = lambda n: -(-n // page)
    for r in range(R):
        if new[r] < 0:
            pool += table[r][:min(pages_of(seq[r]), width)]
    there, asked, taken = len(pool), 0, 0
    before = [list(r) for r in table]
    for r in range(R):
        n, add = max(0, seq[r]), max(0, new[r])
        cu.append(cu[-1] + add)
        have, after = pages_of(n), pages_of(n + add)
        fits = new[r] >= 0 and after <= width and cu[-1] <= T
        want = after - have if fits else 0
        asked += want
        served = fits and (want == 0 or asked <= there)
        if served:
            for i in range(have, after):
                taken += 1
                table[r][i] = pool[there - taken]
        kv.append(0 if new[r] < 0 else n + (add if served else 0))
        for t in range(add):
            pos.append(n + t)
            slots.append(table[r][(n + t) // page] * page + (n + t) % page if served else -1)
    total = cu[-1]
    pos, slots = (pos + [0] * T)[:T], (slots + [-1] * T)[:T]
    left = there - taken
    for i in range(count, left):
        stack[i] = pool[i]
    return kv, [min(c, T) for c in cu], pos, slots, [left, total, max(0, asked - there)], table, stack
