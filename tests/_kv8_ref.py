"""The 8-bit cache by hand, from its description in include/fa.h, for the tests.  numpy only;
nothing of the package."""
from __future__ import annotations

import math

import numpy as np

BLOCK, SATURATE, LEAST = 16, 16384.0, -64


def block_bytes(d):
    return 32 * d + 16


def scale_for(most):
    """The least 2^e, e >= -64, with most <= 127 * 2^e; 0 for 0."""
    if most == 0:
        return 0.0
    e = LEAST
    while most > 127 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def places(d):
    """Byte of a block for (side, token, channel): [2][16][d]."""
    at = np.zeros((2, BLOCK, d), np.int64)
    for j in range(BLOCK):
        for c in range(d):
            at[0, j, c] = j * d + ((c + 64) % 128 if d == 128 and j % 2 else c)
            at[1, j, c] = BLOCK * d + c // 4 * 64 + j // 4 * 16 + c % 4 * 4 + j % 4
    return at


class Block:
    """One block of one head, as bytes."""

    def __init__(self, raw, d):
        self.raw, self.d, self.at = raw, d, places(d)

    def codes(self, side):
        return self.raw[self.at[side]].view(np.int8)

    def scale(self, side):
        return self.raw[32 * self.d + 4 * side:32 * self.d + 4 * side + 4].view(np.float32)

    def marks(self, side):
        return self.raw[32 * self.d + 8 + 2 * side:32 * self.d + 10 + 2 * side].view(np.uint16)

    def values(self, side):
        x = self.codes(side).astype(np.float64) * float(self.scale(side)[0])
        x[[j for j in range(BLOCK) if int(self.marks(side)[0]) >> j & 1]] = np.nan
        return x

    def append(self, side, places_, x):
        """x [n, d] (fp32 values) into the places."""
        nan = np.isnan(x).any(-1)
        x = np.where(nan[:, None], 0, np.clip(x.astype(np.float64), -SATURATE, SATURATE))
        fresh = 0 in places_
        old = 0.0 if fresh else float(self.scale(side)[0])
        scale = max(old, scale_for(np.abs(x).max(initial=0)))
        if old and scale > old:
            for j in range(BLOCK):
                if j not in places_:
                    self.raw[self.at[side, j]] = np.rint(self.codes(side)[j] * (old / scale)).astype(np.int8).view(np.uint8)
        mark = 0 if fresh else int(self.marks(side)[0])
        for j, row, bad in zip(places_, x, nan):
            self.raw[self.at[side, j]] = (np.rint(row / scale) if scale else row * 0).astype(np.int8).view(np.uint8)
            mark = mark & ~(1 << j) | int(bad) << j
        self.scale(side)[0] = scale
        self.marks(side)[0] = mark
        if fresh:
            self.raw[32 * self.d + 12:] = 0


def append(cache, k, v, slots):
    """k, v [T, H, d] into the slots of cache [pages, H, blocks, bytes], in place."""
    page, d = cache.shape[2] * BLOCK, k.shape[2]
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] >= 0 and slots[t + n] // BLOCK == slots[t] // BLOCK:
            n += 1
        where = [int(s) % BLOCK for s in slots[t:t + n]]
        for h in range(k.shape[1]):
            raw = cache[slots[t] // page, h, slots[t] % page // BLOCK]
            for side, x in enumerate((k, v)):
                Block(raw, d).append(side, where, x[t:t + n, h])
        t += n


def slot_values(cache, slots, d):
    """(k, v) fp64 [T, H, d] of the slots, zeros for a negative one."""
    page, H = cache.shape[2] * BLOCK, cache.shape[1]
    out = np.zeros((2, len(slots), H, d))
    known = {}
    for t, s in enumerate(slots):
        if s < 0:
            continue
        for h in range(H):
            key = (int(s) // BLOCK, h)
            if key not in known:
                b = Block(cache[s // page, h, s % page // BLOCK], d)
                known[key] = (b.values(0), b.values(1))
            out[0, t, h], out[1, t, h] = known[key][0][s % BLOCK], known[key][1][s % BLOCK]
    return out


def attention(q, k, v, kv_lens, cu_q, scale, window):
    """(o, lse, size, slack) of requests whose tokens' values are k[r], v[r] [n, Hk, d]: the result, and
    for the bounds per row sum p |v| / l with the subnormal weights' term, and the scores' size."""
    T, Hq, d = q.shape
    o, lse = np.zeros((T, Hq, d)), np.full((T, Hq), -np.inf)
    size, slack = np.zeros((T, Hq, d)), np.zeros((T, Hq))
    for r, n in enumerate(kv_lens):
        q0, q1 = cu_q[r], cu_q[r + 1]
        if n <= 0 or q1 <= q0:
            continue
        G = Hq // k[r].shape[1]
        for i in range(q1 - q0):
            p = n - (q1 - q0) + i
            first = max(0, p - window + 1) if window else 0
            if p < 0:
                continue
            for h in range(Hq):
                kk, vv = k[r][first:p + 1, h // G], v[r][first:p + 1, h // G]
                s = kk @ q[q0 + i, h] * scale
                m = s.max()
                w = np.exp(s - m)
                l = w.sum()
                o[q0 + i, h], lse[q0 + i, h] = w @ vv / l, m + math.log(l)
                size[q0 + i, h] = w @ np.abs(vv) / l + len(s) * 2.0 ** -13 * np.abs(vv).max() / l
                slack[q0 + i, h] = (np.abs(kk) @ np.abs(q[q0 + i, h])).max() * scale
    return o, lse, size, slack
