"""The 8-bit cache's append for calls of many tokens: the steps of _kv8_ref.append, all blocks of a call at
a time.  numpy only; nothing of the package."""
from __future__ import annotations

import numpy as np

import _kv8_ref as ref


def scales_for(most):
    """The least 2^e, e >= -64, with most <= 127 * 2^e; 0 for 0."""
    e = np.full(most.shape, ref.LEAST)
    some = most > 0
    e[some] = np.maximum(np.floor(np.log2(most[some] / 127)).astype(np.int64) - 1, ref.LEAST)
    for _ in range(3):
        e[some & (most > 127 * 2.0 ** e)] += 1
    return np.where(some, 2.0 ** e, 0.0)


def append(cache, k, v, slots):
    """k, v [T, H, d] (fp32 values) into the slots of cache [pages, H, blocks, bytes], in place."""
    page, d, H = cache.shape[2] * ref.BLOCK, k.shape[2], k.shape[1]
    tokens = np.flatnonzero(slots >= 0)
    blk, place = slots[tokens] // ref.BLOCK, slots[tokens] % ref.BLOCK
    begins = np.concatenate([[True], (blk[1:] != blk[:-1]) | (tokens[1:] != tokens[:-1] + 1)])
    run = np.cumsum(begins) - 1
    blocks = blk[begins]
    where = (blocks * ref.BLOCK // page, slice(None), blocks * ref.BLOCK % page // ref.BLOCK)
    raw, n = cache[where].copy(), len(blocks)  # [runs, H, bytes]
    there = np.zeros((n, ref.BLOCK), bool)
    there[run, place] = True
    fresh = there[:, 0]
    at = ref.places(d)
    for side, x in enumerate((k, v)):
        x = x[tokens].astype(np.float64)
        lost = np.isnan(x).any(-1)
        full, bad = np.zeros((n, H, ref.BLOCK, d)), np.zeros((n, H, ref.BLOCK), bool)
        full[run, :, place] = np.where(lost[..., None], 0, np.clip(np.where(np.isnan(x), 0, x), -ref.SATURATE, ref.SATURATE))
        bad[run, :, place] = lost
        tail = raw[:, :, 32 * d:].copy()
        old = tail[..., 4 * side:4 * side + 4].copy().view(np.float32)[..., 0]
        old = np.where(fresh[:, None], np.float32(0), old).astype(np.float64)  # (what was there may be a NaN's bytes)
        scale = np.maximum(old, scales_for(np.abs(full).max((2, 3))))
        codes = raw[:, :, at[side]].view(np.int8).astype(np.float64)
        ratio = np.where((old > 0) & (scale > old), old / np.where(scale > 0, scale, 1.0), 1.0)
        codes = np.rint(codes * ratio[..., None, None])
        new = np.rint(full / np.where(scale > 0, scale, 1.0)[..., None, None])
        codes = np.where(there[:, None, :, None], new, codes).astype(np.int8)
        raw[:, :, at[side].reshape(-1)] = codes.reshape(n, H, -1).view(np.uint8)
        bit = 1 << np.arange(ref.BLOCK)
        marks = np.where(fresh[:, None], 0, tail[..., 8 + 2 * side:10 + 2 * side].copy().view(np.uint16)[..., 0].astype(np.int64))
        marks = marks & ~(there * bit).sum(-1)[:, None] | (bad * bit).sum(-1)
        raw[:, :, 32 * d + 4 * side:32 * d + 4 * side + 4] = scale.astype(np.float32)[..., None].view(np.uint8)
        raw[:, :, 32 * d + 8 + 2 * side:32 * d + 10 + 2 * side] = marks.astype(np.uint16)[..., None].view(np.uint8)
    raw[fresh, :, 32 * d + 12:] = 0
    cache[where] = raw


def values(cache, slots, d):
    """(k, v) fp64 [T, H, d] of slots >= 0."""
    page, at = cache.shape[2] * ref.BLOCK, ref.places(d)
    raw = cache[slots // page, :, slots % page // ref.BLOCK]  # [T, H, bytes]
    out = []
    for side in (0, 1):
        codes = np.take_along_axis(raw[:, :, :32 * d], np.broadcast_to(at[side][slots % ref.BLOCK][:, None], (*raw.shape[:2], d)), 2)
        scale = raw[:, :, 32 * d + 4 * side:32 * d + 4 * side + 4].copy().view(np.float32)[..., 0].astype(np.float64)
        marks = raw[:, :, 32 * d + 8 + 2 * side:32 * d + 10 + 2 * side].copy().view(np.uint16)[..., 0]
        x = codes.view(np.int8) * scale[..., None]
        x[(marks >> (slots % ref.BLOCK)[:, None] & 1).astype(bool)] = np.nan
        out.append(x)
    return out
