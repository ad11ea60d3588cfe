"""The 8-bit cache and the attention that reads it, against plain implementations.

Codes, scales and marks are whole numbers and powers of two and must be equal.  The attention's
bounds are those of the 4-bit cache's (e = eps(type) / 2; w a weight, l their sum):
     |do| <= e |o| + (2^-11 + 2 s + 2^-20) sum w |v| / l + n 2^-24 max |v| / l,  s = 2^-16 |q| |k| scale,
     |dlse| <= s + 2^-20 + 2^-21 |lse|
with twice the term of subnormal weights: a weight for the product, relative to the scale vref of
the values, is rounded to 2^-25 at least, and 127 vref is at most twice the largest value's size.
(The reference's `size` holds the sums with n 2^-13 max |v|, of which 2^-11 is the last term.)
"""
import math

import numpy as np
import pytest
import torch

import _kv8_ref as ref
import _packed_ref
import exact_io_aware_26_gb300 as fa
from _parity import DTYPES, guarded, guards_intact, to_np64

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---------------------------------------------------------------- writing and reading

def special(T, H, d, seed):
    """Rows that are zero, tiny, huge, growing, with ties at half a step, NaN and infinite."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H, d)).astype(np.float32)
    kinds = [lambda g: g * 0, lambda g: g * 1e-6, lambda g: g * 1e-30, lambda g: g * 3000, lambda g: g * 1e6,
             lambda g: np.full_like(g, 127 / 64), lambda g: np.full_like(g, np.nextafter(np.float32(127 / 64), np.float32(9))),
             lambda g: np.arange(len(g)) * 0.25 - 7.875, lambda g: np.where(np.arange(len(g)) == 3, np.inf, g),
             lambda g: np.where(np.arange(len(g)) == 9, -np.inf, g), lambda g: np.where(np.arange(len(g)) == 31, np.nan, g),
             lambda g: np.where(np.arange(len(g)) == 60, np.nan, np.inf), lambda g: g * 1e-38]
    for n, (t, h) in enumerate(np.ndindex(T, H)):
        if n % 2 == 0 or T < 4:
            x[t, h] = kinds[(n // 2 + seed) % len(kinds)](x[t, h])
    return x


def put(cache, want, k, v, slots):
    """The same append on the GPU and by hand; k, v fp32 arrays of values of their type."""
    fa.kv8_append(k, v, dev(slots.astype(np.int32)), cache)
    ref.append(want, k.float().cpu().numpy(), v.float().cpu().numpy(), slots)


@pytest.mark.parametrize("H,d,dtype,page,kind,steps", [
    # tokens of three requests at each step; a negative number goes back that many first
    (1, 64, "bf16", 16, "normal", [(1, 0, 5), (1, 1, 1), (3, 20, 1)]),
    (3, 128, "f16", 32, "normal", [(37, 16, 1), (1, 1, 1), (1, 1, 1), (5, 5, 40)]),
    (2, 64, "f32", 64, "special", [(100, 3, 15), (1, 1, 1), (1, 1, 1), (1, 1, 1), (1, 1, 1), (20, 1, 2)]),
    (5, 128, "bf16", 16, "special", [(33, 4, 1), (1, 2, 3), (1, 1, 1), (7, 1, 1), (1, 1, 30)]),
    (8, 128, "f32", 128, "special", [(129, 200, 0), (1, 1, 1), (2, 2, 2), (-3, -5, 0), (6, 9, 1)]),
    (1, 64, "f16", 4096, "special", [(5, 9, 17), (-2, -9, -1), (4, 20, 3), (1, 1, 1)]),
    (12, 64, "bf16", 64, "normal", [(700, 1, 33), (1, 1, 1)]),
])
def test_append_and_gather(cuda_lib, H, d, dtype, page, kind, steps):
    """Requests that grow, a prompt, single tokens, drafts that are taken back; every byte of the
    cache is as by hand, among pages that hold anything."""
    rng = np.random.default_rng(H + d + page)
    width = -(-max(sum(abs(s[r]) for s in steps) for r in range(3)) // page)
    pages = 3 * width + 2
    table = rng.permutation(pages)[:3 * width].reshape(3, width)
    want = rng.integers(0, 256, (pages, H, page // 16, ref.block_bytes(d))).astype(np.uint8)
    raw, cache = guarded(want.shape, torch.uint8)
    cache.copy_(torch.from_numpy(want))
    held = [0, 0, 0]
    for i, step in enumerate(steps):
        slots = []
        for r in range(3):
            if step[r] < 0:
                held[r] += step[r]
                continue
            at = np.arange(held[r], held[r] + step[r])
            slots.append(table[r][at // page] * page + at % page)
            held[r] += step[r]
        slots = np.concatenate(slots + [np.array([-1, -5])])  # and two that are left out
        T = len(slots)
        x = [special(T, H, d, 7 * i + s) if kind == "special" else rng.standard_normal((T, H, d)).astype(np.float32) for s in (0, 1)]
        packed = torch.cat([torch.from_numpy(s) for s in x], 1).to(DTYPES[dtype]).cuda()
        put(cache, want, packed[:, :H], packed[:, H:], slots)
        got = cache.cpu().numpy()
        assert np.array_equal(got, want), np.argwhere(got != want)[:5]
    assert guards_intact(raw)
    back = np.concatenate([table[r][np.arange(held[r]) // page] * page + np.arange(held[r]) % page for r in range(3)] + [[-1]])
    wk, wv = ref.slot_values(want, back, d)
    for out in ("f32", "bf16", "f16"):
        for heads_first in (False, True):
            raws, res = zip(*(guarded((H, len(back), d) if heads_first else (len(back), H, d), DTYPES[out]) for _ in (0, 1)))
            fa.kv8_gather(cache, dev(back.astype(np.int32)), d, dtype=DTYPES[out], heads_first=heads_first, out=res)
            assert all(map(guards_intact, raws))
            for g, w in zip(res, (wk, wv)):
                g = g.transpose(0, 1) if heads_first else g
                assert np.array_equal(to_np64(g), to_np64(torch.from_numpy(w).to(DTYPES[out])), equal_nan=True)
    assert fa.get_status() == fa.FA_OK


def test_values_are_within_a_step(cuda_lib):
    """Half a step of the block's scale, or, of a token that others joined, what the rounding to
    larger scales adds: half of each of them, less than a step of the last."""
    T, H, d = 64, 2, 128
    rng = np.random.default_rng(2)
    cache = fa.kv8_cache(4, H, d, page_size=16)
    k = torch.from_numpy(rng.standard_normal((T, H, d)) * np.linspace(0.01, 5, T)[:, None, None]).bfloat16().cuda()
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    for t in range(T):
        fa.kv8_append(k[t:t + 1], k[t:t + 1], slots[t:t + 1], cache)
    got = [to_np64(x) for x in fa.kv8_gather(cache, slots, d, dtype=torch.float32)]
    want = to_np64(k)
    whole = fa.kv8_cache(4, H, d, page_size=16)
    fa.kv8_append(k, k, slots, whole)
    once = to_np64(fa.kv8_gather(whole, slots, d, dtype=torch.float32)[0])
    for b in range(T // 16):
        rows = slice(16 * b, 16 * b + 16)
        scale = np.array([ref.scale_for(x) for x in np.abs(want[rows]).max((0, 2))])[:, None]
        assert np.all(np.abs(once[rows] - want[rows]) <= scale / 2)
        for g in got:
            assert np.all(np.abs(g[rows] - want[rows]) <= scale)


def test_slots_outside_the_cache_are_left_out_and_recorded(cuda_lib):
    k = torch.randn(4, 2, 64, device="cuda").bfloat16()
    cache = fa.kv8_cache(3, 2, 64, page_size=16)
    slots = torch.tensor([5, 48, 2 ** 31 - 1, 47], dtype=torch.int32, device="cuda")
    fa.kv8_append(k, k, slots, cache)
    assert fa.get_status() == fa.FA_ERR_INDEX and fa.get_status() == fa.FA_OK
    gk, gv = fa.kv8_gather(cache, slots, 64)
    assert fa.get_status() == fa.FA_ERR_INDEX
    assert float(gk[1:3].abs().sum()) == 0
    assert bool((gk[0] != 0).any()) and bool((gk[3] != 0).any())
    assert int((cache[1] != 0).sum()) == 0


def test_slots_that_are_not_as_they_should_be_touch_their_blocks_alone(cuda_lib):
    """Equal slots, and tokens of a block that are not neighbours: their blocks are void, the others
    are right."""
    T, H, d = 80, 2, 128
    x = torch.randn(T, 2 * H, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    k, v = x[:, :H], x[:, H:]
    slots = np.concatenate([[3] * 40, np.arange(64, 96), [7, 200, 8, 201, 3, 3, 7, 7]])
    cache = fa.kv8_cache(20, H, d, page_size=16)
    fa.kv8_append(k, v, dev(slots.astype(np.int32)), cache)
    assert fa.get_status() == fa.FA_OK
    want = np.zeros(cache.shape, np.uint8)
    ref.append(want, k[40:72].float().cpu().numpy(), v[40:72].float().cpu().numpy(), slots[40:72])
    got = cache.cpu().numpy()
    for blk in range(20):
        if blk not in (0, 200 // 16):
            assert np.array_equal(got[blk], want[blk])


# ---------------------------------------------------------------- attention

def build(kv, new, Hq, Hk, d, dtype, page, seed, spread=1.0, sizes=None):
    """A cache whose pages lie in random order among others that hold anything, the requests' values
    as the cache has them, and queries.  sizes: magnitude of each token's values, from 0 to 1 of the
    request on."""
    rng = np.random.default_rng(seed)
    have = [-(-n // page) for n in kv]
    pages, width = sum(have) + 3, max(max(have), 1) + 1
    order = rng.permutation(pages).astype(np.int32)
    start = rng.integers(0, 256, (pages, Hk, page // 16, ref.block_bytes(d))).astype(np.uint8)
    start[..., 32 * d:] = 0xFF  # scales of NaN, every token marked
    cache = dev(start)
    table = np.full((len(kv), width), -1, np.int32)
    ks, vs = [], []
    at = 0
    for r, n in enumerate(kv):
        table[r, :have[r]] = order[at:at + have[r]]
        at += have[r]
        x = rng.standard_normal((2, n, Hk, d)) * spread
        if sizes is not None and n:
            x *= sizes(np.arange(n) / n)[:, None, None]
        slots = dev((table[r][np.arange(n) // page] * page + np.arange(n) % page).astype(np.int32))
        if n:
            fa.kv8_append(dev(x[0].astype(np.float32)), dev(x[1].astype(np.float32)), slots, cache)
        got = fa.kv8_gather(cache, slots, d, dtype=torch.float32)
        ks.append(to_np64(got[0]))
        vs.append(to_np64(got[1]))
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((int(cu[-1]), Hq, d)) * spread).to(DTYPES[dtype])
    return q, cache, table, np.array(kv, np.int32), cu, ks, vs


def check(o, lse, want, dtype):
    wo, wl, size, slack = want
    s = 2.0 ** -16 * slack
    e = torch.finfo(DTYPES[dtype]).eps / 2
    got, gl = to_np64(o), to_np64(lse)
    bound = e * np.abs(wo) + (2.0 ** -11 + 2 * s[..., None] + 2.0 ** -20) * size + torch.finfo(DTYPES[dtype]).smallest_normal
    assert np.array_equal(np.isfinite(gl), np.isfinite(wl))
    assert np.all(np.abs(got - wo) <= bound), f"o: {(np.abs(got - wo) / bound).max():.3f} of the bound"
    f = np.isfinite(wl)
    assert np.all(gl[~f] == -np.inf) and np.all(got[~f] == 0)
    err = np.abs(gl[f] - wl[f])
    assert np.all(err <= s[f] + 2.0 ** -20 + 2.0 ** -21 * np.abs(wl[f])), f"lse: {err.max():.3e}"


def widened(table):
    """The table with room for 100,000 tokens of 16-token pages, which makes a call take the way in
    shares instead of clusters."""
    out = np.full((table.shape[0], 6250), -1, np.int32)
    out[:, :table.shape[1]] = table
    return out


ATTN = [  # kv, new, Hq, Hk, d, dtype, page, window
    ([1], [1], 1, 1, 64, "bf16", 16, 0),
    ([1], [1], 1, 1, 128, "f16", 64, 0),
    ([15, 16, 17], [1, 1, 1], 4, 4, 64, "f16", 16, 0),
    ([0, 1, 0, 33], [1, 1, 1, 1], 8, 2, 128, "bf16", 32, 0),     # requests without tokens
    ([5, 40], [0, 1], 2, 1, 64, "bf16", 16, 0),                   # no new tokens
    ([700], [1], 8, 1, 128, "bf16", 64, 0),                       # several shares of one tile
    ([3000, 17, 1029], [1, 1, 1], 12, 12, 64, "bf16", 64, 0),
    ([2500, 64, 900], [1, 1, 1], 10, 2, 128, "f16", 128, 0),
    ([100, 257, 64, 31], [1, 4, 3, 2], 8, 4, 64, "f16", 16, 0),   # several tokens, one tile
    ([300, 6, 513], [5, 6, 1], 6, 2, 128, "bf16", 32, 0),         # rows of 15, 18 and 3: two columns blocks
    ([400, 90], [8, 3], 32, 4, 128, "bf16", 64, 0),               # 64 rows: two tiles of 32
    ([130, 35], [35, 35], 6, 3, 64, "f16", 16, 0),                # a prompt, whole
    ([3, 2], [5, 2], 4, 2, 64, "bf16", 16, 0),                    # more queries than tokens: rows that see nothing
    ([500, 20, 1], [1, 1, 1], 4, 1, 128, "f16", 16, 33),
    ([777, 100], [6, 9], 8, 2, 64, "bf16", 64, 50),
    ([900], [4], 16, 2, 128, "bf16", 32, 1),                      # each sees itself only
    ([4000], [1], 24, 1, 64, "f16", 4096, 0),                     # 24 rows of one token
    (list(range(0, 150)), [1] * 150, 3, 1, 64, "bf16", 16, 0),    # more requests than a CTA keeps
    ([i % 41 for i in range(350)], [1] * 350, 2, 2, 64, "f16", 16, 0),  # more tiles than CTAs
    ([600] * 40, [2] * 40, 12, 4, 128, "bf16", 64, 100),
    ([70000], [1], 3, 1, 64, "f16", 64, 0),                       # one tile in hundreds of shares
    ([9000, 50000], [2, 3], 20, 2, 128, "bf16", 128, 0),
    ([12000] + [20 + i for i in range(330)], [1] * 331, 2, 1, 128, "f16", 16, 0),  # and among many of one unit
]


@pytest.mark.parametrize("kv,new,Hq,Hk,d,dtype,page,window", ATTN)
def test_attention(cuda_lib, kv, new, Hq, Hk, d, dtype, page, window):
    q, cache, table, lens, cu, k, v = build(kv, new, Hq, Hk, d, dtype, page, sum(kv) + Hq)
    want = ref.attention(to_np64(q), k, v, lens, cu, 0.3, window)
    raw_o, o = guarded((q.shape[0], Hq, d), DTYPES[dtype])
    raw_l, lse = guarded((q.shape[0], Hq), torch.float32)
    single = all(n == 1 for n in new)
    for cu_q in ([None] if single else []) + [dev(cu)]:
        o.fill_(float("nan"))
        fa.kv8_attention(q.cuda(), cache, dev(table), dev(lens), cu_q=cu_q, max_q_len=max(new), scale=0.3, window=window,
                         out=o, lse=lse)
        assert fa.get_status() == fa.FA_OK
        check(o, lse, want, dtype)
        assert guards_intact(raw_o) and guards_intact(raw_l)
    o.fill_(float("nan"))
    raw_w, ws = guarded((16 << 20,), torch.uint8, fill=0xFF)
    fa.kv8_attention(q.cuda(), cache, dev(widened(table)), dev(lens), cu_q=dev(cu), max_q_len=max(new), scale=0.3,
                     window=window, out=o, lse=lse, workspace=ws[-ws.data_ptr() % 256:])
    assert fa.get_status() == fa.FA_OK
    check(o, lse, want, dtype)
    assert guards_intact(raw_o) and guards_intact(raw_l) and guards_intact(raw_w, fill=0xFF)
    for hint in (1, 2, 100):  # the hint alone changes the tile height, not the result
        o2, l2 = fa.kv8_attention(q.cuda(), cache, dev(table), dev(lens), cu_q=dev(cu), max_q_len=hint, scale=0.3, window=window)
        check(o2, l2, want, dtype)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("spread,scale", [(30.0, 0.5), (1e-3, 1.0), (100.0, 1e-4)])
def test_attention_of_large_and_small_scores(cuda_lib, spread, scale, wide):
    q, cache, table, lens, cu, k, v = build([333, 70], [1, 1], 8, 2, 128, "bf16", 16, 5, spread)
    want = ref.attention(to_np64(q), k, v, lens, cu, scale, 0)
    o, lse = fa.kv8_attention(q.cuda(), cache, dev(widened(table) if wide else table), dev(lens), scale=scale)
    check(o, lse, want, "bf16")


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("d,Hq,sizes", [(64, 4, lambda x: 1e-6 ** x), (128, 2, lambda x: 1e4 * 1e-12 ** (1 - x)),
                                        (128, 16, lambda x: np.where((x * 12).astype(int) % 2, 3000.0, 1e-5)),
                                        (64, 2, lambda x: np.where(x < 0.5, 0.0, 1.0))])
def test_blocks_of_very_different_scales(cuda_lib, d, Hq, sizes, wide):
    """Values whose sizes fall, rise and jump by many powers of two from block to block: each counts
    with its weight, relative to what the row's own weights make of all of them."""
    q, cache, table, lens, cu, k, v = build([500, 97], [1, 2], Hq, 1, d, "bf16", 16, 4, sizes=sizes)
    q = (q.float() * 1e-6).bfloat16()  # even weights
    want = ref.attention(to_np64(q), k, v, lens, cu, 1.0, 0)
    o, lse = fa.kv8_attention(q.cuda(), cache, dev(widened(table) if wide else table), dev(lens), cu_q=dev(cu), max_q_len=2, scale=1.0)
    check(o, lse, want, "bf16")


def test_a_small_value_with_all_of_the_weight(cuda_lib):
    """The key that wins stands among small values, behind a block of large ones and before one: the
    result is its value, to the weights' rounding."""
    d, n = 64, 96
    k, v = np.zeros((n, 1, d), np.float32), np.full((n, 1, d), 8000.0, np.float32)
    v[32:64] = np.random.default_rng(3).standard_normal((32, 1, d)) * 1e-4
    k[40, 0, 0] = 100.0
    cache = fa.kv8_cache(6, 1, d, page_size=16)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    fa.kv8_append(dev(k), dev(v), slots, cache)
    held = to_np64(fa.kv8_gather(cache, slots, d, dtype=torch.float32)[1])
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 2.0
    table = torch.arange(6, dtype=torch.int32, device="cuda")[None]
    for t in (table, torch.cat([table, torch.full((1, 6244), -1, dtype=torch.int32, device="cuda")], 1)):
        o, lse = fa.kv8_attention(q, cache, t, torch.tensor([n], dtype=torch.int32, device="cuda"), scale=1.0)
        # the other weights are e^-200
        assert np.all(np.abs(to_np64(o)[0, 0] - held[40, 0]) <= (2.0 ** -8 + 2.0 ** -11) * np.abs(held[40, 0]))
        assert abs(float(lse) - 200.0) < 1e-3 + 200 * 2.0 ** -9


@pytest.mark.parametrize("n", [2, 30, 200])
def test_small_weights_of_small_values(cuda_lib, n):
    """One token has nearly all of the weight and a value of 0, the others have e^-12 of it each and values
    below 1/2: they are the result, of which no bits are lost to their block's small scale."""
    d, pages = 64, -(-n // 16)
    k, v = np.zeros((n, 1, d), np.float32), np.full((n, 1, d), 0.4375, np.float32)
    k[0, 0, 0], v[0] = 12.0, 0.0
    cache = fa.kv8_cache(pages, 1, d, page_size=16)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    fa.kv8_append(dev(k), dev(v), slots, cache)
    held = [to_np64(x) for x in fa.kv8_gather(cache, slots, d, dtype=torch.float32)]
    q = torch.zeros(1, 2, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    want = ref.attention(to_np64(q), [held[0]], [held[1]], [n], [0, 1], 1.0, 0)
    for t in (table, torch.cat([table, torch.full((1, 6250 - pages), -1, dtype=torch.int32, device="cuda")], 1)):
        check(*fa.kv8_attention(q, cache, t, torch.tensor([n], dtype=torch.int32, device="cuda"), scale=1.0), want, "bf16")


def test_queries_outside_fp16s_range(cuda_lib):
    q, cache, table, lens, cu, k, v = build([200], [1], 4, 1, 64, "bf16", 16, 6)
    for size in (2.0 ** 100, 2.0 ** -100):
        want = ref.attention(to_np64(q) * size, k, v, lens, cu, 0.125 / size, 0)
        o, lse = fa.kv8_attention((q.float() * size).bfloat16().cuda(), cache, dev(table), dev(lens), scale=0.125 / size)
        check(o, lse, want, "bf16")


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_keys_and_values_reach_only_the_rows_that_see_them(cuda_lib, wide, d):
    kv, new, Hk = [40, 60], [4, 4], 2
    q, cache, table, lens, cu, k, v = build(kv, new, 4, Hk, d, "bf16", 16, 9)
    clean = ref.attention(to_np64(q), k, v, lens, cu, 0.3, 0)
    row = torch.zeros(1, Hk, d, device="cuda")
    for r, tok, side in ((0, 38, 0), (1, 58, 1)):  # the last query but one of each request sees them first
        bad = [dev(x[r][tok:tok + 1].astype(np.float32)) for x in (k, v)]
        bad[side] = bad[side] + row
        bad[side][0, 0, 7] = float("nan")
        slot = int(table[r, tok // 16]) * 16 + tok % 16
        fa.kv8_append(bad[0], bad[1], torch.tensor([slot], dtype=torch.int32, device="cuda"), cache)
    o, lse = fa.kv8_attention(q.cuda(), cache, dev(widened(table) if wide else table), dev(lens), cu_q=dev(cu), max_q_len=4, scale=0.3)
    o, lse = to_np64(o), to_np64(lse)
    for r in range(2):
        for i in range(4):
            at = cu[r] + i
            assert np.all(np.isfinite(o[at, 2:])) and np.all(np.isfinite(lse[at, 2:]))  # the other head
            if i < 2:
                assert np.all(np.isfinite(o[at])) and np.abs(o[at] - clean[0][at]).max() < 0.05
            else:
                assert np.isnan(o[at, :2]).all() and np.isnan(lse[at, :2]).all() == (r == 0)


def test_bad_pages_and_lengths_are_recorded_and_contribute_nothing(cuda_lib):
    q, cache, table, lens, cu, k, v = build([100, 50], [1, 1], 4, 2, 64, "bf16", 16, 10)
    want = ref.attention(to_np64(q), k, v, lens, cu, 0.3, 0)
    keep = [j for j in range(100) if j // 16 != 2]
    left = ref.attention(to_np64(q)[:1], [k[0][keep]], [v[0][keep]], [len(keep)], [0, 1], 0.3, 0)
    for bad in (-1, cache.shape[0], 2 ** 31 - 1, -(2 ** 31)):
        t = table.copy()
        t[0, 2] = bad
        for t in (t, widened(t)):
            o, lse = fa.kv8_attention(q.cuda(), cache, dev(t), dev(lens), scale=0.3)
            assert fa.get_status() == fa.FA_ERR_INDEX
            check(o[1:], lse[1:], tuple(w[1:] for w in want), "bf16")
            check(o[:1], lse[:1], left, "bf16")
    long = np.array([table.shape[1] * 16 + 5, 50], np.int32)  # beyond the table: cut to it
    o, lse = fa.kv8_attention(q.cuda(), cache, dev(np.where(table < 0, 0, table)), dev(long), scale=0.3)
    assert fa.get_status() == fa.FA_ERR_INDEX
    check(o[1:], lse[1:], tuple(w[1:] for w in want), "bf16")


def test_rows_outside_and_strides(cuda_lib):
    """Rows of no request stay; queries and results inside packed rows, a cache of one layer among
    several."""
    q, cache, table, lens, cu, k, v = build([70, 300], [1, 2], 6, 3, 128, "bf16", 32, 13)
    want = ref.attention(to_np64(q), k, v, lens, cu, 128 ** -0.5, 0)
    packed = torch.zeros(5, 12, 128, dtype=torch.bfloat16, device="cuda")
    packed[:3, 3:9] = q.cuda()
    layers = torch.zeros((cache.shape[0], 3) + tuple(cache.shape[1:]), dtype=torch.uint8, device="cuda")
    layers[:, 1] = cache
    outp = torch.full((5, 12, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 6), 9.0, device="cuda")
    o, _ = fa.kv8_attention(packed[:, 3:9], layers[:, 1], dev(table), dev(lens), cu_q=dev(cu), max_q_len=2, out=outp[:, 3:9], lse=lse)
    check(o[:3], lse[:3], want, "bf16")
    assert bool((outp[:, :3] == 9).all()) and bool((outp[:, 9:] == 9).all())
    assert bool((outp[3:] == 9).all()) and bool((lse[3:] == 9).all())


def test_a_cache_beyond_32_bit_offsets(cuda_lib):
    H, d, page = 8, 128, 64
    pages = (2 ** 32 + 2 ** 28) // (H * (page // 16) * ref.block_bytes(d))
    cache = torch.zeros(pages, H, page // 16, ref.block_bytes(d), dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(4)
    T = 100
    k, v = (torch.randn(T, H, d, generator=g).bfloat16().cuda() for _ in range(2))
    ids = [pages - 1, 3]
    slots = np.array([ids[t // page] * page + t % page for t in range(T)])
    fa.kv8_append(k, v, dev(slots.astype(np.int32)), cache)
    small = np.zeros((2,) + tuple(cache.shape[1:]), np.uint8)
    ref.append(small, k.float().cpu().numpy(), v.float().cpu().numpy(), np.arange(T))
    assert np.array_equal(torch.stack([cache[i] for i in ids]).cpu().numpy(), small)
    gk, gv = fa.kv8_gather(cache, dev(slots.astype(np.int32)), d, dtype=torch.float32)
    wk, wv = ref.slot_values(small, np.arange(T), d)
    assert np.array_equal(to_np64(gk), wk) and np.array_equal(to_np64(gv), wv)
    q = torch.randn(1, H, d, generator=g).bfloat16()
    want = ref.attention(to_np64(q), [wk], [wv], [T], [0, 1], d ** -0.5, 0)
    o, lse = fa.kv8_attention(q.cuda(), cache, dev(np.array([ids], np.int32)), dev(np.array([T], np.int32)))
    check(o, lse, want, "bf16")


@pytest.mark.parametrize("wide", [False, True])
def test_streams_graphs_and_shared_workspaces(cuda_lib, wide):
    sets = []
    for seed, kv in ((20, [3000, 40]), (21, [5, 1800])):
        q, cache, table, lens, cu, _, _ = build(kv, [1, 1], 8, 2, 128, "bf16", 64, seed)
        args = (q.cuda(), cache, dev(widened(table) if wide else table), dev(lens))
        sets.append((args, fa.kv8_attention(*args)))
    torch.cuda.synchronize()
    side, got = [torch.cuda.Stream() for _ in sets], [None, None]
    for _ in range(10):
        for i, (args, _) in enumerate(sets):
            got[i] = fa.kv8_attention(*args, stream=side[i])
    torch.cuda.synchronize()
    for g, (_, w) in zip(got, sets):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    ws = torch.full((16 << 20,), 255, dtype=torch.uint8, device="cuda")
    graphs = []
    for args, _ in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = fa.kv8_attention(*args, workspace=ws)
        graphs.append((graph, res))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (_, g), (_, w) in zip(graphs, sets):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    assert fa.get_status() == fa.FA_OK


# ---------------------------------------------------------------- together

def test_prompts_then_tokens(cuda_lib):
    """Serving: prompts of different lengths through the packed attention and into the 8-bit cache,
    then steps of single tokens replayed from a graph, then new rows over what is cached, read back.
    Each step's attention is that of the values the cache holds."""
    Hq, Hk, d, page, pages, R, width = 8, 2, 128, 16, 64, 3, 20
    g = torch.Generator().manual_seed(0)
    rows = lambda n: torch.randn(n, Hq + 2 * Hk, d, generator=g).bfloat16().cuda()
    freqs = fa.rope_freqs(d)
    w = torch.ones(d, device="cuda")
    cache = fa.kv8_cache(pages, Hk, d, page_size=page)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table, stack = torch.full((R, width), -1, dtype=torch.int32, device="cuda"), torch.arange(pages, dtype=torch.int32, device="cuda")
    lens, count = i32(0, 0, 0), i32(pages, 0, 0)

    def step(x, new, T):
        plan = fa.paged_plan(lens, new, table, stack, count, page, T, out=dict(kv_lens=lens, cu_q=torch.empty(R + 1, dtype=torch.int32, device="cuda"),
                             positions=torch.empty(T, dtype=torch.int32, device="cuda"), slots=torch.empty(T, dtype=torch.int32, device="cuda"), counts=count))
        q, k = fa.qk_norm_rope(x[None, :, :Hq], x[None, :, Hq:Hq + Hk], w, w, freqs, positions=plan["positions"][None], heads_first=False)
        fa.kv8_append(k[0], x[:, Hq + Hk:], plan["slots"], cache)
        return plan, q[0], k[0]

    prompts = [45, 7, 100]
    x = rows(sum(prompts))
    plan, q, k = step(x, i32(*prompts), sum(prompts))
    o, lse = fa.attention_fwd_packed(q, k, x[:, Hq + Hk:], plan["cu_q"])
    want = _packed_ref.forward(q.cpu(), k.cpu(), x[:, Hq + Hk:].cpu(), prompts, prompts, True, d ** -0.5, 2.0 ** -8, 0.0)
    assert bool(((o.double().cpu() - want[0]).abs() <= want[2]).all())

    def held():  # what the cache holds of each request
        out = []
        for r, n in enumerate(lens.tolist()):
            at = torch.arange(n, device="cuda")
            out.append((table[r][at // page] * page + at % page).int())
        return out

    xs = rows(R)
    ones = i32(1, 1, 1)
    graph = torch.cuda.CUDAGraph()
    warm = torch.cuda.Stream()
    state = [t.clone() for t in (lens, table, stack, count, cache)]
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):  # the calls' first time is not captured
        p, q, _ = step(xs, ones, R)
        fa.kv8_attention(q, cache, table, lens, cu_q=p["cu_q"])
    torch.cuda.current_stream().wait_stream(warm)
    for t, s in zip((lens, table, stack, count, cache), state):
        t.copy_(s)
    with torch.cuda.graph(graph):
        p, q, _ = step(xs, ones, R)
        o, lse = fa.kv8_attention(q, cache, table, lens, cu_q=p["cu_q"])
    for t, s in zip((lens, table, stack, count, cache), state):
        t.copy_(s)
    for i in range(6):
        xs.copy_(rows(R))
        graph.replay()
        torch.cuda.synchronize()
        kv = [[to_np64(a) for a in fa.kv8_gather(cache, s, d, dtype=torch.float32)] for s in held()]
        assert lens.tolist() == [n + i + 1 for n in prompts]
        check(o, lse, ref.attention(to_np64(q), [a for a, _ in kv], [b for _, b in kv], lens.tolist(), [0, 1, 2, 3], d ** -0.5, 0), "bf16")
    # pieces of prompts over what is cached, by both attentions
    more = [20, 33, 1]
    x = rows(sum(more))
    plan, q, _ = step(x, i32(*more), sum(more))
    kv = [fa.kv8_gather(cache, s, d, dtype=torch.bfloat16) for s in held()]
    k16, v16 = (torch.cat([a[i] for a in kv]) for i in (0, 1))
    total = lens.tolist()
    cu_k = i32(0, total[0], total[0] + total[1], sum(total))
    a, la = fa.attention_fwd_packed(q, k16, v16, plan["cu_q"], cu_k)
    b, lb = fa.kv8_attention(q, cache, table, lens, cu_q=plan["cu_q"], max_q_len=33)
    want = _packed_ref.forward(q.cpu(), k16.cpu(), v16.cpu(), more, total, True, d ** -0.5, 2.0 ** -8, 0.0)
    for got, l in ((a, la), (b, lb)):
        assert bool(((got.double().cpu() - want[0]).abs() <= want[2]).all()) and bool(((l.double().cpu() - want[1]).abs() <= want[3]).all())
    assert fa.get_status() == fa.FA_OK


def test_refusals_of_the_binding(cuda_lib):
    k = torch.randn(4, 2, 64, device="cuda").bfloat16()
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    cache, four = fa.kv8_cache(3, 2, 64, page_size=16), fa.kv4_cache(3, 2, 64, page_size=16)
    table, lens, q = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), slots[:1], k[:1]
    for call, error in [
        (lambda: fa.kv8_append(k, k, slots, four), ValueError),
        (lambda: fa.kv4_append(k, k, slots, cache), ValueError),
        (lambda: fa.kv8_append(k, k[:, :1], slots, cache), ValueError),
        (lambda: fa.kv8_append(k, k, slots.long(), cache), TypeError),
        (lambda: fa.kv8_append(k.double(), k, slots, cache), TypeError),
        (lambda: fa.kv8_append(k, k, slots, cache.cpu()), ValueError),
        (lambda: fa.kv8_gather(cache, slots, 128), ValueError),
        (lambda: fa.kv8_attention(q, four, table, lens), ValueError),
        (lambda: fa.kv8_attention(q.float(), cache, table, lens), TypeError),
        (lambda: fa.kv8_attention(q, cache, table, lens, out=q), fa.FaError),
        (lambda: fa.kv8_attention(q, cache, table, lens, window=-1), fa.FaError),
        (lambda: fa.kv8_attention(q[:, :1], cache, table, lens), fa.FaError),
        (lambda: fa.kv8_cache(3, 2, 96), ValueError),
        (lambda: fa.kv8_cache(3, 2, 64, page_size=24), ValueError),
    ]:
        with pytest.raises(error):
            call()
