"""The 4-bit cache, the attention that reads it, and block tables, against plain
64-bit (and whole-number) implementations.

Codes and pairs are whole numbers and must be equal.  The attention's bounds
(e = eps(type) / 2; w a weight, l their sum, at least 1 relative to the largest score):
  weights are rounded to fp16 for the product: 2^-11 of each, or 2^-25 where subnormal;
  a score is off by d roundings of 2^-23 of its terms (fp32 accumulation) and the exponential
  by 2^-22, twice that for numerator and sum together:
     |do| <= e |o| + (2^-11 + 2 s + 2^-20) sum w |v| / l + n 2^-25 max |v| / l,  s = 2^-16 |q| |k| scale,
     |dlse| <= s + 2^-20 + 2^-21 |lse|.
(The reference's `size` holds the sums with n 2^-14 max |v|, of which 2^-11 is the last term.)
"""
import math

import numpy as np
import pytest
import torch

import _ops_ref as ref
import exact_io_aware_26_gb300 as fa
from _parity import DTYPES, guarded, guards_intact, to_np64

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- writing and reading

def special(T, H, d, seed):
    """Rows whose groups are constant, tiny, huge, one-sided, with ties, NaN and infinite."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H, d)).astype(np.float32)
    kinds = [lambda g: np.full_like(g, 1.5), lambda g: g * 0, lambda g: g * 1e-6, lambda g: g * 1e-30,
             lambda g: g * 3000, lambda g: g * 1e6, lambda g: np.abs(g) + 100, lambda g: np.round(g * 4) / 4,
             lambda g: np.arange(len(g)) * 0.5 - 7.75, lambda g: np.where(np.arange(len(g)) == 3, np.inf, g),
             lambda g: np.where(np.arange(len(g)) == 9, -np.inf, g), lambda g: np.where(np.arange(len(g)) == 31, np.nan, g)]
    n = 0
    for t in range(T):
        for h in range(H):
            for c in range(0, d, 32):
                if n % 2 == 0:
                    x[t, h, c:c + 32] = kinds[n // 2 % len(kinds)](x[t, h, c:c + 32])
                n += 1
    return x


@pytest.mark.parametrize("T,H,d,dtype,page,kind", [
    (1, 1, 64, "bf16", 16, "normal"), (17, 3, 128, "f16", 32, "normal"), (100, 2, 64, "f32", 64, "special"),
    (65, 5, 128, "bf16", 16, "special"), (300, 8, 128, "f32", 128, "normal"), (33, 1, 64, "f16", 4096, "normal"),
])
def test_append_and_gather(cuda_lib, T, H, d, dtype, page, kind):
    rng = np.random.default_rng(T + d)
    pages = -(-T // page) + 3
    raw = [special(T, H, d, 7 * i + T) if kind == "special" else rng.standard_normal((T, H, d)).astype(np.float32) for i in (0, 1)]
    packed = torch.cat([torch.from_numpy(r) for r in raw], 1).to(DTYPES[dtype]).cuda()  # strided views
    k, v = packed[:, :H], packed[:, H:]
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    left_out = rng.random(T) < 0.2 if T > 1 else np.zeros(1, bool)
    given = np.where(left_out, -1, slots).astype(np.int32)
    before = rng.integers(0, 255, (pages, H, page // 16, ref.block_bytes(d))).astype(np.uint8)
    raw_c, cache = guarded(before.shape, torch.uint8)
    cache.copy_(torch.from_numpy(before))
    fa.kv4_append(k, v, torch.from_numpy(given).cuda(), cache)
    want = before.copy()
    half = want.shape[3] // 2
    at = (slots // page, slice(None), slots % page // 16, slots % 16)
    for i, x in enumerate((k, v)):
        c, s, b = ref.quantise(x.float().cpu().numpy())
        view = want[..., i * half:(i + 1) * half]
        codes = view[..., :16 * d // 2].reshape(pages, H, page // 16, 16, d // 2)
        pairs = view[..., 16 * d // 2:].reshape(pages, H, page // 16, 16, -1)
        assert np.shares_memory(view, want)
        cb = c[..., 0::2] | (c[..., 1::2] << 4)
        pb = np.ascontiguousarray(np.stack([s, b], -1)).view(np.uint8).reshape(T, H, -1)
        # NaN pairs: any NaN will do
        for t in np.flatnonzero(~left_out):
            p, blk, row = slots[t] // page, slots[t] % page // 16, slots[t] % 16
            want[p, :, blk, i * half + row * d // 2:i * half + (row + 1) * d // 2] = cb[t]
            w = pb.shape[-1]
            o = i * half + 16 * d // 2 + row * w
            want[p, :, blk, o:o + w] = pb[t]
    got = cache.cpu().numpy()
    same = got == want
    if not same.all():  # NaN pairs differ in their bits: compare those as numbers
        pick = lambda a: np.concatenate([np.ascontiguousarray(a[..., i * half + 8 * d:(i + 1) * half]).view(np.float16) for i in (0, 1)], -1)
        codes = lambda a: np.concatenate([a[..., i * half:i * half + 8 * d] for i in (0, 1)], -1)
        assert np.array_equal(codes(got), codes(want))
        assert np.array_equal(pick(got), pick(want), equal_nan=True)
    assert guards_intact(raw_c)
    # what the codes stand for, in each layout and type
    for out in ("f32", "f16", "bf16"):
        for first in (False, True):
            gk, gv = fa.kv4_gather(cache, torch.from_numpy(given).cuda(), d, dtype=DTYPES[out], heads_first=first)
            for g, w in zip((gk, gv), ref.slot_values(got, slots, d)):
                g = g.transpose(0, 1) if first else g
                w = np.where(left_out[:, None, None], 0, w)
                assert np.array_equal(to_np64(g), to_np64(torch.from_numpy(w).to(DTYPES[out])), equal_nan=True)
    # and how near they are: half a step, and the fp16 roundings of scale, base and value
    if kind == "normal":
        for g, x in zip(fa.kv4_gather(cache, torch.from_numpy(slots).cuda(), d, dtype=torch.float32), (k, v)):
            err = np.abs(to_np64(g) - to_np64(x))[~left_out]
            _, s, b = ref.quantise(x.float().cpu().numpy())
            s, b = (np.repeat(np.abs(a.astype(np.float64)), 32, -1)[~left_out] for a in (s, b))
            assert np.all(err <= s / 32 + 2.0 ** -11 * (3 * s + 2 * b))
    assert fa.get_status() == fa.FA_OK


def test_slots_outside_the_cache_are_left_out_and_recorded(cuda_lib):
    k = torch.randn(4, 2, 64, device="cuda").bfloat16()
    cache = fa.kv4_cache(3, 2, 64, page_size=16)
    slots = torch.tensor([5, 48, 2 ** 31 - 1, 47], dtype=torch.int32, device="cuda")
    fa.kv4_append(k, k, slots, cache)
    assert fa.get_status() == fa.FA_ERR_INDEX and fa.get_status() == fa.FA_OK
    gk, gv = fa.kv4_gather(cache, slots, 64)
    assert fa.get_status() == fa.FA_ERR_INDEX
    assert float(gk[1:3].abs().sum()) == 0
    assert bool((gk[0] != 0).any()) and bool((gk[3] != 0).any())
    assert int((cache[1] != 0).sum()) == 0


# ---------------------------------------------------------------- attention

def build(kv, new, Hq, Hk, d, dtype, page, seed, spread=1.0):
    """A cache whose pages lie in random order among others full of NaN, and its queries."""
    rng = np.random.default_rng(seed)
    have = [-(-n // page) for n in kv]
    pages = sum(have) + 3
    width = max(max(have), 1) + 1
    order = rng.permutation(pages).astype(np.int32)
    cache = np.full((pages, Hk, page // 16, ref.block_bytes(d)), 0x7E, np.uint8)  # NaN pairs
    table = np.full((len(kv), width), -1, np.int32)
    half = cache.shape[3] // 2
    at = 0
    for r, n in enumerate(kv):
        x = [(rng.standard_normal((n, Hk, d)) * spread).astype(np.float32) for _ in (0, 1)]
        if not n:
            continue
        full = ref.cache_of(x[0], x[1], page)
        for i in range(have[r]):
            table[r, i] = order[at]
            cache[order[at]] = full[i]
            # behind the last token: NaN, as a reused page may hold
            for row in range(max(0, n - i * page), page):
                blk, o = row // 16, row % 16 * (d // 8)
                for hs in (0, half):
                    cache[order[at], :, blk, hs + 8 * d + o:hs + 8 * d + o + d // 8] = 0x7E
            at += 1
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((int(cu[-1]), Hq, d)) * spread).to(DTYPES[dtype])
    return q, cache, table, np.array(kv, np.int32), cu


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
    ([20000, 40], [4, 1], 4, 1, 64, "bf16", 32, 0),               # the same with 16 rows
    ([12000] + [20 + i for i in range(330)], [1] * 331, 2, 1, 128, "f16", 16, 0),  # and among many of one unit
]


def widened(table):
    """The table with room for 100,000 tokens of 16-token pages: what a call has to reckon
    with, which makes it take the way in shares instead of clusters."""
    out = np.full((table.shape[0], 6250), -1, np.int32)
    out[:, :table.shape[1]] = table
    return out


@pytest.mark.parametrize("kv,new,Hq,Hk,d,dtype,page,window", ATTN)
def test_attention(cuda_lib, kv, new, Hq, Hk, d, dtype, page, window):
    q, cache, table, lens, cu = build(kv, new, Hq, Hk, d, dtype, page, sum(kv) + Hq)
    want = ref.attention(to_np64(q), cache, table, lens, cu, 0.3, window, d)
    raw_o, o = guarded((q.shape[0], Hq, d), DTYPES[dtype])
    raw_l, lse = guarded((q.shape[0], Hq), torch.float32)
    dev = lambda a: torch.from_numpy(a).cuda()
    single = all(n == 1 for n in new)
    for cu_q in ([None] if single else []) + [dev(cu)]:
        o.fill_(float("nan"))
        fa.kv4_attention(q.cuda(), dev(cache), dev(table), dev(lens), cu_q=cu_q, max_q_len=max(new), scale=0.3,
                         window=window, out=o, lse=lse)
        assert fa.get_status() == fa.FA_OK
        check(o, lse, want, dtype)
        assert guards_intact(raw_o) and guards_intact(raw_l)
    o.fill_(float("nan"))
    ws_bytes = 16 << 20
    raw_w, ws = guarded((ws_bytes,), torch.uint8, fill=0xFF)
    aligned = ws[-ws.data_ptr() % 256:]
    fa.kv4_attention(q.cuda(), dev(cache), dev(widened(table)), dev(lens), cu_q=dev(cu), max_q_len=max(new), scale=0.3,
                     window=window, out=o, lse=lse, workspace=aligned)
    assert fa.get_status() == fa.FA_OK
    check(o, lse, want, dtype)
    assert guards_intact(raw_o) and guards_intact(raw_l) and guards_intact(raw_w, fill=0xFF)
    # the hint alone changes the tile height, not the result
    for hint in (1, 2, 100):
        o2, l2 = fa.kv4_attention(q.cuda(), dev(cache), dev(table), dev(lens), cu_q=dev(cu), max_q_len=hint, scale=0.3,
                                  window=window)
        check(o2, l2, want, dtype)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("spread,scale", [(30.0, 0.5), (1e-3, 1.0), (100.0, 1e-4)])
def test_attention_of_large_and_small_scores(cuda_lib, spread, scale, wide):
    q, cache, table, lens, cu = build([333, 70], [1, 1], 8, 2, 128, "bf16", 16, 5, spread)
    want = ref.attention(to_np64(q), cache, table, lens, cu, scale, 0, 128)
    dev = lambda a: torch.from_numpy(a).cuda()
    o, lse = fa.kv4_attention(q.cuda(), dev(cache), dev(widened(table) if wide else table), dev(lens), scale=scale)
    check(o, lse, want, "bf16")


def test_queries_outside_fp16s_range(cuda_lib):
    q, cache, table, lens, cu = build([200], [1], 4, 1, 64, "bf16", 16, 6)
    dev = lambda a: torch.from_numpy(a).cuda()
    for size in (2.0 ** 100, 2.0 ** -100):
        want = ref.attention(to_np64(q) * size, cache, table, lens, cu, 0.125 / size, 0, 64)
        o, lse = fa.kv4_attention((q.float() * size).bfloat16().cuda(), dev(cache), dev(table), dev(lens), scale=0.125 / size)
        check(o, lse, want, "bf16")


@pytest.mark.parametrize("wide", [False, True])
def test_rising_scores_move_the_maximum(cuda_lib, wide):
    """Keys that grow with the position: every block raises the running maximum."""
    n, d = 1000, 64
    rng = np.random.default_rng(8)
    k = (np.ones((n, 1, d)) * np.linspace(0, 40, n)[:, None, None]).astype(np.float32)
    v = rng.standard_normal((n, 1, d)).astype(np.float32)
    cache = ref.cache_of(k, v, 16)
    table = np.arange(cache.shape[0], dtype=np.int32)[None]
    q = torch.ones(1, 2, d, dtype=torch.float16)
    lens, cu = np.array([n], np.int32), np.array([0, 1], np.int32)
    want = ref.attention(to_np64(q), cache, table, lens, cu, 0.5, 0, d)
    dev = lambda a: torch.from_numpy(a).cuda()
    o, lse = fa.kv4_attention(q.cuda(), dev(cache), dev(widened(table) if wide else table), dev(lens), scale=0.5)
    check(o, lse, want, "f16")


@pytest.mark.parametrize("wide", [False, True])
def test_nan_keys_and_values_reach_only_the_rows_that_see_them(cuda_lib, wide):
    kv, new, d = [40, 60], [4, 4], 64
    q, cache, table, lens, cu = build(kv, new, 2, 1, d, "bf16", 16, 9)
    clean = ref.attention(to_np64(q), cache, table, lens, cu, 0.3, 0, d)
    half = cache.shape[3] // 2
    for r, tok, side in ((0, 38, 0), (1, 58, 1)):  # the last query but one of each request sees them first
        p, row = table[r, tok // 16], tok % 16
        cache[p, 0, 0, side * half + 8 * d + row * 8:side * half + 8 * d + row * 8 + 4] = 0x7E
    dev = lambda a: torch.from_numpy(a).cuda()
    o, lse = fa.kv4_attention(q.cuda(), dev(cache), dev(widened(table) if wide else table), dev(lens), cu_q=dev(cu),
                              max_q_len=4, scale=0.3)
    o, lse = to_np64(o), to_np64(lse)
    for r in range(2):
        for i in range(4):
            row = cu[r] + i
            if i < 2:
                assert np.all(np.isfinite(o[row])) and np.abs(o[row] - clean[0][row]).max() < 0.02
            else:
                assert np.isnan(o[row][:, :32]).all()


def test_bad_pages_and_lengths_are_recorded_and_contribute_nothing(cuda_lib):
    q, cache, table, lens, cu = build([100, 50], [1, 1], 4, 2, 64, "bf16", 16, 10)
    want = ref.attention(to_np64(q), cache, table, lens, cu, 0.3, 0, 64)
    dev = lambda a: torch.from_numpy(a).cuda()
    for bad in (-1, cache.shape[0], 2 ** 31 - 1, -(2 ** 31)):
        t = table.copy()
        t[0, 2] = bad
        o, lse = fa.kv4_attention(q.cuda(), dev(cache), dev(t), dev(lens), scale=0.3)
        assert fa.get_status() == fa.FA_ERR_INDEX
        check(o[1:], lse[1:], tuple(w[1:] for w in want), "bf16")
        keep = [j for j in range(100) if j // 16 != 2]
        k, v = ref.slot_values(cache, table[0][np.array(keep) // 16].astype(np.int64) * 16 + np.array(keep) % 16, 64)
        for h in range(4):
            s = k[:, h // 2] @ to_np64(q)[0, h] * 0.3
            w = np.exp(s - s.max())
            assert np.abs(to_np64(o)[0, h] - w @ v[:, h // 2] / w.sum()).max() < 0.01
    # a length beyond the table is cut to it
    long = np.array([table.shape[1] * 16 + 5, 50], np.int32)
    t = np.where(table < 0, 0, table)
    o, lse = fa.kv4_attention(q.cuda(), dev(cache), dev(t), dev(long), scale=0.3)
    assert fa.get_status() == fa.FA_ERR_INDEX
    check(o[1:], lse[1:], tuple(w[1:] for w in want), "bf16")
    # offsets of queries outside q are cut to it
    o, lse = fa.kv4_attention(q.cuda(), dev(cache), dev(table), dev(lens), cu_q=dev(np.array([-5, 1, 100], np.int32)), scale=0.3)
    assert fa.get_status() == fa.FA_OK
    check(o[1:], lse[1:], tuple(w[1:] for w in want), "bf16")


def test_rows_outside_every_request_stay(cuda_lib):
    q, cache, table, lens, cu = build([20, 30], [1, 2], 2, 1, 64, "f16", 16, 12)
    q = torch.cat([q, q, q])
    o = torch.full((9, 2, 64), 3.0, dtype=torch.float16, device="cuda")
    lse = torch.full((9, 2), 5.0, device="cuda")
    dev = lambda a: torch.from_numpy(a).cuda()
    fa.kv4_attention(q.cuda(), dev(cache), dev(table), dev(lens), cu_q=dev(cu), max_q_len=2, out=o, lse=lse)
    assert bool((o[3:] == 3).all()) and bool((lse[3:] == 5).all()) and not bool((o[:3] == 3).any())


def test_strided_queries_results_tables_and_caches(cuda_lib):
    """Views: queries and results inside packed rows, a cache of one layer among several, a
    table with a row pitch."""
    q, cache, table, lens, cu = build([70, 300], [1, 1], 6, 3, 128, "bf16", 32, 13)
    want = ref.attention(to_np64(q), cache, table, lens, cu, 128 ** -0.5, 0, 128)
    packed = torch.zeros(2, 12, 128, dtype=torch.bfloat16, device="cuda")
    packed[:, 3:9] = q.cuda()
    layers = torch.zeros((cache.shape[0], 3) + cache.shape[1:], dtype=torch.uint8, device="cuda")
    layers[:, 1] = torch.from_numpy(cache).cuda()
    wide = torch.full((2, table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + table.shape[1]] = torch.from_numpy(table).cuda()
    outp = torch.full((2, 12, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.kv4_attention(packed[:, 3:9], layers[:, 1], wide[:, 2:2 + table.shape[1]], torch.from_numpy(lens).cuda(),
                              out=outp[:, 3:9])
    check(o, lse, want, "bf16")
    assert bool((outp[:, :3] == 9).all()) and bool((outp[:, 9:] == 9).all())


def test_a_cache_beyond_32_bit_offsets(cuda_lib):
    """Pages past 2^32 bytes into the cache are written and read where they are."""
    H, d, page = 8, 128, 64
    pages = (2 ** 32 + 2 ** 28) // (H * (page // 16) * 2560)
    cache = torch.zeros(pages, H, page // 16, 2560, dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(4)
    T = 100
    k, v = (torch.randn(T, H, d, generator=g).bfloat16().cuda() for _ in range(2))
    ids = [pages - 1, 3]
    slots = torch.tensor([ids[t // page] * page + t % page for t in range(T)], dtype=torch.int32, device="cuda")
    fa.kv4_append(k, v, slots, cache)
    small = torch.stack([cache[i] for i in ids]).cpu().numpy()
    at = np.arange(T)
    gk, gv = fa.kv4_gather(cache, slots, d, dtype=torch.float32)
    wk, wv = ref.slot_values(small, at, d)
    assert np.array_equal(to_np64(gk), wk) and np.array_equal(to_np64(gv), wv)
    c, s, b = ref.quantise(k.float().cpu().numpy())
    assert np.array_equal(wk, ref.values(c, s, b))
    q = torch.randn(1, H, d, generator=g).bfloat16()
    lens = np.array([T], np.int32)
    want = ref.attention(to_np64(q), small, np.array([[0, 1]], np.int32), lens, np.array([0, 1]), d ** -0.5, 0, d)
    o, lse = fa.kv4_attention(q.cuda(), cache, torch.tensor([ids], dtype=torch.int32, device="cuda"),
                              torch.from_numpy(lens).cuda())
    check(o, lse, want, "bf16")


@pytest.mark.parametrize("wide", [False, True])
def test_streams_graphs_and_shared_workspaces(cuda_lib, wide):
    """Two attentions at once on two streams, each with its own workspace; two captured
    graphs that share one workspace, replayed in turn; results equal to plain calls'."""
    dev = lambda a: torch.from_numpy(a).cuda()
    sets = []
    for seed, kv in ((20, [3000, 40]), (21, [5, 1800])):
        q, cache, table, lens, cu = build(kv, [1, 1], 8, 2, 128, "bf16", 64, seed)
        args = (q.cuda(), dev(cache), dev(widened(table) if wide else table), dev(lens))
        sets.append((args, fa.kv4_attention(*args)))
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(10):
        for i, (args, _) in enumerate(sets):
            got[i] = fa.kv4_attention(*args, stream=side[i])
    torch.cuda.synchronize()
    for g, (_, w) in zip(got, sets):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    ws = torch.full((16 << 20,), 255, dtype=torch.uint8, device="cuda")
    graphs = []
    for args, _ in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = fa.kv4_attention(*args, workspace=ws)
        graphs.append((graph, res))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (_, g), (_, w) in zip(graphs, sets):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    assert fa.get_status() == fa.FA_OK


# ---------------------------------------------------------------- block tables

@pytest.mark.parametrize("R,T,page,width,most,spare,ended,seed", [
    (1, 1, 16, 4, 40, 10, 0.0, 0), (5, 40, 16, 9, 100, 30, 0.3, 1), (64, 64, 64, 40, 2000, 500, 0.2, 2),
    (200, 5000, 16, 50, 300, 2000, 0.3, 3), (33, 700, 32, 12, 200, 3, 0.1, 4),   # too few pages
    (40, 100, 16, 20, 250, 400, 0.0, 5),                                         # tokens past T
    (20, 300, 16, 10, 150, 100, 0.2, 6),                                         # tables that are full
    (8, 20000, 7, 3000, 100, 9000, 0.0, 7), (1500, 3000, 16, 8, 100, 1500, 0.5, 8), (8192, 9000, 16, 3, 30, 9000, 0.3, 9),
    (3, 0, 16, 4, 40, 10, 0.7, 10), (10, 50, 16, 12, 100, 0, 1.0, 11),
    (1, 300000, 16, 20000, 100, 20000, 0.0, 12), (300, 300000, 64, 40, 1500, 9000, 0.4, 13),  # many CTAs
])
def test_plan(cuda_lib, R, T, page, width, most, spare, ended, seed):
    rng = np.random.default_rng(seed)
    seq = rng.integers(0, min(most, width * page) + 1, R)
    new = rng.integers(0, max(1, 2 * T // R) + 2, R)
    new[rng.random(R) < ended] = -1
    have = -(-seq // page)
    pages = int(have.sum()) + spare
    pages = max(pages, 1)
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((R, width), -1, np.int32)
    at = 0
    for r in range(R):
        table[r, :have[r]] = order[at:at + have[r]]
        at += have[r]
    stack = np.concatenate([order[at:], order[:at]])
    count = pages - at
    want = ref.plan(seq.tolist(), new.tolist(), table.tolist(), stack.tolist(), count, page, T)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()
    for alias in (False, True):
        wide = torch.full((R, width + 3), -7, dtype=torch.int32, device="cuda")
        wide[:, :width] = dev(table)
        t, s, c, sl = wide[:, :width], dev(stack), dev(np.array([count, 0, 0])), dev(seq)
        raws, outs = zip(*(guarded((max(n, 1),), torch.int32) for n in (R, R + 1, T, T, 3)))
        out = dict(zip(("kv_lens", "cu_q", "positions", "slots", "counts"), (o[:n] for o, n in zip(outs, (R, R + 1, T, T, 3)))))
        if alias:
            out["kv_lens"], out["counts"] = sl, c
        fa.paged_plan(sl, dev(new), t, s, c, page, T, out=out)
        got = [out[n].cpu().tolist() for n in ("kv_lens", "cu_q", "positions", "slots", "counts")]
        for name, g, w in zip(("kv_lens", "cu_q", "positions", "slots", "counts"), got, want):
            assert g == w, name
        assert t.cpu().tolist() == want[5]
        assert s.cpu().tolist() == want[6]
        assert bool((wide[:, width:] == -7).all()) and all(guards_intact(r) for r in raws)
    got = fa.paged_plan(dev(seq), dev(new), dev(table), dev(stack), dev(np.array([count])), page, T)
    assert [got[n].cpu().tolist() for n in ("kv_lens", "cu_q", "positions", "slots", "counts")] == list(want[:5])


# ---------------------------------------------------------------- together

def test_a_training_step(cuda_lib):
    """Projection -> norm and rotation -> attention -> gradients, against the same chain
    in 64 bits (torch autograd).  The chain rounds q and k to bf16 (2^-8 each, so scores to
    about 2^-7 of themselves) and so do its gradients; relative 2-norm errors stay within
    the attention's own 2e-2 gradient bound plus two such roundings."""
    B, N, H, d = 1, 200, 3, 64
    g = torch.Generator().manual_seed(2)
    x = torch.randn(B, N, 3 * H, d, generator=g).bfloat16().cuda()
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2))
    do = torch.randn(B, H, N, d, generator=g).bfloat16().cuda()
    freqs = fa.rope_freqs(d)
    q, k = fa.qk_norm_rope(x[:, :, :H], x[:, :, H:2 * H], wq, wk, freqs)
    v = x[:, :, 2 * H:].transpose(1, 2).contiguous()
    o, lse = fa.attention_fwd(q, k, v, causal=True)
    dq, dk, dv = fa.attention_bwd(q, k, v, o, do, lse, causal=True)
    dx = torch.zeros_like(x)
    _, _, dwq, dwk = fa.qk_norm_rope_bwd(x[:, :, :H], x[:, :, H:2 * H], dq, dk, wq, wk, freqs, dq=dx[:, :, :H],
                                         dk=dx[:, :, H:2 * H])
    X = x.double().cpu().requires_grad_()
    W = [w.double().cpu().requires_grad_() for w in (wq, wk)]
    pos = torch.arange(N).double()[:, None, None]
    ang = pos * 10000.0 ** (-2 * torch.arange(d // 2).double() / d)
    def turn(n):
        a, b = n[..., :d // 2], n[..., d // 2:]
        return torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1).transpose(1, 2)
    Q, K = (turn(t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w) for t, w in
            zip((X[:, :, :H], X[:, :, H:2 * H]), W))
    S = Q @ K.transpose(-1, -2) / math.sqrt(d)
    S = S.masked_fill(~torch.ones(N, N, dtype=torch.bool).tril(), -math.inf)
    (torch.softmax(S, -1) @ X[:, :, 2 * H:].transpose(1, 2) * do.double().cpu()).sum().backward()
    for got, want in ((dx[:, :, :2 * H], X.grad[:, :, :2 * H]), (dwq, W[0].grad), (dwk, W[1].grad)):
        err = float((got.double().cpu() - want).norm() / want.norm())
        assert err <= 2e-2 + 2 * 2.0 ** -7


def test_serving_steps_with_a_graph(cuda_lib):
    """A prompt and then single tokens through plan, norm and rotation, append and
    attention, the single tokens by a captured graph; each step against attention in 64
    bits over the values the cache holds, and the cache against the quantised keys."""
    R, Hq, Hk, d, page, width, pages = 3, 8, 2, 64, 16, 8, 20
    g = torch.Generator().manual_seed(3)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2))
    freqs = fa.rope_freqs(d)
    i32 = lambda *a: torch.tensor(*a, dtype=torch.int32, device="cuda")
    seq, table = i32([0, 0, 0]), torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    stack, counts = torch.randperm(pages, generator=g).to(torch.int32).cuda(), i32([pages, 0, 0])
    cache = fa.kv4_cache(pages, Hk, d, page)

    def step(x, new, T, max_q):
        out = dict(kv_lens=seq, cu_q=cu, positions=pos[:T], slots=slots[:T], counts=counts)
        fa.paged_plan(seq, new, table, stack, counts, page, T, out=out)
        q, k = fa.qk_norm_rope(x[None, :, :Hq], x[None, :, Hq:Hq + Hk], wq, wk, freqs, positions=pos[None, :T], heads_first=False)
        fa.kv4_append(k[0], x[:, Hq + Hk:], slots[:T], cache)
        return q[0], *fa.kv4_attention(q[0], cache, table, seq, cu_q=cu, max_q_len=max_q)

    cu = torch.zeros(R + 1, dtype=torch.int32, device="cuda")
    pos, slots = (torch.zeros(64, dtype=torch.int32, device="cuda") for _ in range(2))

    def verify(q, o, lse, n_tok):
        c = cu.cpu().numpy()
        want = ref.attention(to_np64(q)[:n_tok], cache.cpu().numpy(), table.cpu().numpy(), seq.cpu().numpy(), c, d ** -0.5, 0, d)
        check(o[:n_tok], lse[:n_tok], want, "bf16")
        assert fa.get_status() == fa.FA_OK

    x = torch.randn(64, Hq + 2 * Hk, d, generator=g).bfloat16().cuda()
    q, o, lse = step(x, i32([20, 1, 37]), 64, 37)
    assert seq.tolist() == [20, 1, 37]
    verify(q, o, lse, 58)
    kept = torch.cat([torch.arange(58)])
    gk, gv = fa.kv4_gather(cache, slots[:58].clone(), d, dtype=torch.float32)
    c, s, b = ref.quantise(x[:58, Hq + Hk:].float().cpu().numpy())
    assert np.array_equal(to_np64(gv), ref.values(c, s, b))
    # single tokens by a graph; request 1 ends before the second replay and its pages come back
    xs, new = torch.zeros(R, Hq + 2 * Hk, d, dtype=torch.bfloat16, device="cuda"), i32([1, 1, 1])
    state = [t.clone() for t in (seq, table, stack, counts, cache)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(xs, new, R, 1)
    for t, was in zip((seq, table, stack, counts, cache), state):
        t.copy_(was)
    for turn in range(20):
        xs.copy_(torch.randn(R, Hq + 2 * Hk, d, generator=g).bfloat16())
        new.copy_(i32([1, -1, 1] if turn == 1 else [1, 1, 1] if turn == 0 else [1, 0, 1]))
        graph.replay()
        verify(*held, int(cu[-1]))
    assert seq.tolist() == [40, 0, 57]
    assert int(counts[0]) == pages - 3 - 4


def test_plan_of_lengths_that_are_out_of_range(cuda_lib):
    """Negative lengths count as none; a length beyond the table is not served, and where it
    has ended only the table's pages go back."""
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    table = i32([[5, 6], [7, 8], [1, 2], [3, 4]])
    seq, new, stack, count = [-3, 33, 500, 2 ** 31 - 1], [2, 3, -1, 1000], [0, 9, 0, 0, 0, 0, 0, 0], 2
    want = ref.plan([0, 33, 500, 2 ** 31 - 1], new, table.tolist(), stack, count, 16, 8)
    t, s = table.clone(), i32(stack)
    got = fa.paged_plan(i32(seq), i32(new), t, s, i32([count]), 16, 8)
    assert got["kv_lens"].tolist() == want[0] and got["slots"].tolist() == want[3] and t.tolist() == want[5]
    assert s.tolist() == want[6] and got["counts"].tolist()[0] == want[4][0]


def test_results_lie_apart(cuda_lib):
    """New results never overlap, start at whole 16-byte vectors and keep their values when the
    others are written; a result above 1 MB has a block of its own."""
    R, T = 5, 300000
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = fa.paged_plan(torch.zeros(R, **i32), torch.full((R,), 7, **i32), torch.full((R, 4), -1, **i32),
                         torch.arange(40, **i32), torch.full((1,), 40, **i32), 16, T)
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in plan.values())
    assert all(a % 16 == 0 for a, _ in spans) and all(e <= b for (_, e), (b, _) in zip(spans, spans[1:]))
    blocks = {name: t.untyped_storage().data_ptr() for name, t in plan.items()}
    assert blocks["positions"] != blocks["slots"] != blocks["kv_lens"] == blocks["counts"]
    want = {name: t.clone() for name, t in plan.items()}
    for name in plan:
        plan[name].fill_(-9)
        for other in plan:
            if other != name:
                assert torch.equal(plan[other], want[other])
        plan[name].copy_(want[name])
    assert plan["kv_lens"].tolist() == [7] * R and plan["counts"].tolist() == [35, 35, 0]


def test_results_that_do_not_fit_the_memory(cuda_lib):
    """The allocator's own error, before anything is launched; the next call runs."""
    cache = fa.kv4_cache(4, 8, 64, 16)
    slots = torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda")
    torch.cuda.empty_cache()
    try:
        torch.cuda.set_per_process_memory_fraction(0.001)  # less than the 4 GB of results
        with pytest.raises(torch.OutOfMemoryError):
            fa.kv4_gather(cache, slots, 64, dtype=torch.float32)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    k, v = fa.kv4_gather(cache, slots[:5], 64)
    assert k.shape == (5, 8, 64) and float(k.abs().sum() + v.abs().sum()) == 0
