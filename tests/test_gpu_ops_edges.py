"""Edges of the operators around the attention, and of what the status word says."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import _ops_ref as ref
import exact_io_aware_26_gb300 as fa
from _parity import check_fwd, to_np64
from test_gpu_ops_kv4 import build, check, widened

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kv,new", [([3], [8]), ([3, 40, 0, 100], [8, 45, 3, 2]), ([1, 2, 3], [40, 30, 20])])
def test_a_window_beyond_every_length_hides_nothing(cuda_lib, kv, new, wide):
    """Also where a request has more rows than tokens: the first rows' positions lie before
    token 0, and position - window before -2^31."""
    q, cache, table, lens, cu = build(kv, new, 2, 1, 64, "bf16", 16, 31)
    want = ref.attention(to_np64(q), cache, table, lens, cu, 0.3, 0, 64)
    for window in (2 ** 31 - 1, 2 ** 31 - 4, 2 ** 31 - 40, 2 ** 30, 101):
        o, lse = fa.kv4_attention(q.cuda(), dev(cache), dev(widened(table) if wide else table), dev(lens), cu_q=dev(cu),
                                  max_q_len=max(new), scale=0.3, window=window)
        check(o, lse, want, "bf16")
    assert fa.get_status() == fa.FA_OK


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,Hk,d,dtype", [(2, 1, 64, "bf16"), (8, 2, 128, "f16"), (7, 1, 128, "bf16")])
@pytest.mark.parametrize("side,tok,group,window", [
    (1, 5, 0, 0), (1, 5, 1, 0),       # a value in a unit that every row sees
    (1, 197, 0, 0), (1, 198, 1, 0),   # in one that some rows see a part of
    (1, 160, 1, 0), (1, 199, 0, 0),
    (1, 134, 1, 64), (1, 140, 0, 64), (1, 100, 0, 64),  # the window's end; behind it
    (0, 5, 0, 0), (0, 198, 1, 0), (0, 134, 0, 64),      # a key
])
def test_a_nan_reaches_what_the_formula_says(cuda_lib, side, tok, group, window, Hq, Hk, d, dtype, wide):
    """A NaN value makes its 32 channels NaN for the rows that see it, and nothing else; a NaN
    key the rows' every channel and LSE: whatever the tile's height, the other rows in it and
    the place of the token in its unit."""
    kv, new = [200, 50], [4, 2]
    q, cache, table, lens, cu = build(kv, new, Hq, Hk, d, dtype, 16, 32)
    clean = ref.attention(to_np64(q), cache, table, lens, cu, 0.3, window, d)
    at = side * cache.shape[3] // 2 + 8 * d + tok % 16 * (d // 8) + 4 * group
    cache[table[0, tok // 16], Hk - 1, 0, at:at + 4] = 0x7E  # pages of one block
    with np.errstate(invalid="ignore"):
        dirty = ref.attention(to_np64(q), cache, table, lens, cu, 0.3, window, d)
    for hint in (1, 4, 40):
        o, lse = fa.kv4_attention(q.cuda(), dev(cache), dev(widened(table) if wide else table), dev(lens), cu_q=dev(cu),
                                  max_q_len=hint, scale=0.3, window=window)
        assert np.array_equal(np.isnan(to_np64(o)), np.isnan(dirty[0]))
        assert np.array_equal(np.isnan(to_np64(lse)), np.isnan(dirty[1]))
        zero = lambda x, like: np.where(np.isnan(like), 0, x)
        want = (zero(clean[0], dirty[0]), zero(clean[1], dirty[1]), zero(clean[2], dirty[0]), zero(clean[3], dirty[1]))
        check(torch.where(o.isnan(), 0, o), torch.where(lse.isnan(), 0, lse), want, dtype)
    assert fa.get_status() == fa.FA_OK


def test_plans_of_different_sizes_from_several_host_threads(cuda_lib):
    """The C entry from threads that do not hold a common lock, with requests for more than
    the shared memory that every kernel may have, and for all of it."""
    lib, failed = fa.load(), []

    def work(R, turns):
        i32 = dict(dtype=torch.int32, device="cuda")
        seq, new, table = torch.zeros(R, **i32), torch.ones(R, **i32), torch.full((R, 2), -1, **i32)
        free, count = torch.arange(R, **i32), torch.full((3,), R, **i32)
        outs = [torch.empty(n, **i32) for n in (R, R + 1, R, R, 3)]
        p = fa.FaPlanParams(R, R, 16, R, 2, 2)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        ptrs = [t.data_ptr() for t in (seq, new, table, free, count, *outs)]
        for _ in range(turns):
            status = lib.fa_paged_plan(ctypes.byref(p), *ptrs, stream.cuda_stream)
            if status != fa.FA_OK:
                failed.append((R, status, lib.fa_last_error()))
                break
        stream.synchronize()

    threads = [threading.Thread(target=work, args=a) for a in ((8192, 3000), (2500, 3000), (4000, 3000))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert fa.get_status() == fa.FA_OK


def test_numbers_beyond_32_bits_are_refused(cuda_lib):
    q, cache, table, lens, cu = build([40], [1], 2, 1, 64, "bf16", 16, 33)
    args = (q.cuda(), dev(cache), dev(table), dev(lens))
    with pytest.raises(ValueError):
        fa.kv4_attention(*args, window=2 ** 32 + 1)
    with pytest.raises(ValueError):
        fa.kv4_attention(*args, max_q_len=2 ** 32 + 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = (torch.zeros(1, **i32), torch.ones(1, **i32), torch.full((1, 4), -1, **i32), torch.arange(4, **i32), torch.full((1,), 4, **i32))
    with pytest.raises(ValueError):
        fa.paged_plan(*plan, page_size=2 ** 32 + 16, T=4)
    with pytest.raises(ValueError):
        fa.paged_plan(*plan, page_size=16, T=2 ** 32 + 4)
    assert fa.paged_plan(*plan, page_size=16, T=4)["counts"].tolist() == [3, 1, 0]


def test_a_graph_waits_and_reports_after_another_launch_gave_up(cuda_lib):
    """A launch that is replayed after the status of a later launch's failure was read neither
    gives up at once nor does it keep silent about a wait that runs out."""
    assert fa.get_status() == fa.FA_OK
    old = fa.set_wait_limit_ns(20_000_000)
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fa.selftest_timeout()  # an earlier launch than the next one
        fa.selftest_timeout()
        assert fa.get_status() == fa.FA_ERR_TIMEOUT
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        graph.replay()
        end.record()
        assert fa.get_status() == fa.FA_ERR_TIMEOUT
        assert start.elapsed_time(end) > 15  # its own limit of 20 ms
        assert fa.get_status() == fa.FA_OK
    finally:
        fa.set_wait_limit_ns(old)


@pytest.mark.parametrize("N,H,d,page", [(150, 3, 64, 16), (77, 2, 128, 32)])
def test_cached_tokens_read_back_for_the_dense_attention(cuda_lib, N, H, d, page):
    """Append -> gather -> attention_fwd over a request's cached tokens: the result of
    kv4_attention on the same cache for all of its rows, both against 64 bits."""
    g = torch.Generator().manual_seed(N)
    x = torch.randn(N, 3 * H, d, generator=g).to(torch.float16).cuda()
    w = torch.ones(d, dtype=torch.float16, device="cuda")
    q, k = fa.qk_norm_rope(x[None, :, :H], x[None, :, H:2 * H], w, w, fa.rope_freqs(d), heads_first=False)
    pages = -(-N // page)
    cache = fa.kv4_cache(pages + 2, H, d, page)
    table = torch.randperm(pages + 2, generator=g)[:pages].to(torch.int32)
    slots = (table.long()[torch.arange(N) // page] * page + torch.arange(N) % page).to(torch.int32).cuda()
    fa.kv4_append(k[0], x[:, 2 * H:], slots, cache)
    k16, v16 = fa.kv4_gather(cache, slots, d, dtype=torch.float16, heads_first=True)
    dense, dense_lse = fa.attention_fwd(q.transpose(1, 2).contiguous(), k16[None], v16[None], causal=True)
    o, lse = fa.kv4_attention(q[0], cache, table[None].cuda(), torch.tensor([N], dtype=torch.int32, device="cuda"),
                              cu_q=torch.tensor([0, N], dtype=torch.int32, device="cuda"), max_q_len=N)
    want = ref.attention(to_np64(q[0]), cache.cpu().numpy(), table[None].numpy(), np.array([N]), np.array([0, N]), d ** -0.5, 0, d)
    check(o, lse, want, "f16")
    check_fwd(dense[0].transpose(0, 1), dense_lse[0].T, want[0], want[1], "f16")
    assert fa.get_status() == fa.FA_OK


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,Hk,d,dtype", [(2, 1, 64, "bf16"), (8, 2, 128, "f16"), (24, 1, 128, "bf16")])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 8, 2.0 ** 12, 2.0 ** 15, 2.0 ** 40, 2.0 ** 95])
def test_scores_whose_rounding_is_larger_than_one(cuda_lib, size, Hq, Hk, d, dtype, wide):
    """Scores from 2^4 to 2^123: fp32 keeps them to 2^-24 of themselves, whole powers of the
    weights.  Where one token leads by more than what d fp32 roundings of the scores' terms
    make of two scores, its value is the result: within half a step of the type and the leader's
    weight, in fp16 and at most 2^8 of another, and LSE its score to the same accuracy."""
    if dtype == "f16" and size > 2.0 ** 8:
        pytest.skip("16 * 2^12 is beyond fp16's 65504")
    kv = [1, 2, 300, 900]
    q, cache, table, lens, cu = build(kv, [1] * 4, Hq, Hk, d, dtype, 16, 34, 16.0)
    q = (q.double() * size).to(q.dtype)
    scale = d ** -0.5 * 16
    o, lse = fa.kv4_attention(q.cuda(), dev(cache), dev(widened(table) if wide else table), dev(lens), scale=scale)
    o, lse = to_np64(o), to_np64(lse)
    e, leads = torch.finfo(q.dtype).eps / 2, 0
    for r, n in enumerate(kv):
        j = np.arange(n)
        k, v = ref.slot_values(cache, table[r].astype(np.int64)[j // 16] * 16 + j % 16, d)
        for h in range(Hq):
            s = k[:, h // (Hq // Hk)] @ to_np64(q)[r, h] * scale
            off = 2.0 ** -23 * d * (np.abs(k[:, h // (Hq // Hk)]) @ np.abs(to_np64(q)[r, h])).max() * scale
            best = int(s.argmax())
            assert np.isfinite(lse[r, h]) and np.isfinite(o[r, h]).all()
            assert abs(lse[r, h] - s.max()) <= off + np.log(n) + 2.0 ** -20 * abs(s.max()) + 2.0 ** -20
            if n == 1 or s[best] - np.delete(s, best).max() > 2 * off + 40:  # e^-40: below a bf16 step of any value here
                want = v[best, h // (Hq // Hk)]
                leads += 1
                assert np.all(np.abs(o[r, h] - want) <= (e + 2.0 ** -11 + 2.0 ** -20) * np.abs(want) + 2.0 ** -20)
    assert leads >= 2 * Hq
    assert fa.get_status() == fa.FA_OK


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kv,new,Hq,Hk,d,page,window", [
    ([300, 77, 32], [1, 1, 1], 4, 2, 64, 16, 40), ([500], [3], 8, 2, 128, 16, 1), ([4000, 130], [2, 5], 12, 2, 64, 32, 100),
    ([257], [1], 1, 1, 128, 16, 16),
])
def test_pages_behind_every_window_are_not_looked_at(cuda_lib, kv, new, Hq, Hk, d, page, window, wide):
    """A request whose pages behind the window have gone back to the pool, its table's entries
    with them: the rows' results are those of the whole table, and no bad page is recorded."""
    q, cache, table, lens, cu = build(kv, new, Hq, Hk, d, "bf16", page, 35)
    want = ref.attention(to_np64(q), cache, table, lens, cu, 0.3, window, d)
    for bad in (-1, cache.shape[0] + 5):
        t = table.copy()
        for r, (n, m) in enumerate(zip(kv, new)):
            t[r, :max(0, n - m - window + 1) // page] = bad
        assert (t != table).any()
        o, lse = fa.kv4_attention(q.cuda(), dev(cache), dev(widened(t) if wide else t), dev(lens), cu_q=dev(cu), max_q_len=max(new),
                                  scale=0.3, window=window)
        assert fa.get_status() == fa.FA_OK
        check(o, lse, want, "bf16")


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("pair", [0x7C007C00, 0xFC007C00, 0x7BFF7BFF])
def test_tokens_that_no_row_sees_may_hold_anything(cuda_lib, pair, wide):
    """Infinite pairs, of both signs, and pairs whose values overflow, behind the last token,
    behind the window and in the other pages."""
    q, cache, table, lens, cu = build([70, 300, 1, 47], [1, 3, 1, 2], 6, 2, 128, "bf16", 16, 36)
    want = ref.attention(to_np64(q), cache, table, lens, cu, 0.3, 33, 128)
    pairs = cache.reshape(-1, 2, cache.shape[3] // 2)[..., 8 * 128:].copy().view(np.uint32)
    pairs[pairs == 0x7E7E7E7E] = pair  # what build() leaves in tokens that are no request's
    cache.reshape(-1, 2, cache.shape[3] // 2)[..., 8 * 128:] = pairs.view(np.uint8)
    for r, (n, m) in enumerate(zip([70, 300, 1, 47], [1, 3, 1, 2])):
        for tok in range(max(0, n - m - 33 + 1)):  # behind the window of every row
            at = 8 * 128 + tok % 16 * 16
            for half in (0, cache.shape[3] // 2):
                cache[table[r, tok // 16], :, 0, half + at:half + at + 16] = np.full(4, pair, np.uint32).view(np.uint8)
    o, lse = fa.kv4_attention(q.cuda(), dev(cache), dev(widened(table) if wide else table), dev(lens), cu_q=dev(cu), max_q_len=3,
                              scale=0.3, window=33)
    check(o, lse, want, "bf16")
    assert fa.get_status() == fa.FA_OK
