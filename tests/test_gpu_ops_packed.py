"""Attention of packed sequences and its gradient against plain 64-bit implementations, with the
bounds that _packed_ref.py derives."""
import math

import pytest
import torch

import _packed_ref as ref
import exact_io_aware_26_gb300 as fa
from _parity import DTYPES, guarded, guards_intact

pytestmark = pytest.mark.gpu


def half_step(dtype):
    return torch.finfo(DTYPES[dtype]).eps / 2


def tiny(dtype):
    return 2.0 ** -24 if dtype == "f16" else 0.0


def offsets(lengths, first=0):
    at = [first]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def make(new, keys, Hq, Hk, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, do = (torch.randn(sum(new), Hq, d, generator=g).to(DTYPES[dtype]) for _ in (0, 1))
    kv = torch.randn(sum(keys), 2 * Hk, d, generator=g).to(DTYPES[dtype])
    return q, kv[:, :Hk], kv[:, Hk:], do


def check_fwd(o, lse, q, k, v, new, keys, causal, scale, dtype):
    wo, wl, bo, bl = ref.forward(q, k, v, new, keys, causal, scale, half_step(dtype), tiny(dtype))
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.equal(torch.isinf(lse), torch.isinf(wl)) and bool((o[torch.isinf(wl)] == 0).all())
    eo = (o - wo).abs() - bo
    assert bool((eo <= 0).all()), f"o: {(o - wo).abs().max():.3e}, past its bound by {eo.max():.3e}"
    el = ((lse - wl).abs() - bl)[~torch.isinf(wl)]
    assert bool((el <= 0).all()), f"lse past its bound by {el.max():.3e}"


def check_bwd(grads, q, k, v, o, do, lse, new, keys, causal, scale, dtype):
    want, bounds = ref.backward(q, k, v, o.cpu(), do, lse.cpu(), new, keys, causal, scale, half_step(dtype), tiny(dtype))
    for name, g, w, b in zip(("dq", "dk", "dv"), grads, want, bounds):
        e = (g.double().cpu() - w).abs() - b
        assert bool((e <= 0).all()), f"{name}: {(g.double().cpu() - w).abs().max():.3e}, past its bound by {e.max():.3e}"


CASES = [
    # new, keys (None: the same), Hq, Hk, d, dtype, causal
    ([1], None, 1, 1, 64, "bf16", True),
    ([1, 2, 0, 3], None, 2, 1, 128, "f16", True),
    ([127, 128, 129], None, 2, 2, 64, "f16", True),
    ([127, 128, 129], None, 2, 2, 128, "bf16", False),
    ([300, 1, 0, 77], [300, 1, 3, 77], 4, 2, 64, "bf16", True),
    ([31, 32, 33, 64], None, 8, 2, 128, "bf16", True),     # 32 tokens a tile
    ([17, 50], None, 40, 1, 64, "f16", True),              # 40 heads to a key head: 3 tokens a tile
    ([5, 9], [200, 9], 128, 1, 128, "bf16", True),         # 128: one token a tile
    ([26, 100], [140, 300], 10, 2, 128, "f16", True),      # 25 tokens of 5 heads: 125 rows
    ([64, 130], [900, 2000], 10, 2, 64, "f16", False),
    ([200, 50], [100, 0], 3, 3, 128, "bf16", True),        # rows that see no key, a sequence without keys
    ([0, 0], [130, 5], 2, 1, 64, "f16", True),             # keys without a query
    ([4, 1, 0, 2, 3], [1, 2, 0, 11, 5], 3, 3, 128, "f16", True),  # gradients below fp16's normal numbers
    ([1, 1, 4], [4000, 257, 1000], 8, 8, 64, "bf16", True),
    ([16], [6000], 8, 1, 128, "f16", True),                # cut along the keys
    ([700], None, 4, 1, 64, "bf16", True),                 # backward cut along the queries
]


@pytest.mark.parametrize("new,keys,Hq,Hk,d,dtype,causal", CASES)
def test_forward_and_gradient(cuda_lib, new, keys, Hq, Hk, d, dtype, causal):
    keys = keys or new
    q, k, v, do = make(new, keys, Hq, Hk, d, dtype, seed=sum(new) + d)
    scale = 1 / math.sqrt(d)
    dev = [x.cuda() for x in (q, k, v, do)]
    cu_q, cu_k = offsets(new), offsets(keys)
    raw_o, o = guarded(q.shape, q.dtype)
    raw_l, lse = guarded(q.shape[:2], torch.float32)
    got = fa.attention_fwd_packed(*dev[:3], cu_q, cu_k, causal=causal, out=o, lse=lse)
    assert got[0] is o and got[1] is lse
    assert fa.get_status() == fa.FA_OK and guards_intact(raw_o) and guards_intact(raw_l)
    check_fwd(o, lse, q, k, v, new, keys, causal, scale, dtype)
    raws, grads = zip(*(guarded(x.shape, x.dtype) for x in (q, k, v)))
    fa.attention_bwd_packed(*dev[:3], o, dev[3], lse, cu_q, cu_k, causal=causal, dq=grads[0], dk=grads[1], dv=grads[2])
    assert fa.get_status() == fa.FA_OK and all(map(guards_intact, raws))
    check_bwd(grads, q, k, v, o, do, lse, new, keys, causal, scale, dtype)


@pytest.mark.parametrize("seed", range(6))
def test_drawn_sizes(cuda_lib, seed):
    rng = torch.Generator().manual_seed(100 + seed)
    draw = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=rng))
    d, dtype, Hk = (64, 128)[draw(0, 1)], ("bf16", "f16")[draw(0, 1)], draw(1, 3)
    Hq, causal, R = Hk * (1, 2, 3, 5, 8)[draw(0, 4)], draw(0, 4) > 0, draw(1, 8)
    new = [draw(0, (5, 60, 400)[draw(0, 2)]) for _ in range(R)]
    keys = [max(0, n + draw(-20, (5, 700)[draw(0, 1)])) for n in new]
    new[0], keys[0] = new[0] + 1, keys[0] + 1
    scale = 0.3 / math.sqrt(d)
    q, k, v, do = make(new, keys, Hq, Hk, d, dtype, seed)
    dev = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.attention_fwd_packed(*dev[:3], offsets(new), offsets(keys), causal=causal, scale=scale)
    check_fwd(o, lse, q, k, v, new, keys, causal, scale, dtype)
    grads = fa.attention_bwd_packed(*dev[:3], o, dev[3], lse, offsets(new), offsets(keys), causal=causal, scale=scale)
    check_bwd(grads, q, k, v, o, do, lse, new, keys, causal, scale, dtype)
    assert fa.get_status() == fa.FA_OK


def test_sequences_of_one_length_are_the_batched_attention(cuda_lib):
    """Beside attention_fwd and attention_bwd, on the same data in the other layout."""
    B, H, N, d = 3, 4, 333, 64
    g = torch.Generator().manual_seed(5)
    q, k, v, do = (torch.randn(B, H, N, d, generator=g).bfloat16().cuda() for _ in range(4))
    o, lse = fa.attention_fwd(q, k, v, causal=True)
    want = fa.attention_bwd(q, k, v, o, do, lse, causal=True)
    flat = lambda x: x.transpose(1, 2).reshape(B * N, H, -1)
    cu = offsets([N] * B)
    po, pl = fa.attention_fwd_packed(flat(q), flat(k), flat(v), cu)
    e = half_step("bf16")
    assert bool(((po - flat(o)).abs() <= 4 * e * flat(o).abs() + 2 * e).all())  # weights and results rounded on both sides
    assert bool(((pl - flat(lse[..., None])[..., 0]).abs() <= 1e-4).all())
    got = fa.attention_bwd_packed(flat(q), flat(k), flat(v), flat(o).contiguous(), flat(do), flat(lse[..., None])[..., 0].contiguous(), cu)
    for a, b in zip(got, want):
        assert float((a - flat(b)).float().norm() / flat(b).float().norm()) < 2 * e


@pytest.mark.parametrize("d,Hq,Hk", [(64, 4, 2), (128, 10, 2)])
def test_rows_outside_and_what_they_hold(cuda_lib, d, Hq, Hk):
    """NaN and infinities before the first sequence, behind the last one and in the neighbours of a
    sequence reach nothing of it; rows in no sequence are not written."""
    new, keys, pad_q, pad_k = [70, 40, 150], [70, 300, 150], 9, 13
    q, k, v, do = make(new, keys, Hq, Hk, d, "bf16", 3)
    scale = 1 / math.sqrt(d)
    middle_q, middle_k = slice(pad_q + 70, pad_q + 110), slice(pad_k + 70, pad_k + 370)
    dirty = []
    for x, pad, middle in ((q, pad_q, middle_q), (k, pad_k, middle_k), (v, pad_k, middle_k), (do, pad_q, middle_q)):
        y = torch.full((x.shape[0] + 2 * pad, *x.shape[1:]), float("nan"), dtype=x.dtype)
        y[pad:-pad] = x
        y[0] = float("inf")
        y[-1] = -float("inf")
        y[middle][::2] = float("nan")  # the middle sequence is lost
        y[middle][1::4] = float("inf")
        dirty.append(y.cuda())
    cu_q, cu_k = offsets(new, pad_q), offsets(keys, pad_k)
    o = torch.full(dirty[0].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(o.shape[:2], 7.0, device="cuda")
    fa.attention_fwd_packed(*dirty[:3], cu_q, cu_k, out=o, lse=lse)
    for x in (o, lse):
        assert bool((x[:pad_q] == 7).all()) and bool((x[-pad_q:] == 7).all())
    wo, wl, bo, bl = ref.forward(q, k, v, new, keys, True, scale, half_step("bf16"), 0.0)
    own_q = torch.cat([torch.arange(70), torch.arange(110, 260)])
    own_k = torch.cat([torch.arange(70), torch.arange(370, 520)])
    assert bool(((o.double().cpu()[own_q + pad_q] - wo[own_q]).abs() <= bo[own_q]).all())
    assert bool(((lse.double().cpu()[own_q + pad_q] - wl[own_q]).abs() <= bl[own_q]).all())
    assert bool(o[middle_q].isnan().any(-1).all())
    grads = [torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in dirty[:3]]
    fa.attention_bwd_packed(*dirty[:3], o, dirty[3], lse, cu_q, cu_k, dq=grads[0], dk=grads[1], dv=grads[2])
    assert fa.get_status() == fa.FA_OK
    clean_o = torch.where(o[pad_q:-pad_q].isfinite(), o[pad_q:-pad_q], 0.0)
    clean_l = torch.where(lse[pad_q:-pad_q].isfinite(), lse[pad_q:-pad_q], 0.0)
    want, bounds = ref.backward(q, k, v, clean_o.cpu(), do, clean_l.cpu(), new, keys, True, scale, half_step("bf16"), 0.0)
    for g, w, b, pad, own in zip(grads, want, bounds, (pad_q, pad_k, pad_k), (own_q, own_k, own_k)):
        assert bool((g[:pad] == 7).all()) and bool((g[-pad:] == 7).all())
        assert bool(((g.double().cpu()[own + pad] - w[own]).abs() <= b[own]).all())


@pytest.mark.parametrize("d,Hq,Hk,dtype,n,m", [(64, 2, 1, "f16", 200, 200), (128, 4, 2, "bf16", 200, 333), (128, 8, 1, "f16", 9, 5000)])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(cuda_lib, d, Hq, Hk, dtype, n, m):
    q, k, v, _ = make([n], [m], Hq, Hk, d, dtype, 11)
    at = m - 5 if n < 100 else m - n + 100
    clean_v, clean_k = v.clone(), k.clone()
    v, k = v.clone(), k.clone()
    v[at, 0, 3], v[at, 0, 5], v[at + 1, 0, d - 1] = float("nan"), float("inf"), -float("inf")
    first = at - (m - n)  # the first row that sees the token
    wo, wl, bo, bl = ref.forward(q, clean_k, clean_v, [n], [m], True, d ** -0.5, half_step(dtype), tiny(dtype))
    o, lse = (x.cpu() for x in fa.attention_fwd_packed(q.cuda(), k.cuda(), v.cuda(), offsets([n]), offsets([m])))
    G = Hq // Hk
    assert bool(((lse.double() - wl).abs() <= bl).all())
    hit = torch.zeros(o.shape, dtype=torch.bool)
    hit[first:, :G, 3] = hit[first:, :G, 5] = True
    hit[first + 1:, :G, d - 1] = True
    assert bool(o[first:, :G, 3].isnan().all()) and bool((o[first:, :G, 5] == math.inf).all())
    assert bool((o[first + 1:, :G, d - 1] == -math.inf).all())
    assert bool(((o.double() - wo).abs() <= bo)[~hit].all())
    k[at, 0, 7] = float("nan")
    o, lse = (x.cpu() for x in fa.attention_fwd_packed(q.cuda(), k.cuda(), clean_v.cuda(), offsets([n]), offsets([m])))
    assert bool(o[first:, :G].isnan().all()) and bool(lse[first:, :G].isnan().all())
    assert bool(((o.double() - wo).abs() <= bo)[:first].all()) and bool(((o.double() - wo).abs() <= bo)[:, G:].all())
    assert bool(((lse.double() - wl).abs() <= bl)[:first].all())


@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 24, 2.0 ** 40])
def test_scores_of_any_size(cuda_lib, size):
    """One key far above the others has all of the weight, however large the scores."""
    q = torch.zeros(140, 2, 64, dtype=torch.bfloat16)
    k, v = torch.zeros(140, 1, 64, dtype=torch.bfloat16), torch.randn(140, 1, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    q[:, :, 0], k[:, 0, 0] = size, 1.0
    k[50, 0, 0] = 2.0
    o, lse = fa.attention_fwd_packed(q.cuda(), k.cuda(), v.cuda(), offsets([140]), scale=1.0)
    o, lse = o.cpu(), lse.cpu()
    assert torch.equal(o[50:], v[50].expand(90, 2, 64)) and torch.equal(lse[50:], torch.full((90, 2), 2 * size))
    mean = v[:, 0].double().cumsum(0) / torch.arange(1, 141)[:, None]
    assert bool(((o[:50].double() - mean[:50, None]).abs() <= 2 ** -8 * mean[:50, None].abs() + 1e-5).all())


def test_offsets_that_are_wrong_stay_in_the_tensors(cuda_lib):
    """Offsets outside the tensors or not in order are recorded; the sequences that are right are
    computed."""
    q, k, v, do = make([300], [300], 4, 2, 64, "bf16", 8)
    dev = [x.cuda() for x in (q, k, v, do)]
    for bad in ([0, 100, 5000], [0, 100, 50], [0, 100, -7], [0, 100, 2 ** 31 - 1], [-2 ** 31, 100, 90]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        o, lse = fa.attention_fwd_packed(*dev[:3], cu)
        assert fa.get_status() == fa.FA_ERR_INDEX
        check_fwd(o[:100], lse[:100], q[:100], k[:100], v[:100], [100], [100], True, 0.125, "bf16")
        o, lse = fa.attention_fwd_packed(*dev[:3], offsets([100, 200]))
        grads = fa.attention_bwd_packed(*dev[:3], o, dev[3], lse, cu)
        assert fa.get_status() == fa.FA_ERR_INDEX
        check_bwd([g[:100] for g in grads], q[:100], k[:100], v[:100], o[:100], do[:100], lse[:100], [100], [100], True, 0.125, "bf16")


@pytest.mark.parametrize("R", [31, 32, 33])
@pytest.mark.parametrize("most", [512, 513])
def test_where_the_work_list_begins(cuda_lib, R, most):
    """Up to 32 sequences over up to 512 rows of keys go without a work list."""
    rng = torch.Generator().manual_seed(R)
    new = torch.randint(0, 4, (R,), generator=rng).tolist()
    keys = torch.randint(0, 9, (R,), generator=rng).tolist()
    new[-1], keys[-1] = 200, 0
    keys[-1] = most - sum(keys)
    q, k, v, do = make(new, keys, 6, 2, 64, "bf16", 14)
    for causal in (True, False):
        o, lse = fa.attention_fwd_packed(q.cuda(), k.cuda(), v.cuda(), offsets(new), offsets(keys), causal=causal)
        check_fwd(o, lse, q, k, v, new, keys, causal, 0.125, "bf16")
    # offsets that are wrong: behind the tensors, back again
    cu_q, cu_k = offsets(new), offsets(keys)
    cu_q[-1], cu_k[-1] = 2 ** 30, -3
    o, lse = fa.attention_fwd_packed(q.cuda(), k.cuda(), v.cuda(), cu_q, cu_k)
    assert fa.get_status() == fa.FA_ERR_INDEX
    a, b = sum(new[:-1]), sum(keys[:-1])
    check_fwd(o[:a], lse[:a], q[:a], k[:b], v[:b], new[:-1], keys[:-1], True, 0.125, "bf16")
    assert bool((o[a:] == 0).all()) and bool((lse[a:] == -math.inf).all())


@pytest.mark.parametrize("d,Hq,Hk,dtype", [(64, 3, 1, "bf16"), (128, 2, 2, "f16")])
def test_a_long_sequence(cuda_lib, d, Hq, Hk, dtype):
    """140,001 tokens: the rows and keys at its end, rows from all over it, and its first rows."""
    N, last = 140001, 40
    g = torch.Generator().manual_seed(15)
    q, do = (torch.randn(N, Hq, d, generator=g).to(DTYPES[dtype]) for _ in range(2))
    k, v = (torch.randn(N, Hk, d, generator=g).to(DTYPES[dtype]) for _ in range(2))
    scale, cu = d ** -0.5, offsets([N])
    o, lse = fa.attention_fwd_packed(q.cuda(), k.cuda(), v.cuda(), cu)
    grads = fa.attention_bwd_packed(q.cuda(), k.cuda(), v.cuda(), o, do.cuda(), lse, cu)
    assert fa.get_status() == fa.FA_OK
    o, lse, grads = o.cpu(), lse.cpu(), [x.cpu() for x in grads]
    for a, b in [(0, 50), (N - last, N)] + [(int(x), int(x) + 1) for x in torch.randint(0, N, (4,), generator=g)]:
        rows = [x[a:b] for x in (q, o, lse, do)]
        check_fwd(*rows[1:3], rows[0], k[:b], v[:b], [b - a], [b], True, scale, dtype)
        want, bounds = ref.backward(rows[0], k[:b], v[:b], rows[1], rows[3], rows[2], [b - a], [b], True, scale,
                                    half_step(dtype), tiny(dtype))
        assert bool(((grads[0][a:b].double() - want[0]).abs() <= bounds[0]).all())
        if b == N:  # only these rows see the last keys
            for i in (1, 2):
                assert bool(((grads[i][a:].double() - want[i][a:]).abs() <= bounds[i][a:]).all())


def test_offsets_beyond_32_bits(cuda_lib):
    """Rows 2^26 elements apart: the results of the same rows next to each other."""
    new, step = [30, 13], 1 << 26
    T = sum(new)
    q, k, v, do = (x.cuda() for x in make(new, new, 4, 2, 128, "bf16", 16))
    cu = offsets(new)
    o, lse = fa.attention_fwd_packed(q, k, v, cu)
    want = fa.attention_bwd_packed(q, k, v, o, do, lse, cu)
    room = torch.empty((T - 1) * step + (1 << 16), dtype=torch.bfloat16, device="cuda")
    at = lambda i, H: room.as_strided((T, H, 128), (step, 128, 1), i << 10)
    far = [at(i, x.shape[1]).copy_(x) for i, x in enumerate((q, k, v, do))]
    fo, fl = fa.attention_fwd_packed(*far[:3], cu, out=at(4, 4))
    assert torch.equal(fo, o) and torch.equal(fl, lse)
    got = fa.attention_bwd_packed(*far[:3], fo, far[3], fl, cu, dq=at(5, 4), dk=at(6, 2), dv=at(7, 2))
    assert all(torch.equal(a, b) for a, b in zip(got, want))  # one key tile a row: dq, too, repeats
    assert fa.get_status() == fa.FA_OK


def test_layouts(cuda_lib):
    """Views of packed projections, heads before tokens, results inside wider rows."""
    new = [33, 90]
    g = torch.Generator().manual_seed(2)
    packed = torch.randn(123, 8 + 2 * 2, 128, generator=g).half().cuda()
    q, k, v = packed[:, :8], packed[:, 8:10], packed[:, 10:]
    do = torch.randn(123, 8, 128, generator=g).half().cuda()
    cu = offsets(new)
    o, lse = fa.attention_fwd_packed(q, k, v, cu)
    check_fwd(o, lse, q.cpu(), k.cpu(), v.cpu(), new, new, True, 128 ** -0.5, "f16")
    grads = fa.attention_bwd_packed(q, k, v, o, do, lse, cu)
    turned = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v, do)]
    assert turned[0].stride() == (128, 123 * 128, 1)
    wide = torch.full((123, 12, 128), 3.0, dtype=torch.half, device="cuda")
    fa.attention_fwd_packed(*turned[:3], cu, out=wide[:, 2:10])
    assert torch.equal(wide[:, 2:10], o) and bool((wide[:, :2] == 3).all()) and bool((wide[:, 10:] == 3).all())
    dpacked = torch.zeros_like(packed)
    fa.attention_bwd_packed(*turned[:3], turned[3], turned[3], lse, cu)  # other values of o: only its layout
    got = fa.attention_bwd_packed(*turned[:3], wide[:, 2:10], turned[3], lse, cu, dq=dpacked[:, :8], dk=dpacked[:, 8:10],
                                  dv=dpacked[:, 10:])
    assert torch.equal(got[1], grads[1]) and torch.equal(got[2], grads[2]) and torch.equal(dpacked[:, 8:10], grads[1])
    check_bwd(got, q.cpu(), k.cpu(), v.cpu(), o, do.cpu(), lse, new, new, True, 128 ** -0.5, "f16")
    # dq over its query
    over = q.clone()
    fa.attention_bwd_packed(over, k, v, o, do, lse, cu, dq=over)
    check_bwd([over, grads[1], grads[2]], q.cpu(), k.cpu(), v.cpu(), o, do.cpu(), lse, new, new, True, 128 ** -0.5, "f16")


def test_same_results_again_and_from_graphs(cuda_lib):
    """Forward, dk and dv repeat bit for bit; captured calls that share a workspace take the
    lengths that are there when they are replayed; two streams at once."""
    new, keys, other = [64, 500, 3], [2000, 500, 9], [100, 400, 67]
    q, k, v, do = (x.cuda() for x in make(new, keys, 8, 2, 64, "bf16", 6))
    cu_q, cu_k = offsets(new), offsets(keys)
    want = [fa.attention_fwd_packed(q, k, v, cu_q, cu_k)]
    want.append(fa.attention_fwd_packed(q, k, v, offsets(other), cu_k))
    grads = [fa.attention_bwd_packed(q, k, v, w[0], do, w[1], c, cu_k) for w, c in zip(want, (cu_q, offsets(other)))]
    for _ in range(3):
        o, lse = fa.attention_fwd_packed(q, k, v, cu_q, cu_k)
        again = fa.attention_bwd_packed(q, k, v, o, do, lse, cu_q, cu_k)
        assert torch.equal(o, want[0][0]) and torch.equal(lse, want[0][1])
        assert torch.equal(again[1], grads[0][1]) and torch.equal(again[2], grads[0][2])
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    live = cu_q.clone()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.attention_fwd_packed(q, k, v, live, cu_k, workspace=ws)
    with torch.cuda.graph(second):
        got = fa.attention_bwd_packed(q, k, v, o, do, lse, live, cu_k, workspace=ws)
    for i in (0, 1, 0):
        live.copy_((cu_q, offsets(other))[i])
        ws.fill_(255)
        graph.replay()
        second.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
        assert torch.equal(got[1], grads[i][1]) and torch.equal(got[2], grads[i][2])
    side = [torch.cuda.Stream() for _ in (0, 1)]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    both = [fa.attention_fwd_packed(q, k, v, c, cu_k, stream=s) for c, s in zip((cu_q, offsets(other)), side)]
    torch.cuda.synchronize()
    for b, w in zip(both, want):
        assert torch.equal(b[0], w[0]) and torch.equal(b[1], w[1])
    assert fa.get_status() == fa.FA_OK


@pytest.mark.parametrize("d,Hq,Hk,new,keys", [(128, 6, 2, [200, 1, 31], [200, 900, 3]), (64, 5, 1, [33, 20, 90], [33, 700, 90])])
def test_what_other_rows_hold_changes_no_bit(cuda_lib, d, Hq, Hk, new, keys):
    """Neighbours of any size, and what earlier calls left in the places of rows that are nobody's (with
    3 and 5 heads to a key head a tile has 126 and 125)."""
    q, k, v, do = (x.cuda() for x in make(new, keys, Hq, Hk, d, "bf16", 17))
    cu_q, cu_k = offsets(new), offsets(keys)

    def run():
        o, lse = fa.attention_fwd_packed(q, k, v, cu_q, cu_k)
        return (o, lse) + fa.attention_bwd_packed(q, k, v, o, do, lse, cu_q, cu_k)

    want = [x.clone() for x in run()]
    full = torch.rand(60000, 2, d, device="cuda").bfloat16()
    for size in (1e6, -1e12, 1e24, float("inf"), float("nan")):
        fa.attention_fwd_packed(full * size, full, full, offsets([200] * 300))  # all 128 rows of every CTA's tiles
        got = run()
        assert all(torch.equal(got[i], want[i]) for i in (0, 1, 3, 4))
    middle_q, middle_k = slice(new[0], new[0] + new[1]), slice(keys[0], keys[0] + keys[1])
    for x, at in ((q, middle_q), (do, middle_q), (k, middle_k), (v, middle_k)):
        x[at] *= 1e4
    got = run()
    rest_q = [i for i in range(sum(new)) if not middle_q.start <= i < middle_q.stop]
    rest_k = [i for i in range(sum(keys)) if not middle_k.start <= i < middle_k.stop]
    for i, rest in ((0, rest_q), (1, rest_q), (3, rest_k), (4, rest_k)):
        assert torch.equal(got[i][rest], want[i][rest])
    assert fa.get_status() == fa.FA_OK


def test_many_sequences(cuda_lib):
    """More sequences than the work list's kernel has threads, most of them short or empty."""
    rng = torch.Generator().manual_seed(9)
    new = torch.randint(0, 4, (2500,), generator=rng).tolist()
    new[1000] = 300
    q, k, v, do = make(new, new, 2, 1, 64, "f16", 10)
    dev = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.attention_fwd_packed(*dev[:3], offsets(new))
    check_fwd(o, lse, q, k, v, new, new, True, 0.125, "f16")
    grads = fa.attention_bwd_packed(*dev[:3], o, dev[3], lse, offsets(new))
    check_bwd(grads, q, k, v, o, do, lse, new, new, True, 0.125, "f16")


@pytest.mark.parametrize("R,most,Hq,Hk,d", [(40, 60, 96, 96, 64), (1500, 5, 4, 4, 64), (30, 200, 64, 64, 128)])
def test_many_units(cuda_lib, R, most, Hq, Hk, d):
    """So many tiles for each CTA that the list goes sequence by sequence; with sequences without
    queries or keys among them."""
    rng = torch.Generator().manual_seed(R)
    new = torch.randint(0, most + 1, (R,), generator=rng).tolist()
    keys = [n + int(torch.randint(0, 3, (1,), generator=rng)) if i % 7 else 0 for i, n in enumerate(new)]
    q, k, v, do = make(new, keys, Hq, Hk, d, "bf16", 12)
    dev = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.attention_fwd_packed(*dev[:3], offsets(new), offsets(keys))
    check_fwd(o, lse, q, k, v, new, keys, True, d ** -0.5, "bf16")
    grads = fa.attention_bwd_packed(*dev[:3], o, dev[3], lse, offsets(new), offsets(keys))
    check_bwd(grads, q, k, v, o, do, lse, new, keys, True, d ** -0.5, "bf16")
    assert fa.get_status() == fa.FA_OK


def test_empty_tensors(cuda_lib):
    z = lambda T, H: torch.zeros(T, H, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.attention_fwd_packed(z(0, 4), z(0, 2), z(0, 2), offsets([0]))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    o, lse = fa.attention_fwd_packed(z(5, 4), z(0, 2), z(0, 2), offsets([5]), offsets([0]))
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    dq, dk, dv = fa.attention_bwd_packed(z(5, 4), z(0, 2), z(0, 2), o, o, lse, offsets([5]), offsets([0]))
    assert bool((dq == 0).all()) and dk.shape == (0, 2, 64)
    dq, dk, dv = fa.attention_bwd_packed(z(0, 4), z(5, 2), z(5, 2), z(0, 4), z(0, 4), lse[:0], offsets([0]), offsets([5]))
    assert bool((dk == 0).all()) and bool((dv == 0).all()) and dq.shape == (0, 4, 64)
    assert fa.get_status() == fa.FA_OK


def test_refusals_of_the_binding(cuda_lib):
    q, k, v, do = (x.cuda() for x in make([8], [8], 4, 2, 64, "bf16"))
    cu = offsets([8])
    o, lse = fa.attention_fwd_packed(q, k, v, cu)
    other = torch.empty_like(k)
    for call, error in [
        (lambda: fa.attention_fwd_packed(q.float(), k, v, cu), TypeError),
        (lambda: fa.attention_fwd_packed(q, k.half(), v, cu), TypeError),
        (lambda: fa.attention_fwd_packed(q, k[:4], v[:4], cu), ValueError),
        (lambda: fa.attention_fwd_packed(q, k, v[:, :1], cu), ValueError),
        (lambda: fa.attention_fwd_packed(q, k, v, cu.long()), TypeError),
        (lambda: fa.attention_fwd_packed(q, k, v, cu[:1]), ValueError),
        (lambda: fa.attention_fwd_packed(q, k, v, cu, offsets([4, 4])), ValueError),
        (lambda: fa.attention_fwd_packed(q.cpu(), k, v, cu), ValueError),
        (lambda: fa.attention_fwd_packed(q, k, v, cu, lse=lse[:, :2]), ValueError),
        (lambda: fa.attention_fwd_packed(q[:, :3], k, v, cu), fa.FaError),
        (lambda: fa.attention_fwd_packed(q, k, v, cu, out=q), fa.FaError),
        (lambda: fa.attention_fwd_packed(k, k, v, cu, out=v), fa.FaError),
        (lambda: fa.attention_fwd_packed(q, k[:, :1].expand(8, 2, 64), v, cu), fa.FaError),
        (lambda: fa.attention_fwd_packed(q, k, v, cu, scale=-1.0), fa.FaError),
        (lambda: fa.attention_fwd_packed(q, k, v, cu, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")), fa.FaError),
        (lambda: fa.attention_bwd_packed(q, k, v, o, do, None, cu), ValueError),
        (lambda: fa.attention_bwd_packed(q, k, v, o, do[:4], lse, cu), ValueError),
        (lambda: fa.attention_bwd_packed(q, k, v, o, do, lse, cu, dk=k), fa.FaError),
        (lambda: fa.attention_bwd_packed(q, k, v, o, do, lse, cu, dk=other, dv=other), fa.FaError),
        (lambda: fa.attention_bwd_packed(q, k, v, o, do, lse, cu, dq=do.float()), TypeError),
    ]:
        with pytest.raises(error):
            call()
    o2, _ = fa.attention_fwd_packed(q, k, v, cu)
    assert torch.equal(o, o2)
