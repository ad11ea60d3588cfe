"""The range of packed attention's gradient: incoming gradients, weights and scores of any size.

Inputs are chosen so that the gradients have a closed form and every term of a sum has the same sign:
what one of them loses the sum loses too.  q and k are orthogonal, so that all m keys of a row weigh
1 / m; keys come in two halves, with values +-v and, in a channel that no query has, +-kappa:
     D = 0, dS = +-delta v d' / m  (d' channels),  dQ = scale delta v d' kappa,
     dK = +-scale (rows x G) delta v d' / m * (the queries' size),  dV = (rows x G) delta / m.
Bounds, with e = eps(type) / 2: P, dS and the result are rounded once each, LSE (log m, at most 2^-20 of
fp32 roundings) and the sums in fp32 (lengths times 2^-24, all terms of a sign) less than 2^-11 together
for the lengths here; so 4 e of the result in fp16, and half of its least number."""
import math

import pytest
import torch

import _packed_ref as ref
import exact_io_aware_26_gb300 as fa
from _parity import DTYPES

pytestmark = pytest.mark.gpu


def offsets(lengths, first=0):
    return torch.tensor([first] + list(lengths), dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


def halves(n, m, Hq, Hk, d, delta, v=1.0, kappa=512.0, size=512.0, wide=False):
    """(q, k, v, do) of one sequence and (dq, dk, dv) as scale times and without; wide: all channels of v
    and do, not one."""
    sign = torch.where(torch.arange(m) < m // 2, 1.0, -1.0)[:, None]
    q, k, V, do = torch.zeros(n, Hq, d), torch.zeros(m, Hk, d), torch.zeros(m, Hk, d), torch.zeros(n, Hq, d)
    at = slice(None) if wide else slice(0, 1)
    V[:, :, at], do[:, :, at] = v * sign[..., None], delta
    q[:, :, 2], k[:, :, 3] = size, kappa * sign
    ds = delta * v * (d if wide else 1) / m
    dq, dk, dv = torch.zeros(n, Hq, d, dtype=torch.float64), *(torch.zeros(m, Hk, d, dtype=torch.float64) for _ in (0, 1))
    dq[:, :, 3] = ds * m * kappa
    dk[:, :, 2] = sign.double() * (n * Hq // Hk) * ds * size
    dv[:, :, at] = (n * Hq // Hk) * delta / m
    return (q, k, V, do), (dq, dk, dv)


def run(sequences, dtype, scale=0.125, causal=False, pad=0, padding=0.0):
    """The gradients of the sequences, one behind the other, with `pad` rows of `padding` around them."""
    x = []
    for i in range(4):
        parts = [s[i] for s in sequences]
        edge = torch.full((pad, *parts[0].shape[1:]), padding)
        x.append(torch.cat([edge, *parts, edge]).to(DTYPES[dtype]).cuda())
    q, k, v, do = x
    cu_q, cu_k = (offsets([s[i].shape[0] for s in sequences], pad) for i in (0, 1))
    o, lse = fa.attention_fwd_packed(q, k, v, cu_q, cu_k, causal=causal, scale=scale)
    grads = fa.attention_bwd_packed(q, k, v, o, do, lse, cu_q, cu_k, causal=causal, scale=scale)
    assert fa.get_status() == fa.FA_OK
    return [g[pad:g.shape[0] - pad].double().cpu() for g in grads]


def check(grads, want, dtype, scale=0.125):
    e = torch.finfo(DTYPES[dtype]).eps / 2
    least = 2.0 ** -25 if dtype == "f16" else 0.0
    at_q = at_k = 0
    for w in want:
        n, m = w[0].shape[0], w[1].shape[0]
        rows, cols = slice(at_q, at_q + n), slice(at_k, at_k + m)
        for name, g, x in (("dq", grads[0][rows], w[0] * scale), ("dk", grads[1][cols], w[1] * scale), ("dv", grads[2][cols], w[2])):
            err = (g - x).abs() - 4 * e * x.abs() - least
            assert bool((err <= 0).all()), f"{name}: {((g - x).abs() / x.abs().clamp(min=1e-30)).max():.2e} of it"
        at_q, at_k = at_q + n, at_k + m


@pytest.mark.parametrize("d,Hq,Hk", [(64, 2, 1), (128, 3, 3), (128, 10, 2)])
@pytest.mark.parametrize("n,m,delta", [(70, 6000, 1e-4), (3, 16384, 2.0 ** -13), (200, 4096, 1e-3), (6000, 256, 2.0 ** -18), (130, 130, 2.0 ** -20)])
def test_small_incoming_gradients(cuda_lib, d, Hq, Hk, n, m, delta):
    """dS far below fp16's least number; 6000 rows over 256 keys: cut along the queries."""
    x, want = halves(n, m, Hq, Hk, d, float(torch.tensor(delta).half()))
    for dtype in ("f16", "bf16"):
        if dtype == "bf16":
            x, want = halves(n, m, Hq, Hk, d, float(torch.tensor(delta).bfloat16()))
        check(run([x], dtype), [want], dtype)


@pytest.mark.parametrize("m", [60000, 302291])
def test_many_keys(cuda_lib, m):
    """Weights of 1 / m, below fp16's normal numbers: what they make of dV."""
    x, want = halves(100, m - m % 2, 2, 1, 64, 256.0, v=2.0 ** -6)
    check(run([x], "f16"), [want], "f16")


@pytest.mark.parametrize("d,delta,v", [(64, 300.0, 200.0), (128, 1000.0, 1000.0)])
def test_large_incoming_gradients(cuda_lib, d, delta, v):
    """dS above fp16's largest number, and gradients within it."""
    x, want = halves(2, 8, 2, 2, d, delta, v, kappa=2.0 ** -12, size=2.0 ** -12, wide=True)
    check(run([x], "f16"), [want], "f16")


@pytest.mark.parametrize("d,Hq,Hk", [(64, 2, 1), (128, 2, 2)])
def test_sequences_of_different_size_in_one_call(cuda_lib, d, Hq, Hk):
    """Each sequence's gradients are as exact beside large neighbours as alone; rows outside hold
    infinities, and rows that see no key anything."""
    both = [halves(70, 3000, Hq, Hk, d, 2.0 ** -13), halves(40, 200, Hq, Hk, d, 30000.0, 1000.0, kappa=2.0 ** -14, size=2.0 ** -14),
            halves(1, 4096, Hq, Hk, d, 2.0 ** -20), halves(200, 30, Hq, Hk, d, 2.0 ** -16)]
    none = [torch.full((s, h, d), 60000.0) for s, h in ((9, Hq), (0, Hk), (0, Hk), (9, Hq))]
    grads = run([b[0] for b in both] + [none], "f16", pad=5, padding=float("inf"))
    check(grads, [b[1] for b in both] + [[torch.zeros(9, Hq, d), torch.zeros(0, Hk, d), torch.zeros(0, Hk, d)]], "f16")


def test_heads_of_different_size(cuda_lib):
    """Key heads whose incoming gradients differ by 2^20."""
    small, want = halves(64, 2048, 2, 1, 64, 2.0 ** -16)
    large, more = halves(64, 2048, 2, 1, 64, 512.0, 64.0, kappa=2.0 ** -9, size=2.0 ** -4)
    grads = run([[torch.cat([a, b], 1) for a, b in zip(small, large)]], "f16")
    check(grads, [[torch.cat([a, b], 1) for a, b in zip(want, more)]], "f16")


def test_what_is_not_finite_stays_in_its_sequence(cuda_lib):
    """NaN and infinities in a sequence's do, v or q leave the others' gradients as they are, bit for bit."""
    parts = [halves(50, 900, 2, 1, 64, 2.0 ** -14)[0] for _ in range(3)]
    clean = run(parts, "f16")
    for i, bad in ((3, math.inf), (2, math.inf), (0, math.nan), (3, math.nan)):
        dirty = [list(p) for p in parts]
        dirty[1][i] = dirty[1][i].clone()
        dirty[1][i][7, 0, 1] = bad
        grads = run(dirty, "f16")
        for g, c in zip(grads[1:], clean[1:]):
            assert torch.equal(g[:900], c[:900]) and torch.equal(g[1800:], c[1800:])
        assert not bool(grads[2][900:1800].isfinite().all()) or not bool(grads[1][900:1800].isfinite().all())


def test_rows_that_see_no_key_have_no_say(cuda_lib):
    """More queries than keys: the first rows see none, and their do of any size changes no bit."""
    (q, k, v, do), _ = halves(90, 60, 2, 1, 64, 2.0 ** -16, kappa=8.0, size=8.0)
    grads = []
    for size in (0.0, 2.0 ** -16, 60000.0):
        do[:30] = size
        grads.append(run([(q, k, v, do)], "f16", causal=True))
    for g in grads[1:]:
        assert bool((g[0][:30] == 0).all()) and all(torch.equal(a[30:] if i == 0 else a, b[30:] if i == 0 else b)
                                                    for i, (a, b) in enumerate(zip(g, grads[0])))


@pytest.mark.parametrize("dtype,a,b,scale", [("bf16", 160.0, 640.0, 1.0), ("f16", 1001.0, 999.0, 1.0), ("f16", 1001.0, 999.0, 0.3337),
                                             ("bf16", 2.0 ** 12, 2.0 ** 12 * 1.25, 0.7), ("bf16", 2.0 ** 20, 2.0 ** 20, 1.1)])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_any_size(cuda_lib, d, dtype, a, b, scale):
    """One key far above the others has all of a head's weight, however large the scores: its dV is the
    sum of the rows' do.  The other head of the key head has ordinary scores in the same tiles."""
    T, at = 300, 50
    g = torch.Generator().manual_seed(3)
    q, do = (torch.randn(T, 2, d, generator=g) for _ in (0, 1))
    k, v = (torch.randn(T, 1, d, generator=g) for _ in (0, 1))
    q[:, 0], q[:, 1, 0] = 0.0, 0.0
    q[:, 0, 0], k[:, 0, 0], k[at, 0, 0] = a, 0.0, b
    q[:, 1] *= (d ** -0.5 / scale)
    do[:at, 0] = 0.0
    q, k, v, do = (x.to(DTYPES[dtype]) for x in (q, k, v, do))
    o, lse = fa.attention_fwd_packed(q.cuda(), k.cuda(), v.cuda(), offsets([T]), scale=scale)
    dq, dk, dv = (x.double().cpu() for x in fa.attention_bwd_packed(q.cuda(), k.cuda(), v.cuda(), o, do.cuda(), lse, offsets([T]), scale=scale))
    assert fa.get_status() == fa.FA_OK
    o, lse = o.cpu(), lse.cpu()
    e, tiny = torch.finfo(DTYPES[dtype]).eps / 2, 2.0 ** -24 if dtype == "f16" else 0.0
    want, bounds = ref.backward(q[:, 1:], k, v, o[:, 1:], do[:, 1:], lse[:, 1:], [T], [T], True, scale, e, tiny)
    # the first head's part: P = 1 at one key, in fp32 sums of T terms
    more = do[at:, 0].double().sum(0)
    slack = do[at:, 0].double().abs().sum(0) * (T * 2.0 ** -23 + 2.0 ** -20)
    got, total = dv[at, 0], want[2][at, 0] + more
    bound = bounds[2][at, 0] + slack + e * more.abs()
    assert bool(((got - total).abs() <= bound).all()), f"dv: {((got - total).abs() / bound).max():.1f} of the bound"
    rest = [j for j in range(T) if j != at]
    assert bool(((dv[rest] - want[2][rest]).abs() <= bounds[2][rest]).all())
    assert bool(((dq[:, 1:] - want[0]).abs() <= bounds[0]).all())
    # the first head's dS is 0 but for fp32 roundings, and its queries are 0 in these channels
    assert bool(((dk[:, :, 1:] - want[1][:, :, 1:]).abs() <= bounds[1][:, :, 1:]).all())
    assert bool(dq.isfinite().all()) and bool(dk.isfinite().all())


def random_batch(new, keys, Hq, Hk, d, seed):
    g = torch.Generator().manual_seed(seed)
    q, do = (torch.randn(sum(new), Hq, d, generator=g).half().cuda() for _ in (0, 1))
    k, v = (torch.randn(sum(keys), Hk, d, generator=g).half().cuda() for _ in (0, 1))
    return q, k, v, do


@pytest.mark.parametrize("R,d,Hq,Hk", [(4, 64, 6, 2), (40, 128, 2, 2), (1100, 64, 2, 1)])
def test_neighbours_change_no_bit_in_fp16(cuda_lib, R, d, Hq, Hk):
    """A sequence's dk and dv are the same bits whatever the others hold, with and without a lane for each
    sequence, and with their offsets in shared memory or not."""
    rng = torch.Generator().manual_seed(R)
    new = torch.randint(0, 200 if R < 10 else 60 if R < 100 else 4, (R,), generator=rng).tolist()
    new[1], new[2] = 70, 33
    keys = [n + (5 if i % 3 else 0) for i, n in enumerate(new)]
    q, k, v, do = random_batch(new, keys, Hq, Hk, d, R)
    cu_q, cu_k = offsets(new), offsets(keys)

    def call():
        o, lse = fa.attention_fwd_packed(q, k, v, cu_q, cu_k)
        return fa.attention_bwd_packed(q, k, v, o, do, lse, cu_q, cu_k)

    want = [x.clone() for x in call()]
    at_q, at_k = slice(new[0], new[0] + 70), slice(keys[0], keys[0] + keys[1])
    v[at_k] *= 100
    do[at_q] *= 1000
    got = call()
    rest = [i for i in range(sum(keys)) if not at_k.start <= i < at_k.stop]
    assert torch.equal(got[1][rest], want[1][rest]) and torch.equal(got[2][rest], want[2][rest])
    rows = [i for i in range(sum(new)) if not at_q.start <= i < at_q.stop]
    # dq: a sum of at most 3 parts in any order, and a step of fp16 (as in test_graphs_in_fp16)
    w = want[0][rows].float().abs()
    close = (got[0][rows].float() - want[0][rows].float()).abs() <= 2.0 ** -10 * w + 2.0 ** -24 + 2.0 ** -14 * float(w.max())
    assert bool(close.all())
    assert fa.get_status() == fa.FA_OK


def test_graphs_in_fp16(cuda_lib):
    """A captured call takes the lengths and sizes that are there when it is replayed, and its workspace's
    contents do not matter."""
    new, other, keys = [64, 500, 3], [100, 400, 67], [2000, 500, 9]
    q, k, v, do = random_batch(new, keys, 8, 2, 64, 6)
    live, cu_k = offsets(new), offsets(keys)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    want = []
    for i, (c, size) in enumerate(((new, 1.0), (other, 1e-3), (new, 300.0))):
        w = fa.attention_fwd_packed(q, k, v, offsets(c), cu_k)
        want.append((c, size, w, fa.attention_bwd_packed(q, k, v, w[0], do * size, w[1], offsets(c), cu_k)))
    o, lse, grad = torch.empty_like(want[0][2][0]), torch.empty_like(want[0][2][1]), do.clone()
    o.copy_(want[0][2][0])
    lse.copy_(want[0][2][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.attention_bwd_packed(q, k, v, o, grad, lse, live, cu_k, workspace=ws)
    for c, size, w, g in want + want[:1]:
        live.copy_(offsets(c))
        o.copy_(w[0])
        lse.copy_(w[1])
        grad.copy_(do * size)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[1], g[1]) and torch.equal(got[2], g[2])
        # dq is a fp32 sum of up to 16 parts (2000 keys) in any order: off by 16 * 2^-24 of the parts' sum, with each part
        # at most 4 times the largest result 2^-14 of that; and rounded to fp16, a step of which is at most
        # 2^-10 of it, or 2^-24 below the normal numbers
        w = g[0].float().abs()
        close = (got[0].float() - g[0].float()).abs() <= 2.0 ** -10 * w + 2.0 ** -24 + 2.0 ** -14 * float(w.max())
        assert bool(close.all())
    assert fa.get_status() == fa.FA_OK


def test_wrong_offsets_and_empty_tensors_in_fp16(cuda_lib):
    q, k, v, do = random_batch([300], [300], 4, 2, 64, 8)
    good = offsets([100, 200])
    o, lse = fa.attention_fwd_packed(q, k, v, good)
    want = fa.attention_bwd_packed(q, k, v, o, do, lse, good)
    for bad in ([0, 100, 5000], [0, 100, 50], [0, 100, -7], [0, 100, 2 ** 31 - 1], [-2 ** 31, 100, 90]):
        grads = fa.attention_bwd_packed(q, k, v, o, do, lse, torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert fa.get_status() == fa.FA_ERR_INDEX
        assert torch.equal(grads[1][:100], want[1][:100]) and torch.equal(grads[2][:100], want[2][:100])
    z = lambda T, H: torch.zeros(T, H, 64, dtype=torch.half, device="cuda")
    none = torch.full((5, 4), -math.inf, device="cuda")
    dq, dk, dv = fa.attention_bwd_packed(q[:5], z(0, 2), z(0, 2), z(5, 4), do[:5], none, offsets([5]), offsets([0]))
    assert bool((dq == 0).all()) and dk.shape == (0, 2, 64)
    dq, dk, dv = fa.attention_bwd_packed(z(0, 4), k[:5], v[:5], z(0, 4), z(0, 4), none[:0], offsets([0]), offsets([5]))
    assert bool((dk == 0).all()) and bool((dv == 0).all()) and dq.shape == (0, 4, 64)
    assert fa.get_status() == fa.FA_OK
