"""Norms and rotation of queries and keys, and their gradient, against 64-bit formulas.

Bounds (u = 2^-24, the fp32 rounding; e = eps(type) / 2, the rounding of the result):
  y:  the sum of squares of a lane's 16 values and its tree is off by at most 20 u, r by half
      of that and the 4 u of the reciprocal root; with the two products n is off by
      16 u |n|.  cos and sin: an angle off by pi 2^-25 for the phase and as much for its
      conversion, 2 ulp for the function: 8 u.  So |dy| <= e |y| + 32 u (|n_a| + |n_b|).
  dx: two such sums and their products: e |dx| + 128 u times the sizes of its terms.
  dw: rows are summed in chains of at most 128 on top of the terms' 24 u: 256 u sum |dz h|.
"""
import numpy as np
import pytest
import torch

import _ops_ref as ref
import exact_io_aware_26_gb300 as fa
from _parity import DTYPES, guarded, guards_intact, to_np64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(DTYPES[dtype]).eps / 2


def tiny(dtype):  # half a step of the least subnormal
    return torch.finfo(DTYPES[dtype]).smallest_normal * torch.finfo(DTYPES[dtype]).eps / 2


def make(B, N, Hq, Hk, d, dtype, seed, packed=True, w_f32=False, size=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, N, Hq + 2 * Hk, d, generator=g) * size).to(DTYPES[dtype]).cuda()
    q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    wt = torch.float32 if w_f32 else DTYPES[dtype]
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(wt).cuda() for _ in range(2))
    return q, k, wq, wk, g


def turns_of(freqs):
    return freqs.cpu().numpy().view(np.uint64)


def where(positions, B, N):
    if positions is None:
        return np.broadcast_to(np.arange(N), (B, N))
    return np.broadcast_to(positions.cpu().numpy().astype(np.int64), (B, N))


def partner_sum(n, rot, interleaved):
    pair, _ = ref._partners(n.shape[-1], rot, interleaved)
    out = np.abs(n).copy()
    for c in range(rot):
        a = [k for k in range(rot) if pair[k] == pair[c]]
        out[..., c] = np.abs(n[..., a[0]]) + np.abs(n[..., a[1]])
    return out


CASES = [  # B, N, Hq, Hk, d, dtype, rot, interleaved, heads_first, positions
    (1, 1, 1, 1, 64, "bf16", 64, False, True, None),
    (1, 1, 5, 1, 128, "f16", 128, False, False, "far"),
    (2, 33, 3, 3, 64, "bf16", 64, False, True, None),
    (1, 65, 12, 12, 64, "f32", 64, True, True, None),
    (3, 17, 8, 2, 128, "bf16", 128, True, False, "far"),
    (1, 40, 4, 1, 128, "f32", 64, False, True, "far"),
    (2, 31, 2, 2, 128, "f16", 48, False, False, "row"),
    (1, 9, 3, 1, 64, "bf16", 16, False, True, None),
    (1, 11, 2, 1, 64, "f32", 34, False, True, "far"),    # halves that are no whole chunks
    (1, 13, 3, 2, 128, "bf16", 126, False, False, None),
    (1, 7, 2, 1, 128, "f16", 30, True, True, "far"),
    (1, 5, 2, 1, 64, "bf16", 0, False, True, None),      # norms only
    (1, 8, 2, 1, 64, "f32", 2, False, False, "negative"),
    (1, 700, 12, 4, 64, "bf16", 64, False, True, None),  # several tiles and turns
    (2, 300, 40, 8, 128, "bf16", 128, False, True, "far"),
    (2, 40, 3, 1, 64, "bf16", 48, False, False, "row"),  # a rotated part of a 64-channel head
    (1, 1500, 20, 4, 64, "f32", 32, False, True, None),
    (1, 900, 12, 12, 128, "f32", 90, False, False, "far"),
    (2, 33, 3, 2, 64, "f32", 24, True, False, None),
    (2, 50, 2, 1, 128, "f32", 96, False, True, None),
]


def positions_of(kind, B, N, g):
    if kind is None:
        return None
    if kind == "row":
        return torch.randint(0, 5000, (N,), generator=g).to(torch.int32).cuda()
    lo, hi = (-(2 ** 31), 0) if kind == "negative" else (0, 2 ** 31)
    return torch.randint(lo, hi, (B, N), generator=g).to(torch.int32).cuda()


@pytest.mark.parametrize("B,N,Hq,Hk,d,dtype,rot,interleaved,heads_first,positions", CASES)
def test_forward(cuda_lib, B, N, Hq, Hk, d, dtype, rot, interleaved, heads_first, positions):
    q, k, wq, wk, g = make(B, N, Hq, Hk, d, dtype, 11 * N + d)
    pos = positions_of(positions, B, N, g)
    freqs = fa.rope_freqs(rot)
    shape = (lambda h: (B, h, N, d)) if heads_first else (lambda h: (B, N, h, d))
    raws, outs = zip(*(guarded(shape(h), DTYPES[dtype]) for h in (Hq, Hk)))
    fa.qk_norm_rope(q, k, wq, wk, freqs, positions=pos, eps=1e-5, interleaved=interleaved, heads_first=heads_first,
                    out=outs)
    for x, w, y, raw in ((q, wq, outs[0], raws[0]), (k, wk, outs[1], raws[1])):
        want, n = ref.norm_rope(to_np64(x), to_np64(w), where(pos, B, N), turns_of(freqs), np.float32(1e-5), interleaved)
        got = to_np64(y)
        got = got.transpose(0, 2, 1, 3) if heads_first else got
        bound = half_step(dtype) * np.abs(want) + 32 * U * partner_sum(n, rot, interleaved) + tiny(dtype)
        assert np.all(np.abs(got - want) <= bound), f"worst excess {(np.abs(got - want) / bound).max():.3f} of the bound"
        assert guards_intact(raw)
    assert fa.get_status() == fa.FA_OK


@pytest.mark.parametrize("B,N,Hq,Hk,d,dtype,rot,interleaved,heads_first,positions", CASES)
def test_backward(cuda_lib, B, N, Hq, Hk, d, dtype, rot, interleaved, heads_first, positions):
    q, k, wq, wk, g = make(B, N, Hq, Hk, d, dtype, 13 * N + d, w_f32=N % 2 == 1)
    pos = positions_of(positions, B, N, g)
    freqs = fa.rope_freqs(rot)
    shape = (lambda h: (B, h, N, d)) if heads_first else (lambda h: (B, N, h, d))
    dyq, dyk = (torch.randn(shape(h), generator=g).to(DTYPES[dtype]).cuda() for h in (Hq, Hk))
    # gradients into a packed buffer whose value part must stay as it is
    packed = torch.full((B, N, Hq + 2 * Hk, d), 7.0, dtype=DTYPES[dtype], device="cuda")
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(q, k, dyq, dyk, wq, wk, freqs, positions=pos, eps=1e-5,
                                           interleaved=interleaved, heads_first=heads_first,
                                           dq=packed[:, :, :Hq], dk=packed[:, :, Hq:Hq + Hk])
    assert bool((packed[:, :, Hq + Hk:] == 7).all())
    for x, dy, w, dx, dw in ((q, dyq, wq, dq, dwq), (k, dyk, wk, dk, dwk)):
        gy = to_np64(dy)
        gy = gy.transpose(0, 2, 1, 3) if heads_first else gy
        wx, ww, sx, sw = ref.norm_rope_bwd(to_np64(x), gy, to_np64(w), where(pos, B, N), turns_of(freqs),
                                           np.float32(1e-5), interleaved)
        err = np.abs(to_np64(dx) - wx)
        bound = half_step(dtype) * np.abs(wx) + 128 * U * sx + tiny(dtype)
        assert np.all(err <= bound), f"dx worst excess {(err / bound).max():.3f} of the bound"
        err = np.abs(to_np64(dw) - ww)
        assert np.all(err <= 256 * U * sw + 1e-30), f"dw worst excess {(err / (256 * U * sw)).max():.3f} of the bound"
    assert fa.get_status() == fa.FA_OK


def test_gradient_against_differences_of_the_kernel(cuda_lib):
    """fp32: the kernel's gradient against central differences of the kernel's own forward,
    along random directions (step 2^-9: the third-order term is below 1e-4 of the sum and
    the rounding of the results, 2^-20 of each of 512, below 1e-3 of it)."""
    q, k, wq, wk, g = make(1, 4, 1, 1, 64, "f32", 5, packed=False)
    freqs = fa.rope_freqs(64)
    dyq, dyk = (torch.randn(1, 1, 4, 64, generator=g).cuda() for _ in range(2))
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(q, k, dyq, dyk, wq, wk, freqs, eps=1e-2)
    def loss(q, k, wq, wk):
        a, b = fa.qk_norm_rope(q, k, wq, wk, freqs, eps=1e-2)
        return float((a.double() * dyq.double()).sum() + (b.double() * dyk.double()).sum())
    at = [q, k, wq, wk]
    for i, grad in enumerate((dq, dk, dwq, dwk)):
        step = torch.randn(at[i].shape, generator=g).cuda()
        plus, minus = list(at), list(at)
        plus[i], minus[i] = at[i] + step * 2.0 ** -9, at[i] - step * 2.0 ** -9
        want = (loss(*plus) - loss(*minus)) * 2.0 ** 8
        size = float((grad.double() * step.double()).abs().sum())
        assert abs(float((grad.double() * step.double()).sum()) - want) <= 2e-3 * size


def test_in_place_and_zero_tokens(cuda_lib):
    q, k, wq, wk, _ = make(2, 21, 4, 2, 128, "bf16", 9)
    freqs = fa.rope_freqs(128)
    want = fa.qk_norm_rope(q, k, wq, wk, freqs, heads_first=False)
    fa.qk_norm_rope(q, k, wq, wk, freqs, heads_first=False, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    q0, k0 = q[:, :0], k[:, :0]
    yq, yk = fa.qk_norm_rope(q0, k0, wq, wk, freqs)
    assert yq.shape == (2, 4, 0, 128) and yk.shape == (2, 2, 0, 128)
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(q0, k0, yq, yk, wq, wk, freqs)
    assert float(dwq.abs().sum()) == 0 and float(dwk.abs().sum()) == 0


@pytest.mark.parametrize("dtype,d,rot", [("bf16", 128, 128), ("f32", 64, 32), ("f16", 64, 18)])
def test_gradients_over_their_inputs(cuda_lib, dtype, d, rot):
    """dq, dk written over q, k and over dyq, dyk: the same bits as elsewhere."""
    q, k, wq, wk, g = make(2, 300, 5, 2, d, dtype, 17, packed=False)
    freqs = fa.rope_freqs(rot)
    dyq, dyk = (torch.randn(x.shape, generator=g).to(x.dtype).cuda() for x in (q, k))
    want = fa.qk_norm_rope_bwd(q, k, dyq, dyk, wq, wk, freqs, heads_first=False)
    over_dy = [x.clone() for x in (dyq, dyk)]
    got = fa.qk_norm_rope_bwd(q, k, *over_dy, wq, wk, freqs, heads_first=False, dq=over_dy[0], dk=over_dy[1])
    assert got[0].data_ptr() == over_dy[0].data_ptr() and all(torch.equal(a, b) for a, b in zip(got, want))
    got = fa.qk_norm_rope_bwd(q, k, dyq, dyk, wq, wk, freqs, heads_first=False, dq=q, dk=k)
    assert got[0].data_ptr() == q.data_ptr() and all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_calls_at_once(cuda_lib):
    """Forward and backward passes of two inputs on two streams; results equal to plain calls'."""
    sets = []
    for seed, (N, rot) in enumerate(((2000, 64), (700, 30))):
        q, k, wq, wk, g = make(1, N, 8, 8, 64, "bf16", 40 + seed)
        dyq, dyk = (torch.randn(1, 8, N, 64, generator=g).bfloat16().cuda() for _ in range(2))
        sets.append((q, k, dyq, dyk, wq, wk, fa.rope_freqs(rot)))
    run = lambda q, k, dyq, dyk, wq, wk, f, stream=None: (fa.qk_norm_rope(q, k, wq, wk, f, stream=stream)
                                                         + fa.qk_norm_rope_bwd(q, k, dyq, dyk, wq, wk, f, stream=stream))
    want = [run(*s) for s in sets]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(10):
        got += [[run(*s, stream=t), w] for s, t, w in zip(sets, side, want)]
    torch.cuda.synchronize()
    for g, w in got:
        assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_rows_of_zeros_infinities_and_nans_stay_in_their_rows(cuda_lib):
    q, k, wq, wk, _ = make(1, 16, 2, 1, 64, "f32", 21, packed=False)
    freqs = fa.rope_freqs(64)
    want = fa.qk_norm_rope(q, k, wq, wk, freqs, heads_first=False)
    q[0, 3, 1, 5], q[0, 7, 0, 0], q[0, 9] = float("nan"), float("inf"), 0.0
    got = fa.qk_norm_rope(q, k, wq, wk, freqs, heads_first=False)
    clean = torch.ones(1, 16, 2, dtype=torch.bool)
    clean[0, 3, 1] = clean[0, 7, 0] = clean[0, 9] = False
    assert torch.equal(got[0].cpu()[clean], want[0].cpu()[clean]) and torch.equal(got[1], want[1])
    assert bool(got[0][0, 3, 1].isnan().all())
    assert float(got[0][0, 9].abs().sum()) == 0


def test_another_stream_and_graph(cuda_lib):
    q, k, wq, wk, g = make(1, 70, 4, 4, 64, "bf16", 31)
    freqs = fa.rope_freqs(64)
    dyq, dyk = (torch.randn(1, 4, 70, 64, generator=g).bfloat16().cuda() for _ in range(2))
    want = fa.qk_norm_rope(q, k, wq, wk, freqs) + fa.qk_norm_rope_bwd(q, k, dyq, dyk, wq, wk, freqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.qk_norm_rope(q, k, wq, wk, freqs, stream=side) + fa.qk_norm_rope_bwd(q, k, dyq, dyk, wq, wk, freqs, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = fa.qk_norm_rope(q, k, wq, wk, freqs) + fa.qk_norm_rope_bwd(q, k, dyq, dyk, wq, wk, freqs)
    for t in held:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))
