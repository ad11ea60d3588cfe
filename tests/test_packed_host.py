"""Host-side checks of packed attention: the plain reference against differences, and the argument
checks of the C entries (before any CUDA call)."""
import ctypes

import pytest
import torch

import _packed_ref as ref
import exact_io_aware_26_gb300 as fa

OK = 1 << 20  # an aligned address that is never dereferenced
L2 = ctypes.c_longlong * 2


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.load()


@pytest.mark.parametrize("causal", [True, False])
def test_reference_gradient_against_differences(causal):
    g = torch.Generator().manual_seed(1)
    new, keys, scale = [3, 2, 4], [3, 5, 2], 0.7
    x = [torch.randn(n, h, 8, generator=g, dtype=torch.float64) for n, h in ((9, 4), (10, 2), (10, 2), (9, 4))]
    q, k, v, do = x
    fwd = lambda: ref.forward(q, k, v, new, keys, causal, scale, 0.0, 0.0)
    o, lse, _, _ = fwd()
    grads, _ = ref.backward(q, k, v, o, do, lse, new, keys, causal, scale, 0.0, 0.0)
    for t, grad in zip((q, k, v), grads):
        for i in range(0, t.numel(), 7):
            was = t.view(-1)[i].item()
            f = []
            for step in (1e-6, -1e-6):
                t.view(-1)[i] = was + step
                f.append((fwd()[0] * do).sum().item())
            t.view(-1)[i] = was
            assert abs((f[0] - f[1]) / 2e-6 - grad.reshape(-1)[i].item()) < 1e-7


def params(**kw):
    base = dict(R=2, Tq=8, Tk=8, Hq=4, Hk=2, d=64, dtype=fa.FA_BF16, causal=1, scale=0.1)
    for n in ("q", "o", "do", "dq"):
        base[n + "_stride"] = L2(256, 64)
    for n in ("k", "v", "dk", "dv"):
        base[n + "_stride"] = L2(128, 64)
    return fa.FaPackedParams(**{**base, **kw})


BAD = [({"R": 0}, -1), ({"R": 1 << 24}, -2), ({"Tq": -1}, -1), ({"Tk": -1}, -1), ({"d": 96}, -2), ({"dtype": fa.FA_F32}, -2),
       ({"dtype": 7}, -1), ({"Hq": 3}, -1), ({"Hq": 0}, -1), ({"Hk": 0}, -1), ({"Hq": 258, "Hk": 2}, -2), ({"scale": 0.0}, -1),
       ({"scale": float("nan")}, -1), ({"Tq": 1 << 30}, -2), ({"Tk": (1 << 30) + 1, "Hk": 1}, -2), ({"q_stride": L2(257, 64)}, -1),
       ({"k_stride": L2(128, -64)}, -1), ({"v_stride": L2(0, 64)}, -2), ({"q_stride": L2(256, 0)}, -2), ({"k_stride": L2(1 << 38, 64)}, -2)]


@pytest.mark.parametrize("kw,code", BAD + [({"o_stride": L2(64, 64)}, -1)])
def test_forward_refusals(lib, kw, code):
    p = ctypes.byref(params(**kw))
    assert lib.fa_fwd_packed_workspace_size(p) == 0
    assert lib.fa_fwd_packed(p, *[OK + (i << 20) for i in range(8)], 1 << 40, None) == code


@pytest.mark.parametrize("kw,code", BAD + [({"dq_stride": L2(64, 64)}, -1), ({"dk_stride": L2(64, 64)}, -1), ({"dv_stride": L2(0, 64)}, -1),
                                           ({"do_stride": L2(0, 64)}, -2)])
def test_backward_refusals(lib, kw, code):
    p = ctypes.byref(params(**kw))
    assert lib.fa_bwd_packed_workspace_size(p) == 0
    assert lib.fa_bwd_packed(p, *[OK + (i << 20) for i in range(12)], 1 << 40, None) == code


def test_pointers(lib):
    p = ctypes.byref(params())
    for entry, size, n in ((lib.fa_fwd_packed, lib.fa_fwd_packed_workspace_size(p), 7),
                           (lib.fa_bwd_packed, lib.fa_bwd_packed_workspace_size(p), 11)):
        assert size > 0
        good = [OK + (i << 20) for i in range(n + 1)]
        null_ok = 4 if n == 7 else 7  # cu_k
        for i in range(n):
            for bad in (good[i] + 2,) if i == null_ok else (None, good[i] + 2):
                a = list(good)
                a[i] = bad
                assert entry(p, *a, size, None) == fa.FA_ERR_INVALID
        for ws, nbytes in ((None, size), (OK, size - 1), (OK + 16, size)):
            assert entry(p, *good[:-1], ws, nbytes, None) == fa.FA_ERR_WORKSPACE
        assert entry(None, *good, size, None) == fa.FA_ERR_INVALID
    for j in (0, 1, 2):  # o over q, k, v
        a = [OK + (i << 20) for i in range(8)]
        a[5] = a[j]
        assert lib.fa_fwd_packed(p, *a, 1 << 40, None) == fa.FA_ERR_INVALID
    b = [OK + (i << 20) for i in range(12)]
    # dk, dv over q, k, v, do; gradients over each other
    for i, j in [(i, j) for i in (9, 10) for j in (0, 1, 2, 4)] + [(9, 8), (10, 8), (10, 9)]:
        c = list(b)
        c[i] = c[j]
        assert lib.fa_bwd_packed(p, *c, 1 << 40, None) == fa.FA_ERR_INVALID
    without = [OK + (i << 20) for i in range(8)]
    without[4] = None
    assert lib.fa_fwd_packed(ctypes.byref(params(Tk=9)), *without, 1 << 40, None) == fa.FA_ERR_INVALID
    assert b"cu_k" in lib.fa_last_error()
