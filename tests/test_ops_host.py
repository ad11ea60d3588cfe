"""Host-side checks of the operators around the attention: the plain references, the
argument checks of the C entries (before any CUDA call) and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

import _ops_ref as ref
import exact_io_aware_26_gb300 as fa

OK = 1 << 20  # an aligned address that is never dereferenced


def apart(n):
    """n such addresses, none over another."""
    return [OK + (i << 20) for i in range(n)]


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.load()


def test_reference_gradient_against_differences():
    """The backward's 64-bit formula against central differences of the forward's."""
    rng = np.random.default_rng(3)
    for interleaved in (False, True):
        x, w, dy = rng.standard_normal((1, 2, 1, 8)), rng.standard_normal(8), rng.standard_normal((1, 2, 1, 8))
        pos, turns = np.array([[5, 70001]]), np.array([2 ** 61, 12345 * 2 ** 40], np.uint64)
        loss = lambda x, w: (ref.norm_rope(x, w, pos, turns, 1e-3, interleaved)[0] * dy).sum()
        dx, dw, _, _ = ref.norm_rope_bwd(x, dy, w, pos, turns, 1e-3, interleaved)
        for idx in np.ndindex(x.shape):
            e = np.zeros_like(x)
            e[idx] = 1e-6
            assert abs((loss(x + e, w) - loss(x - e, w)) / 2e-6 - dx[idx]) < 1e-7
        for c in range(8):
            e = np.zeros_like(w)
            e[c] = 1e-6
            assert abs((loss(x, w + e) - loss(x, w - e)) / 2e-6 - dw[c]) < 1e-7


def test_reference_quantiser():
    """Each value within half a step of its input and the fp16 roundings; constants are kept."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 2, 64)).astype(np.float32)
    c, s, b = ref.quantise(x)
    err = np.abs(ref.values(c, s, b) - x)
    S, B = (np.repeat(np.abs(a.astype(np.float64)), 32, -1) for a in (s, b))
    assert np.all(err <= S / 32 + 2.0 ** -11 * (3 * S + 2 * B)) and c.min() == 0 and c.max() == 15
    flat = np.full((1, 1, 64), 1.5, np.float32)
    assert np.all(ref.values(*ref.quantise(flat)) == 1.5)
    k = ref.cache_of(x, 2 * x, 16)
    got = ref.slot_values(k, np.arange(50), 64)
    assert np.array_equal(got[0], ref.values(c, s, b))


def test_reference_plan():
    kv, cu, pos, slots, counts, table, stack = ref.plan([3, 5, 0], [2, -1, 3], [[7, -1], [4, 1], [-1, -1]], [2, 9, 0], 2, 4, 6)
    assert (kv, cu, pos, slots) == ([5, 0, 3], [0, 2, 2, 5], [3, 4, 0, 1, 2, 0], [31, 4, 16, 17, 18, -1])
    assert counts == [2, 5, 0] and table == [[7, 1], [4, 1], [4, -1]] and stack == [2, 9, 0]


def test_rope_freqs():
    f = fa.rope_freqs(64, device="cpu")
    want = 10000.0 ** (-2 * np.arange(32) / 64) / (2 * np.pi)
    assert f.dtype == torch.int64 and np.allclose(f.numpy().view(np.uint64) / 2.0 ** 64, want, rtol=1e-15)
    g = fa.rope_freqs(4, inv_freq=[-1.0, 0.5], device="cpu").numpy().view(np.uint64) / 2.0 ** 64
    assert np.allclose(g, [1 - 1 / (2 * np.pi), 0.5 / (2 * np.pi)])
    assert fa.rope_freqs(0, device="cpu").numel() == 0
    for bad in (dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=4, inv_freq=[1.0]), dict(rot_dim=2, inv_freq=[float("nan")])):
        with pytest.raises(ValueError):
            fa.rope_freqs(**bad, device="cpu")


L3 = ctypes.c_longlong * 3
L2 = ctypes.c_longlong * 2


def qk(**kw):
    base = dict(B=2, N=8, Hq=4, Hk=2, d=64, dtype=fa.FA_BF16, weight_dtype=fa.FA_F32, rot_dim=64, interleaved=0, eps=1e-6,
                pos_stride=8, q_stride=L3(4096, 512, 64), k_stride=L3(4096, 512, 64), yq_stride=L3(2048, 64, 512),
                yk_stride=L3(1024, 64, 512), dq_stride=L3(4096, 512, 64), dk_stride=L3(4096, 512, 64))
    base.update(kw)
    return fa.FaQkParams(**base)


QK_BAD = [({"B": 0}, -1), ({"N": -1}, -1), ({"Hq": 0}, -1), ({"d": 96}, -2), ({"dtype": 9}, -1), ({"weight_dtype": fa.FA_F16}, -1),
          ({"rot_dim": 3}, -1), ({"rot_dim": 66}, -1), ({"rot_dim": -2}, -1), ({"eps": 0.0}, -1), ({"eps": float("nan")}, -1),
          ({"pos_stride": -1}, -1), ({"q_stride": L3(4096, 516, 64)}, -1), ({"q_stride": L3(-8, 512, 64)}, -1),
          ({"B": 1 << 16, "N": 1 << 16}, -2)]


@pytest.mark.parametrize("kw,code", QK_BAD + [({"yq_stride": L3(2048, 64, 0)}, -1), ({"yq_stride": L3(2048, 64, 256)}, -1),
                                              ({"yk_stride": L3(512, 64, 512)}, -1)])
def test_qk_norm_rope_refusals(lib, kw, code):
    assert lib.fa_qk_norm_rope(ctypes.byref(qk(**kw)), *[OK] * 8, None) == code


@pytest.mark.parametrize("kw,code", QK_BAD + [({"dq_stride": L3(4096, 64, 64)}, -1)])
def test_qk_norm_rope_bwd_refusals(lib, kw, code):
    p = qk(**kw)
    assert lib.fa_qk_norm_rope_bwd_workspace_size(ctypes.byref(p)) == 0
    assert lib.fa_qk_norm_rope_bwd(ctypes.byref(p), *[OK] * 13, 1 << 30, None) == code


def test_qk_pointers(lib):
    p = ctypes.byref(qk())
    for i in range(8):  # q k wq wk freqs positions yq yk
        for bad in ((None, OK + 2) if i != 5 else (OK + 2,)):
            a = apart(8)
            a[i] = bad
            assert lib.fa_qk_norm_rope(p, *a, None) == fa.FA_ERR_INVALID
    assert lib.fa_qk_norm_rope(None, *[OK] * 8, None) == fa.FA_ERR_INVALID
    need = lib.fa_qk_norm_rope_bwd_workspace_size(p)
    assert need > 0
    for ws, n in ((None, need), (OK, need - 1), (OK + 16, need)):
        assert lib.fa_qk_norm_rope_bwd(p, *apart(12), ws, n, None) == fa.FA_ERR_WORKSPACE
    assert b"workspace" in lib.fa_last_error()


def cache(**kw):
    return fa.FaKv4Cache(**{**dict(num_pages=10, page_size=64, Hk=2, d=64, page_stride=2 * 4 * 1280), **kw})


CACHE_BAD = [({"num_pages": 0}, -1), ({"Hk": 0}, -1), ({"d": 32}, -2), ({"page_size": 8}, -2), ({"page_size": 48}, -2),
             ({"page_size": 8192}, -2), ({"page_stride": 2 * 4 * 1280 - 16}, -1), ({"page_stride": 2 * 4 * 1280 + 8}, -1),
             ({"num_pages": 1 << 26}, -2)]


@pytest.mark.parametrize("kw,code", CACHE_BAD)
def test_cache_refusals(lib, kw, code):
    c, rows = ctypes.byref(cache(**kw)), ctypes.byref(fa.FaKv4Rows(4, fa.FA_BF16, L2(128, 64), L2(128, 64)))
    assert lib.fa_kv4_append(c, rows, *[OK] * 4, None) == code
    assert lib.fa_kv4_gather(c, rows, *[OK] * 4, None) == code
    assert lib.fa_kv4_attention_workspace_size(c, ctypes.byref(attn())) == 0
    assert lib.fa_kv4_attention(c, ctypes.byref(attn()), *[OK] * 8, 1 << 30, None) == code


@pytest.mark.parametrize("rows,code", [((-1, 2, (128, 64)), -1), ((4, 7, (128, 64)), -1), ((4, 2, (129, 64)), -1), ((4, 2, (-8, 64)), -1)])
def test_rows_refusals(lib, rows, code):
    T, dt, st = rows
    r = ctypes.byref(fa.FaKv4Rows(T, dt, L2(*st), L2(128, 64)))
    assert lib.fa_kv4_append(ctypes.byref(cache()), r, *[OK] * 4, None) == code
    overlapping = ctypes.byref(fa.FaKv4Rows(4, 2, L2(64, 64), L2(128, 64)))
    assert lib.fa_kv4_gather(ctypes.byref(cache()), overlapping, *[OK] * 4, None) == fa.FA_ERR_INVALID
    good = ctypes.byref(fa.FaKv4Rows(4, 2, L2(128, 64), L2(128, 64)))
    for i in range(4):
        for bad in (None, OK + 2):
            a = [OK] * 4
            a[i] = bad
            assert lib.fa_kv4_append(ctypes.byref(cache()), good, *a, None) == fa.FA_ERR_INVALID
            assert lib.fa_kv4_gather(ctypes.byref(cache()), good, *a, None) == fa.FA_ERR_INVALID


def attn(**kw):
    return fa.FaKv4AttnParams(**{**dict(R=2, T=2, Hq=4, dtype=fa.FA_BF16, max_q_len=1, window=0, table_width=5, scale=0.1,
                                        table_stride=5, q_stride=L2(256, 64), o_stride=L2(256, 64)), **kw})


@pytest.mark.parametrize("kw,code", [({"R": 0}, -1), ({"T": -1}, -1), ({"Hq": 3}, -1), ({"Hq": 0}, -1), ({"dtype": fa.FA_F32}, -2),
                                     ({"dtype": 8}, -1), ({"max_q_len": 0}, -1), ({"window": -1}, -1), ({"table_width": 0}, -1),
                                     ({"table_stride": 4}, -1), ({"scale": 0.0}, -1), ({"scale": float("inf")}, -1),
                                     ({"q_stride": L2(257, 64)}, -1), ({"o_stride": L2(64, 64)}, -1),
                                     ({"T": 1 << 30}, -2), ({"table_width": 1 << 28, "table_stride": 1 << 28}, -2)])
def test_attention_refusals(lib, kw, code):
    c, p = ctypes.byref(cache()), ctypes.byref(attn(**kw))
    assert lib.fa_kv4_attention_workspace_size(c, p) == 0
    assert lib.fa_kv4_attention(c, p, *[OK] * 8, 1 << 30, None) == code


def test_attention_pointers(lib):
    c, p = ctypes.byref(cache()), ctypes.byref(attn())
    need = lib.fa_kv4_attention_workspace_size(c, p)
    assert need > 0
    for i, may_be_null in enumerate((False, False, False, False, True, False, True)):  # q cache table lens cu o lse
        for bad in (OK + 2,) if may_be_null else (None, OK + 2):
            a = [OK] * 7
            a[i] = bad
            assert lib.fa_kv4_attention(c, p, *a, OK, need, None) == fa.FA_ERR_INVALID
    for ws, n in ((None, need), (OK, need - 1), (OK + 16, need)):
        assert lib.fa_kv4_attention(c, p, *[OK] * 7, ws, n, None) == fa.FA_ERR_WORKSPACE
    a = [OK] * 7  # a result over its queries, which other CTAs still read
    assert lib.fa_kv4_attention(c, p, *a, OK, need, None) == fa.FA_ERR_INVALID
    assert b"over q" in lib.fa_last_error()


@pytest.mark.parametrize("kw,code", [({"R": 0}, -1), ({"T": -1}, -1), ({"page_size": 0}, -1), ({"num_pages": 0}, -1),
                                     ({"R": 8193}, -2), ({"table_width": 0}, -1), ({"table_stride": 3}, -1)])
def test_plan_refusals(lib, kw, code):
    p = fa.FaPlanParams(**{**dict(R=4, T=4, page_size=16, num_pages=10, table_width=4, table_stride=4), **kw})
    assert lib.fa_paged_plan(ctypes.byref(p), *[OK] * 10, None) == code
    good = fa.FaPlanParams(4, 4, 16, 10, 4, 4)
    for i in range(10):
        for bad in (None, OK + 2):
            a = [OK] * 10
            a[i] = bad
            assert lib.fa_paged_plan(ctypes.byref(good), *a, None) == fa.FA_ERR_INVALID


def test_sizes_that_would_overflow_are_refused(lib):
    good = dict(R=4, T=4, page_size=16, num_pages=10, table_width=4, table_stride=4)
    for kw in ({"T": (1 << 30) + 1}, {"num_pages": (1 << 30) + 1}):
        assert lib.fa_paged_plan(ctypes.byref(fa.FaPlanParams(**{**good, **kw})), *[OK] * 10, None) == fa.FA_ERR_UNSUPPORTED
    assert lib.fa_qk_norm_rope(ctypes.byref(qk(Hq=1 << 23, Hk=1 << 23)), *[OK] * 8, None) == fa.FA_ERR_UNSUPPORTED
    far = L3(1 << 40, 1 << 31, 64)
    assert lib.fa_qk_norm_rope(ctypes.byref(qk(q_stride=far)), *[OK] * 8, None) == fa.FA_ERR_UNSUPPORTED
    rows = fa.FaKv4Rows(4, fa.FA_BF16, L2(1 << 31, 64), L2(128, 64))
    assert lib.fa_kv4_append(ctypes.byref(cache()), ctypes.byref(rows), *[OK] * 4, None) == fa.FA_ERR_UNSUPPORTED


def test_results_over_their_inputs_need_the_same_strides(lib):
    """In place with another layout would overwrite rows before they are read."""
    a = apart(8)
    a[7] = a[1]  # yk over k, whose strides are others
    assert lib.fa_qk_norm_rope(ctypes.byref(qk()), *a, None) == fa.FA_ERR_INVALID
    assert b"strides" in lib.fa_last_error()


def test_launch_registers_and_forgets():
    """The extension knows a combination only once it is registered, tells sizes, strides,
    types and scalars apart, and forgets when the library changes."""
    from exact_io_aware_26_gb300 import _launch
    _launch.clear()
    t = torch.zeros(4, 6)
    assert _launch.run(99, (t, None), (1, 2.0)) is None
    _launch.register(99, (t, None), (1, 2.0), 0, 0, [(2, 0)] * 7, [], [], None)
    for tensors, scalars in (((t.t(), None), (1, 2.0)), ((t.double(), None), (1, 2.0)), ((t, t), (1, 2.0)),
                             ((t[:, :5], None), (1, 2.0)), ((t, None), (1, 3.0))):
        assert _launch.run(99, tensors, scalars) is None
    with pytest.raises(TypeError):
        _launch.run(99, ([1], None), (1, 2.0))
    with pytest.raises(ValueError):
        _launch.register(99, (t,), (), 0, 0, [(2, 0)] * 3, [], [], None)
    with pytest.raises(ValueError):
        _launch.register(99, (t,), (), 0, 0, [(0, 5)] * 7, [], [], None)
    fa.use_library(fa.use_library(fa.LIB_PATH))
    assert _launch.run(99, (t, None), (1, 2.0)) is None
    fa.load()


def test_block_bytes(lib):
    assert [fa.kv4_block_bytes(d) for d in (32, 64, 128)] == [0, 1280, 2560] == [0] + [ref.block_bytes(d) for d in (64, 128)]


def test_binding_rejects_cpu_tensors():
    q, w = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16), torch.ones(64)
    f = fa.rope_freqs(64, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(1, 1, 1, 1280, dtype=torch.uint8)
    for call in (lambda: fa.qk_norm_rope(q, q, w, w, f), lambda: fa.qk_norm_rope_bwd(q, q, q, q, w, w, f),
                 lambda: fa.kv4_append(q[0], q[0], i, c), lambda: fa.kv4_gather(c, i, 64),
                 lambda: fa.kv4_attention(q[0], c, i[None], i, scale=1.0),
                 lambda: fa.paged_plan(i, i, i[None].expand(2, 2).contiguous(), i, i, 16, 2)):
        with pytest.raises(ValueError):
            call()
    for bad in (dict(d=96), dict(page_size=24), dict(page_size=8)):
        with pytest.raises(ValueError):
            fa.kv4_cache(**{**dict(num_pages=1, heads=1, d=64, page_size=16, device="cpu"), **bad})
