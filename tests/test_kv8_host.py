"""Host-side checks of the 8-bit cache: the plain reference, and the argument checks of the C entries
(before any CUDA call)."""
import ctypes

import numpy as np
import pytest

import _kv8_ref as ref
import exact_io_aware_26_gb300 as fa

OK = 1 << 20  # an aligned address that is never dereferenced
L2 = ctypes.c_longlong * 2


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.load()


@pytest.mark.parametrize("d", [64, 128])
def test_reference(d):
    """Every byte of a block has one place; values come back within half a step, and within a step
    of the larger scale where later tokens raised it; marks come and go with their tokens."""
    at = ref.places(d)
    assert sorted(at.reshape(-1)) == list(range(32 * d)) and ref.block_bytes(d) == 32 * d + 16
    rng = np.random.default_rng(0)
    x = rng.standard_normal((20, 2, d)).astype(np.float32)
    cache = np.full((2, 2, 1, ref.block_bytes(d)), 0xFF, np.uint8)
    ref.append(cache, x, 2 * x, np.arange(20))
    k, v = ref.slot_values(cache, np.arange(20), d)
    for rows in (slice(0, 16), slice(16, 20)):
        step = np.array([ref.scale_for(m) for m in np.abs(x[rows]).max((0, 2))])[:, None]
        assert np.all(np.abs(k[rows] - x[rows]) <= step / 2) and np.all(np.abs(v[rows] - 2 * x[rows]) <= step)
    big = np.full((1, 2, d), 50.0, np.float32)
    bad = big.copy()
    bad[0, 1, 3] = np.nan
    ref.append(cache, big, bad, np.array([20]))
    k2, v2 = ref.slot_values(cache, np.arange(21), d)
    assert np.all(np.abs(k2[16:20] - x[16:20]) <= 0.5) and np.array_equal(k2[:16], k[:16]) and np.all(k2[20] == 50)
    assert np.isnan(v2[20, 1]).all() and np.all(v2[20, 0] == 50) and np.isfinite(v2[:20]).all()
    ref.append(cache, big, big, np.array([20]))
    assert np.all(ref.slot_values(cache, np.array([20]), d)[1] == 50)


def test_scales():
    for most, want in ((0, 0), (127, 1), (127.5, 2), (63.5, 0.5), (np.nextafter(np.float32(63.5), np.float32(64)), 1), (1e-38, 2.0 ** -64),
                       (16384, 256)):
        assert ref.scale_for(float(most)) == want


def cache(**kw):
    return fa.FaKv4Cache(**{**dict(num_pages=10, page_size=64, Hk=2, d=64, page_stride=2 * 4 * 2064), **kw})


def attn(**kw):
    return fa.FaKv4AttnParams(**{**dict(R=2, T=2, Hq=4, dtype=fa.FA_BF16, max_q_len=1, window=0, table_width=5, scale=0.1,
                                        table_stride=5, q_stride=L2(256, 64), o_stride=L2(256, 64)), **kw})


@pytest.mark.parametrize("kw,code", [({"num_pages": 0}, -1), ({"Hk": 0}, -1), ({"d": 32}, -2), ({"page_size": 8}, -2), ({"page_size": 48}, -2),
                                     ({"page_size": 8192}, -2), ({"page_stride": 2 * 4 * 2064 - 16}, -1), ({"page_stride": 2 * 4 * 2064 + 8}, -1),
                                     ({"num_pages": 1 << 26}, -2), ({"Hk": 1 << 20, "page_stride": 1 << 40}, -2)])
def test_cache_refusals(lib, kw, code):
    c, rows = ctypes.byref(cache(**kw)), ctypes.byref(fa.FaKv4Rows(4, fa.FA_BF16, L2(128, 64), L2(128, 64)))
    assert lib.fa_kv8_append(c, rows, *[OK] * 4, None) == code
    assert lib.fa_kv8_gather(c, rows, *[OK] * 4, None) == code
    assert lib.fa_kv8_attention_workspace_size(c, ctypes.byref(attn())) == 0
    assert lib.fa_kv8_attention(c, ctypes.byref(attn()), *[OK] * 8, 1 << 30, None) == code


@pytest.mark.parametrize("rows,code", [((-1, 2, (128, 64)), -1), ((4, 7, (128, 64)), -1), ((4, 2, (129, 64)), -1), ((4, 2, (-8, 64)), -1),
                                       ((1 << 29, 2, (128, 64)), -2), ((4, 2, (1 << 31, 64)), -2)])
def test_rows_refusals(lib, rows, code):
    T, dt, st = rows
    r = ctypes.byref(fa.FaKv4Rows(T, dt, L2(*st), L2(128, 64)))
    assert lib.fa_kv8_append(ctypes.byref(cache()), r, *[OK] * 4, None) == code
    overlapping = ctypes.byref(fa.FaKv4Rows(4, 2, L2(64, 64), L2(128, 64)))
    assert lib.fa_kv8_gather(ctypes.byref(cache()), overlapping, *[OK] * 4, None) == fa.FA_ERR_INVALID
    good = ctypes.byref(fa.FaKv4Rows(4, 2, L2(128, 64), L2(128, 64)))
    for i in range(4):
        for bad in (None, OK + 2):
            a = [OK] * 4
            a[i] = bad
            assert lib.fa_kv8_append(ctypes.byref(cache()), good, *a, None) == fa.FA_ERR_INVALID
            assert lib.fa_kv8_gather(ctypes.byref(cache()), good, *a, None) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("kw,code", [({"R": 0}, -1), ({"T": -1}, -1), ({"Hq": 3}, -1), ({"dtype": fa.FA_F32}, -2), ({"max_q_len": 0}, -1),
                                     ({"window": -1}, -1), ({"table_width": 0}, -1), ({"table_stride": 4}, -1), ({"scale": 0.0}, -1),
                                     ({"q_stride": L2(257, 64)}, -1), ({"o_stride": L2(64, 64)}, -1), ({"T": 1 << 30}, -2)])
def test_attention_refusals(lib, kw, code):
    c, p = ctypes.byref(cache()), ctypes.byref(attn(**kw))
    assert lib.fa_kv8_attention_workspace_size(c, p) == 0
    assert lib.fa_kv8_attention(c, p, *[OK] * 8, 1 << 30, None) == code


def test_attention_pointers(lib):
    c, p = ctypes.byref(cache()), ctypes.byref(attn())
    size = lib.fa_kv8_attention_workspace_size(c, p)
    assert size > 0 and lib.fa_kv8_block_bytes(64) == 2064 and lib.fa_kv8_block_bytes(128) == 4112 and lib.fa_kv8_block_bytes(96) == 0
    apart = [OK + (i << 20) for i in range(8)]
    for i, may_be_null in enumerate((False, False, False, False, True, False, True)):  # q cache table lens cu o lse
        for bad in (apart[i] + 2,) if may_be_null else (None, apart[i] + 2):
            a = list(apart)
            a[i] = bad
            assert lib.fa_kv8_attention(c, p, *a, size, None) == fa.FA_ERR_INVALID
    for ws, n in ((None, size), (OK, size - 1), (OK + 16, size)):
        assert lib.fa_kv8_attention(c, p, *apart[:7], ws, n, None) == fa.FA_ERR_WORKSPACE
    a = list(apart)
    a[5] = a[0]  # o over q
    assert lib.fa_kv8_attention(c, p, *a, size, None) == fa.FA_ERR_INVALID
