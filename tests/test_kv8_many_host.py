"""The append of many tokens by hand against the one that goes block by block."""
import numpy as np
import pytest

import _kv8_many as many
import _kv8_ref as ref


@pytest.mark.parametrize("d,H,page", [(64, 3, 16), (128, 2, 64)])
def test_the_same_bytes(d, H, page):
    rng = np.random.default_rng(d)
    pages = 12 * 64 // page
    a = rng.integers(0, 256, (pages, H, page // 16, ref.block_bytes(d))).astype(np.uint8)
    a[..., 32 * d:32 * d + 8] = np.array([0.5, 2.0 ** -9], np.float32).view(np.uint8)
    b, order = a.copy(), rng.permutation(pages * page // 16)
    at = 0
    for n in (5, 40, 1, 17, 200):
        slots = np.concatenate([order[(np.arange(at, at + n)) // 16] * 16 + np.arange(at, at + n) % 16, [-1], order[40 + n % 7] * 16 + np.array([3, 4])])
        at += n
        x = rng.standard_normal((2, len(slots), H, d)).astype(np.float32) * 10.0 ** rng.integers(-30, 6, (2, len(slots), H, 1))
        x[0, 0, 0, 3], x[1, -1, 1, 0], x[0, 1 % n, 1, 5], x[1, 0] = np.nan, np.nan, np.inf, 0
        ref.append(a, x[0], x[1], slots)
        many.append(b, x[0], x[1], slots)
        assert np.array_equal(a, b)
        some = slots[slots >= 0]
        for g, w in zip(many.values(b, some, d), ref.slot_values(a, some, d)):
            assert np.array_equal(g, w, equal_nan=True)


def test_scales():
    most = np.abs(np.random.default_rng(0).standard_normal(2000)) * 10.0 ** np.random.default_rng(1).integers(-40, 4, 2000)
    most = np.concatenate([most, [0, 127, 127.5, 63.5, 16384, 1e-300], 127 * 2.0 ** np.arange(-70, 7)])
    assert np.array_equal(many.scales_for(most), [ref.scale_for(m) for m in most])
