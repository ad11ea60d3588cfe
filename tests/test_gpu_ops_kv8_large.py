"""The 8-bit cache's append of so many tokens that a warp takes several blocks, or both sides of them: every
byte as by hand."""
import numpy as np
import pytest
import torch

import _kv8_many as many
import _kv8_ref as ref
import exact_io_aware_26_gb300 as fa
from _parity import DTYPES, guarded, guards_intact, to_np64

pytestmark = pytest.mark.gpu


def rows(T, H, d, dtype, seed):
    """T rows of keys and values, one packed projection; some of them zero, huge, tiny, NaN or infinite."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, 2 * H, d, generator=g, device="cuda")
    odd = torch.rand(T, 2 * H, generator=g, device="cuda")
    for at, f in ((0.01, 0.0), (0.02, 1e3), (0.03, 1e-4), (0.04, 1e4)):
        x[(odd < at) & (odd >= at - 0.01)] *= f
    x[..., 7][(odd > 0.99) & (odd < 0.995)] = float("nan")
    x[..., 9][odd >= 0.995] = float("inf")
    x = x.to(DTYPES[dtype])
    return x[:, :H], x[:, H:]


@pytest.mark.parametrize("H,d,dtype,span", [
    # `span`: the tokens among which a warp's blocks begin, 2 T H / (64 warps for each SM), at most 16
    (12, 64, "bf16", 16), (12, 64, "f16", 16), (1, 64, "bf16", 20),   # both sides a warp
    (12, 64, "f32", 16), (8, 128, "bf16", 16), (8, 128, "f16", 3), (3, 128, "f32", 17),
    (5, 64, "bf16", 7), (7, 128, "f32", 2), (2, 64, "f16", 15.9)])
def test_large_calls(cuda_lib, H, d, dtype, span):
    sms, page, R = torch.cuda.get_device_properties(0).multi_processor_count, 64, 5
    T = int(span * sms * 32 / H) + 33
    rng = np.random.default_rng(T)
    # a prompt of most of the rows, short ones around it, one that is left out; each in two calls after a few tokens
    news = [[5, 0, 1, 16, 3], [7, T - 500, 31, 16, 300], [1, T - 300, 90, 100, 0]]
    most = [sum(n[r] for n in news) for r in range(R)]
    have = [-(-m // page) for m in most]
    order = rng.permutation(sum(have) + 3)
    first = np.concatenate([[0], np.cumsum(have)])
    want = rng.integers(0, 256, (sum(have) + 3, H, page // 16, ref.block_bytes(d))).astype(np.uint8)
    raw, cache = guarded(want.shape, torch.uint8)
    cache.copy_(torch.from_numpy(want))
    held = np.zeros(R, int)
    for i, new in enumerate(news):
        slots = []
        for r, n in enumerate(new):
            t = np.arange(held[r], held[r] + n)
            slots += [order[first[r] + t // page] * page + t % page, [-1] * (i * r % 3)]
            held[r] += n
        slots = np.concatenate(slots).astype(np.int64)
        k, v = rows(len(slots), H, d, dtype, 10 * i)
        fa.kv8_append(k, v, torch.from_numpy(slots.astype(np.int32)).cuda(), cache)
        many.append(want, k.float().cpu().numpy(), v.float().cpu().numpy(), slots)
        got = cache.cpu().numpy()
        assert np.array_equal(got, want), np.argwhere(got != want)[:5]
    assert guards_intact(raw) and fa.get_status() == fa.FA_OK
    back = np.concatenate([order[first[r] + np.arange(held[r]) // page] * page + np.arange(held[r]) % page for r in range(R)])
    back = np.concatenate([back[1:], back[:1]])[:20001]  # groups of four that begin anywhere in a block
    for g, w in zip(fa.kv8_gather(cache, torch.from_numpy(back.astype(np.int32)).cuda(), d, dtype=torch.float32), many.values(want, back, d)):
        assert np.array_equal(to_np64(g), w, equal_nan=True)
