"""Small weights in the 8-bit cache's attention: a channel's result is as exact as its own values
allow, whatever the scales of the blocks that came before.

Bound of a channel, with e = eps(type) / 2, w a weight relative to the row's largest and l their sum:
     |do| <= e |o| + (2^-11 + 2 s + 2^-20) sum w |v| / l + 2^-25 sum |v| / l,  s = 2^-16 |q| |k| scale,
the bound of test_gpu_ops_kv8.py with the last term summed over what the channel itself holds: a
weight is rounded to fp16 (half a step is 2^-11 of it, or 2^-25 below fp16's normal numbers), times a
power of two that is 1 at least."""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_26_gb300 as fa
from _parity import to_np64

pytestmark = pytest.mark.gpu


def attend(k, v, q, dtype, wide, window=0):
    """(o, lse) of one request's newest token q [Hq, d] over the cached k, v [n, Hk, d], and what the
    cache holds of them."""
    n, Hk, d = k.shape
    pages = -(-n // 16)
    cache = fa.kv8_cache(pages, Hk, d, page_size=16)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    fa.kv8_append(*(torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda() for x in (k, v)), slots, cache)
    held = [to_np64(x) for x in fa.kv8_gather(cache, slots, d, dtype=torch.float32)]
    table = torch.full((1, 6250 if wide else pages), -1, dtype=torch.int32, device="cuda")  # wide: in shares
    table[0, :pages] = torch.arange(pages, dtype=torch.int32)
    q = torch.from_numpy(q).to(dtype)
    o, lse = fa.kv8_attention(q[None].cuda(), cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), scale=1.0)
    assert fa.get_status() == fa.FA_OK
    return to_np64(o)[0], to_np64(lse)[0], to_np64(q), held


def check(o, lse, q, held, dtype):
    e, G = torch.finfo(dtype).eps / 2, q.shape[0] // held[0].shape[1]
    for h in range(q.shape[0]):
        k, v = held[0][:, h // G], held[1][:, h // G]
        x = k @ q[h]
        w = np.exp(x - x.max())
        l = w.sum()
        s = 2.0 ** -16 * (np.abs(k) @ np.abs(q[h])).max()
        want = w @ v / l
        bound = e * np.abs(want) + (2.0 ** -11 + 2 * s + 2.0 ** -20) * (w @ np.abs(v)) / l + 2.0 ** -25 * np.abs(v).sum(0) / l
        err = np.abs(o[h] - want)
        assert np.all(err <= bound), f"head {h}: {(err / np.maximum(bound, 1e-300)).max():.1f} of the bound"
        assert abs(lse[h] - (x.max() + math.log(l))) <= s + 2.0 ** -20 + 2.0 ** -21 * abs(lse[h])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("d,Hq", [(64, 1), (128, 2), (64, 12), (128, 24)])
@pytest.mark.parametrize("less,small", [(11.0, 0.4375), (12.0, 0.4375), (12.0, 0.875), (12.0, 3.5), (14.0, 0.001)])
def test_behind_a_block_of_large_values(cuda_lib, wide, d, Hq, less, small):
    """A token has nearly all of the weight and no value but a large one in one channel; the others
    have e^-less of it each and small values, which are the result of every other channel."""
    n = 200
    k, v = np.zeros((n, 1, d)), np.full((n, 1, d), small)
    k[0, 0, 0], v[0] = less, 0.0
    v[0, 0, 7] = 100.0
    q = np.zeros((Hq, d))
    q[:, 0] = 1.0
    check(*attend(k, v, q, torch.bfloat16, wide), torch.bfloat16)
    v[100, 0, 9] = 8000.0  # and another in their midst
    check(*attend(k, v, q, torch.bfloat16, wide), torch.bfloat16)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("d,Hq,Hk", [(64, 4, 2), (128, 10, 1), (128, 20, 1)])
def test_any_order_of_scales(cuda_lib, wide, d, Hq, Hk):
    """Blocks whose values differ by many powers of two, in any order, some of them with a large
    value in a channel of their own, and weights from 1 to e^-16."""
    rng = np.random.default_rng(d + Hq)
    n = 700
    k, v = rng.standard_normal((2, n, Hk, d))
    v *= 2.0 ** -rng.choice([0, 3, 6, 7, 8, 9, 12, 20], (-(-n // 16), Hk)).repeat(16, 0)[:n, :, None]
    for b in rng.choice(n // 16, 12, replace=False):
        v[16 * b + b % 16, :, b % d] = 200.0
    q = rng.standard_normal((Hq, d)) * 4 / math.sqrt(d)
    check(*attend(k, v, q, torch.bfloat16, wide), torch.bfloat16)
