"""The debug build's checks over packed attention and the 8-bit cache: each passes (status FA_OK), and
the results are the release build's, bit for bit (dq, a sum in any order, within two roundings)."""
import pytest
import torch

import exact_io_aware_26_gb300 as fa

pytestmark = pytest.mark.gpu


def both(run):
    """What `run` gives with the release build and with the debug build."""
    got = []
    old = None
    try:
        for debug in (False, True):
            path = fa.build(debug=debug)
            before = fa.use_library(path)
            old = before if old is None else old
            got.append(run())
            torch.cuda.synchronize()
            assert fa.get_status() == fa.FA_OK
    finally:
        fa.use_library(old)
        fa.load()
    return got


def offsets(lengths):
    return torch.tensor([0] + lengths, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


@pytest.mark.parametrize("new,keys,Hq,Hk,d,causal", [
    ([3, 0, 17], [3, 5, 17], 4, 2, 64, True),            # without a work list
    ([200, 1, 31], [200, 900, 3], 6, 2, 128, True),
    ([40], [5000], 8, 1, 64, False),                     # cut
    ([150] * 30, [150] * 30, 64, 64, 64, True),          # sequence by sequence
])
def test_packed_attention(cuda_lib, new, keys, Hq, Hk, d, causal):
    g = torch.Generator().manual_seed(sum(new))
    q, do = (torch.randn(sum(new), Hq, d, generator=g).bfloat16().cuda() for _ in range(2))
    k, v = (torch.randn(sum(keys), Hk, d, generator=g).bfloat16().cuda() for _ in range(2))
    cu_q, cu_k = offsets(new), offsets(keys)

    def run():
        o, lse = fa.attention_fwd_packed(q, k, v, cu_q, cu_k, causal=causal)
        return (o, lse) + fa.attention_bwd_packed(q, k, v, o, do, lse, cu_q, cu_k, causal=causal)

    release, debug = both(run)
    for i, (a, b) in enumerate(zip(release, debug)):
        if i == 2:
            assert bool(((a.float() - b.float()).abs() <= 2 ** -7 * a.float().abs() + 1e-5).all())
        else:
            assert torch.equal(a, b)


@pytest.mark.parametrize("d,Hq,Hk,page,rows", [(64, 4, 2, 16, 1), (128, 8, 1, 64, 1), (64, 40, 2, 64, 5)])
def test_8_bit_cache(cuda_lib, d, Hq, Hk, page, rows):
    lens = [1, 300, 77]
    g = torch.Generator().manual_seed(d + rows)
    width = -(-max(lens) // page)
    table = torch.randperm(3 * width, generator=g).view(3, width).to(torch.int32)
    slots = torch.cat([table[r].long()[torch.arange(n) // page] * page + torch.arange(n) % page for r, n in enumerate(lens)])
    slots = slots.to(torch.int32).cuda()
    k, v = (torch.randn(sum(lens), Hk, d, generator=g).half().cuda() for _ in range(2))
    q = torch.randn(3 * rows, Hq, d, generator=g).half().cuda()
    lengths = torch.tensor([n + rows - 1 for n in lens], dtype=torch.int32).clamp(max=width * page).cuda()

    def run():
        cache = fa.kv8_cache(3 * width, Hk, d, page)
        fa.kv8_append(k, v, slots, cache)
        back = fa.kv8_gather(cache, slots, d, dtype=torch.float16)
        return (cache, *back, *fa.kv8_attention(q, cache, table.cuda(), lengths, cu_q=offsets([rows] * 3), max_q_len=rows))

    release, debug = both(run)
    assert all(torch.equal(a, b) for a, b in zip(release, debug))
