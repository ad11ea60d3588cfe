"""Pieces of prompts over what the 8-bit cache holds, with the slots of whole requests made on the GPU from
their lengths and the block table, as the README has it; captured, and replayed for other lengths of the
same sum."""
import pytest
import torch

import _packed_ref
import exact_io_aware_26_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,Hq,Hk,page", [(64, 4, 2, 16), (128, 10, 2, 64)])
def test_pieces_over_the_cache(cuda_lib, d, Hq, Hk, page):
    held, new, R = [[200, 0, 35, 61], [9, 130, 140, 17]], [5, 40, 1, 30], 4
    total, T = sum(held[0]) + sum(new), sum(new)
    assert sum(held[1]) + sum(new) == total
    pages, width = 60, 20
    g = torch.Generator().manual_seed(d)
    table = torch.randperm(R * width, generator=g).view(R, width).int().cuda() % pages  # shared pages: what they hold is the test's
    cache = fa.kv8_cache(pages, Hk, d, page)
    x = torch.randn(pages * page, 2 * Hk, d, generator=g).bfloat16().cuda()
    fa.kv8_append(x[:, :Hk], x[:, Hk:], torch.arange(pages * page, dtype=torch.int32, device="cuda"), cache)
    q = torch.randn(T, Hq, d, generator=g).bfloat16().cuda()
    cu_q = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).int().cuda()
    kv_lens = torch.tensor([h + n for h, n in zip(held[0], new)], dtype=torch.int32, device="cuda")

    def call():
        lens = kv_lens.long()
        cu_k = torch.nn.functional.pad(lens.cumsum(0), (1, 0))
        r = torch.repeat_interleave(lens, output_size=total)
        t = torch.arange(total, device="cuda") - cu_k[r]
        all_slots = (table[r, t // page] * page + t % page).int()
        k16, v16 = fa.kv8_gather(cache, all_slots, d)
        return (k16, v16) + fa.attention_fwd_packed(q, k16, v16, cu_q, cu_k.int())

    got = [call()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = call()
    for h in held:
        lens = [a + b for a, b in zip(h, new)]
        kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        slots = torch.cat([table[r, torch.arange(n, device="cuda") // page] * page + torch.arange(n, device="cuda") % page for r, n in enumerate(lens)])
        wk, wv = fa.kv8_gather(cache, slots.int(), d)
        assert torch.equal(captured[0], wk) and torch.equal(captured[1], wv)
        want = _packed_ref.forward(q.cpu(), wk.cpu(), wv.cpu(), new, lens, True, d ** -0.5, 2.0 ** -8, 0.0)
        for o, lse in [captured[2:]] + [w[2:] for w in got]:
            assert bool(((o.double().cpu() - want[0]).abs() <= want[2]).all()) and bool(((lse.double().cpu() - want[1]).abs() <= want[3]).all())
        got = []
    assert fa.get_status() == fa.FA_OK
