"""Edges of the operators around the attention."""
import numpy as np
import pytest
import torch

import _ops_ref as ref
import exact_io_aware_26_gb300 as fa
from _parity import to_np64
from test_gpu_ops_kv4 import build, check, widened

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kv,new", [([3], [8]), ([3, 40, 0, 100], [8, 45, 3, 2]), ([1, 2, 3], [40, 30, 20])])
def test_a_window_beyond_every_length_hides_nothing(cuda_lib, kv, new, wide):
    """Also where a request has more rows than tokens: the first rows' positions lie before
    token 0, and position - window before -2^31."""
    q, cache, table, lens, cu = build(kv, new, 2, 1, 64, "bf16", 16, 31)
    want = ref.attention(to_np64(q), cache, table, lens, cu, 0.3, 0, 64)
    for window in (2 ** 31 - 1, 2 ** 31 - 4, 2 ** 31 - 40, 2 ** 30, 101):
        o, lse = fa.kv4_attention(q.cuda(), dev(cache), dev(widened(table) if wide else table), dev(lens), cu_q=dev(cu),
                                  max_q_len=max(new), scale=0.3, window=window)
        check(o, lse, want, "bf16")
    assert fa.get_status() == fa.FA_OK
