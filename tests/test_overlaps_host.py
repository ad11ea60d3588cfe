"""Results over inputs or over each other: what the entries of packed attention and of the caches' attention
refuse before any CUDA call, and what they let through (which ends at the device that is not
there, or, with a GPU in the machine, is not called)."""
import ctypes
import itertools

import pytest
import torch

import exact_io_aware_26_gb300 as fa

L2 = ctypes.c_longlong * 2
BASE, E = 1 << 30, 2  # an aligned address that is never dereferenced; bytes of an element


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.load()


class View:
    """A tensor [T, H, d] at an element offset, by its strides."""

    def __init__(self, at, T, H, d, token, head, e=E):
        self.at, self.T, self.H, self.d, self.token, self.head, self.e = at, T, H, d, token, head, e

    def places(self):
        """Its bytes."""
        return {(self.at + t * self.token + h * self.head + c) * self.e + b
                for t in range(self.T) for h in range(self.H) for c in range(0, self.d, 8) for b in range(0, 8 * self.e, 8)}


def far(i, T, H, d):
    return View((i + 1) << 24, T, H, d, H * d, d)


def address(v):
    return BASE + v.at * v.e


def packed_call(lib, views, bwd, lse=None):
    q, k = views["q"], views["k"]
    p = fa.FaPackedParams(R=1, Tq=q.T, Tk=k.T, Hq=q.H, Hk=k.H, d=q.d, dtype=fa.FA_BF16, causal=1, scale=0.1,
                          **{n + "_stride": L2(v.token, v.head) for n, v in views.items()})
    at = {n: address(v) for n, v in views.items()}
    cu, ws = BASE + (200 << 24), BASE + (220 << 24)
    lse = BASE + (210 << 24) if lse is None else lse
    r = ctypes.byref(p)
    if bwd:
        return lib.fa_bwd_packed(r, at["q"], at["k"], at["v"], at["o"], at["do"], lse, cu, cu, at["dq"], at["dk"], at["dv"], ws, 1 << 40, None)
    return lib.fa_fwd_packed(r, at["q"], at["k"], at["v"], cu, cu, at["o"], lse, ws, 1 << 40, None)


NAMES = ("q", "k", "v", "o", "do", "dq", "dk", "dv")
T, HQ, HK, D = 6, 4, 2, 64


def apart_views():
    return {n: far(i, T, HK if n in ("k", "v", "dk", "dv") else HQ, D) for i, n in enumerate(NAMES)}


def over(name, at, token=None, head=None):
    """A view of the name's sizes at an element offset."""
    H = HK if name in ("k", "v", "dk", "dv") else HQ
    return View(at, T, H, D, token or H * D, head or D)


ROW = (HQ + 2 * HK) * D  # of a packed projection
LAYOUTS = [  # (offsets of q, k, v in elements, token stride, head stride): views of one buffer
    ((0, HQ * D, (HQ + HK) * D), ROW, D),              # [T, Hq + 2 Hk, d]
    ((0, HQ * T * D, (HQ + HK) * T * D), D, T * D),    # heads before tokens
]


@pytest.mark.skipif(torch.cuda.is_available(), reason="lets calls through to the device")
def test_what_is_apart_is_let_through(lib):
    for bwd in (False, True):
        assert packed_call(lib, apart_views(), bwd) == fa.FA_ERR_CUDA
    for (a, b, c), token, head in LAYOUTS:
        views = apart_views()
        views.update(q=View(a, T, HQ, D, token, head), k=View(b, T, HK, D, token, head), v=View(c, T, HK, D, token, head))
        assert packed_call(lib, views, False) == fa.FA_ERR_CUDA
        # gradients in one buffer of the same kind; dq over its query, o over do is nobody's business
        far_off = 100 << 24
        views.update(dq=View(far_off + a, T, HQ, D, token, head), dk=View(far_off + b, T, HK, D, token, head), dv=View(far_off + c, T, HK, D, token, head))
        assert packed_call(lib, views, True) == fa.FA_ERR_CUDA
        views["dq"] = views["q"]
        assert packed_call(lib, views, True) == fa.FA_ERR_CUDA
    # a result in the free heads of the inputs' rows; heads that take turns within a token; tokens that do
    views = apart_views()
    row = ROW + HQ * D
    views.update(q=View(0, T, HQ, D, row, D), k=View(HQ * D, T, HK, D, row, D), v=View((HQ + HK) * D, T, HK, D, row, D),
                 o=View(ROW, T, HQ, D, row, D))
    assert packed_call(lib, views, False) == fa.FA_ERR_CUDA
    views = apart_views()
    views.update(q=View(0, T, HQ, D, HQ * 3 * D, 3 * D), o=View(2 * D, T, HQ, D, HQ * 3 * D, 3 * D))
    assert packed_call(lib, views, False) == fa.FA_ERR_CUDA
    views.update(q=View(0, T, HQ, D, 2 * HQ * D, D), o=View(HQ * D, T, HQ, D, 2 * HQ * D, D))
    assert packed_call(lib, views, False) == fa.FA_ERR_CUDA
    views.update(q=View(HQ * D * T, T, HQ, D, HQ * D, D), o=View(0, T, HQ, D, HQ * D, D))  # one ends where the other begins
    assert packed_call(lib, views, False) == fa.FA_ERR_CUDA


@pytest.mark.parametrize("shift", [0, 8, D, HK * D, (T - 1) * HQ * D, -8, -HK * D])
def test_o_over_an_input(lib, shift):
    """At any distance: a vector, a head, a row, the last row."""
    for name in ("q", "k", "v"):
        views = apart_views()
        views["o"] = over("o", views[name].at + shift)
        if not views["o"].places() & views[name].places():
            continue
        assert packed_call(lib, views, False) == fa.FA_ERR_INVALID and b"o lies over" in lib.fa_last_error()


def test_o_in_the_inputs_heads(lib):
    """out=packed[:, 2:10] with q, k and v in `packed`."""
    (a, b, c), token, head = LAYOUTS[0]
    for at in range(0, ROW - HQ * D + 1, D):
        views = apart_views()
        views.update(q=View(a, T, HQ, D, token, head), k=View(b, T, HK, D, token, head), v=View(c, T, HK, D, token, head),
                     o=View(at, T, HQ, D, token, head))
        assert packed_call(lib, views, False) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("result,other", [(r, o) for r in ("dk", "dv") for o in ("q", "k", "v", "do")] +
                         [("dk", "dv"), ("dq", "dk"), ("dq", "dv")])
@pytest.mark.parametrize("shift", [0, 8, D, HK * D, (T - 1) * HK * D, -8])
def test_gradients_over_inputs_and_each_other(lib, result, other, shift):
    views = apart_views()
    views[result] = over(result, views[other].at + shift)
    if not views[result].places() & views[other].places():
        pytest.skip("apart")
    assert packed_call(lib, views, True) == fa.FA_ERR_INVALID and b"over" in lib.fa_last_error()


def test_lse_over_inputs_and_o(lib):
    for name in ("q", "k", "v", "o"):
        views = apart_views()
        for shift in (0, 4, -4, 64):
            assert packed_call(lib, views, False, lse=address(views[name]) + shift) == fa.FA_ERR_INVALID


def test_every_pair_of_small_layouts(lib):
    """What shares a byte is always refused."""
    strides = [(HQ * D, D), (D, T * D), (2 * HQ * D, D), (3 * HQ * D, 3 * D), (HQ * D + 8, D), (D + 8, T * (D + 8))]
    hit = 0
    for (qt, qh), (ot, oh), shift in itertools.product(strides, strides, [0, 8, D - 8, D, 3 * D, 5 * D + 8, HQ * D, 40 * D]):
        views = apart_views()
        views["q"], views["o"] = View(1 << 20, T, HQ, D, qt, qh), View((1 << 20) + shift, T, HQ, D, ot, oh)
        if views["q"].places() & views["o"].places():
            hit += 1
            assert packed_call(lib, views, False) == fa.FA_ERR_INVALID
    assert hit > 100


@pytest.mark.parametrize("bits", [4, 8])
def test_cache_attention(lib, bits):
    block = {4: 1280, 8: 2064}[bits]
    c = fa.FaKv4Cache(num_pages=10, page_size=64, Hk=2, d=64, page_stride=2 * 4 * block)
    entry = lib.fa_kv4_attention if bits == 4 else lib.fa_kv8_attention

    def call(q, o, lse):
        p = fa.FaKv4AttnParams(R=T, T=T, Hq=HQ, dtype=fa.FA_BF16, max_q_len=1, window=0, table_width=5, scale=0.1, table_stride=5,
                               q_stride=L2(q.token, q.head), o_stride=L2(o.token, o.head))
        other = [BASE + ((150 + i) << 24) for i in range(4)]
        return entry(ctypes.byref(c), ctypes.byref(p), address(q), other[0], other[1], other[2], None, address(o), lse,
                     other[3], 1 << 40, None)

    q, free = far(0, T, HQ, D), BASE + (140 << 24)
    for shift in (0, 8, D, HQ * D, -HQ * D):
        assert call(q, View(q.at + shift, T, HQ, D, HQ * D, D), free) == fa.FA_ERR_INVALID
    for shift in (0, 4, -4):
        assert call(q, far(1, T, HQ, D), address(q) + shift) == fa.FA_ERR_INVALID
        assert call(q, far(1, T, HQ, D), address(far(1, T, HQ, D)) + shift) == fa.FA_ERR_INVALID
    if not torch.cuda.is_available():
        row = 2 * HQ * D
        for o in (far(1, T, HQ, D), View(q.at + HQ * D, T, HQ, D, row, D)):
            assert call(q if o.token != row else View(q.at, T, HQ, D, row, D), o, free) == fa.FA_ERR_CUDA
            assert call(q if o.token != row else View(q.at, T, HQ, D, row, D), o, None) == fa.FA_ERR_CUDA
