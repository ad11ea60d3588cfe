"""The C structs and functions of the operators around the attention, for ctypes.  Apart
from the binding (``ops.py``), so that the library loads without torch and the extension
that repeats the binding's calls."""
from __future__ import annotations

import ctypes

I64x2, I64x3 = ctypes.c_longlong * 2, ctypes.c_longlong * 3


class _Params(ctypes.Structure):
    """A struct that refuses numbers its C ints do not hold (ctypes would keep their low bits,
    and the call be made with another size)."""

    def __init__(self, *args, **kw):
        given = {**dict(zip((name for name, _ in self._fields_), args)), **kw}
        for name, kind in self._fields_:
            if kind is ctypes.c_int and not -2 ** 31 <= given.get(name, 0) < 2 ** 31:
                raise ValueError(f"{name} = {given[name]} is beyond 32 bits")
        super().__init__(*args, **kw)


class FaQkParams(_Params):
    """Mirror of ``fa_qk_params``."""
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("Hq", ctypes.c_int), ("Hk", ctypes.c_int),
                ("d", ctypes.c_int), ("dtype", ctypes.c_int), ("weight_dtype", ctypes.c_int),
                ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("eps", ctypes.c_float),
                ("pos_stride", ctypes.c_longlong), ("q_stride", I64x3), ("k_stride", I64x3),
                ("yq_stride", I64x3), ("yk_stride", I64x3), ("dq_stride", I64x3), ("dk_stride", I64x3)]


class FaKv4Cache(_Params):
    """Mirror of ``fa_kv4_cache``."""
    _fields_ = [("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("Hk", ctypes.c_int), ("d", ctypes.c_int),
                ("page_stride", ctypes.c_longlong)]


class FaKv4Rows(_Params):
    """Mirror of ``fa_kv4_rows``."""
    _fields_ = [("T", ctypes.c_int), ("dtype", ctypes.c_int), ("k_stride", I64x2), ("v_stride", I64x2)]


class FaKv4AttnParams(_Params):
    """Mirror of ``fa_kv4_attn_params``."""
    _fields_ = [("R", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("dtype", ctypes.c_int),
                ("max_q_len", ctypes.c_int), ("window", ctypes.c_int), ("table_width", ctypes.c_int),
                ("scale", ctypes.c_float), ("table_stride", ctypes.c_longlong), ("q_stride", I64x2),
                ("o_stride", I64x2)]


class FaPlanParams(_Params):
    """Mirror of ``fa_plan_params``."""
    _fields_ = [("R", ctypes.c_int), ("T", ctypes.c_int), ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("table_width", ctypes.c_int), ("table_stride", ctypes.c_longlong)]


def signatures() -> dict:
    """(result, arguments) of the C functions of the operators."""
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    QP, CP, RP, AP, PP = (ctypes.POINTER(t) for t in (FaQkParams, FaKv4Cache, FaKv4Rows, FaKv4AttnParams, FaPlanParams))
    return {
        "fa_qk_norm_rope": (I, [QP] + [P] * 9),
        "fa_qk_norm_rope_bwd_workspace_size": (S, [QP]),
        "fa_qk_norm_rope_bwd": (I, [QP] + [P] * 13 + [S, P]),
        "fa_kv4_block_bytes": (I, [I]),
        "fa_kv4_append": (I, [CP, RP] + [P] * 5),
        "fa_kv4_gather": (I, [CP, RP] + [P] * 5),
        "fa_kv4_attention_workspace_size": (S, [CP, AP]),
        "fa_kv4_attention": (I, [CP, AP] + [P] * 8 + [S, P]),
        "fa_paged_plan": (I, [PP] + [P] * 11),
    }
