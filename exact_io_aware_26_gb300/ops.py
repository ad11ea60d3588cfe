"""The operators around the attention: norms and rotation of queries and keys, the
4-bit paged cache with the attention that reads it, and block tables from request
lengths.  Binding only, like the package's front: arguments are checked and turned
into the C ABI of ``include/fa.h``; the kernels do the rest.

Training, from a packed projection [B, N, Hq + 2 Hk, d] to the attention's layout:

    freqs = fa.rope_freqs(d)                                   # once
    q, k = fa.qk_norm_rope(qkv[:, :, :H], qkv[:, :, H:2*H], wq, wk, freqs)
    o, lse = fa.attention_fwd(q, k, v, causal=True)
    dq, dk, dv = fa.attention_bwd(q, k, v, o, do, lse, causal=True)
    dxq, dxk, dwq, dwk = fa.qk_norm_rope_bwd(qkv[:, :, :H], qkv[:, :, H:2*H], dq, dk, wq, wk, freqs)

Serving, one step of R requests:

    plan = fa.paged_plan(seq_lens, new_lens, block_table, free_pages, free_count, page_size, T)
    q, k = fa.qk_norm_rope(xq[None], xk[None], wq, wk, freqs, positions=plan["positions"][None], heads_first=False)
    fa.kv4_append(k[0], v, plan["slots"], cache)
    o, lse = fa.kv4_attention(q[0], cache, block_table, plan["kv_lens"], cu_q=plan["cu_q"])

Every tensor lies on the current device.  Results and workspaces are allocated on
``stream`` (default: the current one); inputs that another stream may free are marked
as used there.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional

import torch

from . import FA_BF16, FA_F16, FA_F32, _check, load

KV4_GROUP = 32    # channels that share a (scale, base) pair
KV4_BLOCK = 16    # tokens of a cache block
KV4_SATURATE = 16384.0
PLAN_MAX_REQUESTS = 8192

_CODES = {torch.float32: FA_F32, torch.float16: FA_F16, torch.bfloat16: FA_BF16}
_I64x2, _I64x3 = ctypes.c_longlong * 2, ctypes.c_longlong * 3


class FaQkParams(ctypes.Structure):
    """Mirror of ``fa_qk_params``."""
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("Hq", ctypes.c_int), ("Hk", ctypes.c_int),
                ("d", ctypes.c_int), ("dtype", ctypes.c_int), ("weight_dtype", ctypes.c_int),
                ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("eps", ctypes.c_float),
                ("pos_stride", ctypes.c_longlong), ("q_stride", _I64x3), ("k_stride", _I64x3),
                ("yq_stride", _I64x3), ("yk_stride", _I64x3), ("dq_stride", _I64x3), ("dk_stride", _I64x3)]


class FaKv4Cache(ctypes.Structure):
    """Mirror of ``fa_kv4_cache``."""
    _fields_ = [("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("Hk", ctypes.c_int), ("d", ctypes.c_int),
                ("page_stride", ctypes.c_longlong)]


class FaKv4Rows(ctypes.Structure):
    """Mirror of ``fa_kv4_rows``."""
    _fields_ = [("T", ctypes.c_int), ("dtype", ctypes.c_int), ("k_stride", _I64x2), ("v_stride", _I64x2)]


class FaKv4AttnParams(ctypes.Structure):
    """Mirror of ``fa_kv4_attn_params``."""
    _fields_ = [("R", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("dtype", ctypes.c_int),
                ("max_q_len", ctypes.c_int), ("window", ctypes.c_int), ("table_width", ctypes.c_int),
                ("scale", ctypes.c_float), ("table_stride", ctypes.c_longlong), ("q_stride", _I64x2),
                ("o_stride", _I64x2)]


class FaPlanParams(ctypes.Structure):
    """Mirror of ``fa_plan_params``."""
    _fields_ = [("R", ctypes.c_int), ("T", ctypes.c_int), ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("table_width", ctypes.c_int), ("table_stride", ctypes.c_longlong)]


def signatures() -> dict:
    """(result, arguments) of the C functions that this module calls."""
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


# ---------------------------------------------------------------- checks
# A call's checks and its C parameters depend on its arguments' sizes, strides, types and
# devices alone.  They are done once for each such signature; later calls with the same
# one look it up (a call on sixteen tokens takes the GPU a few microseconds: the checks
# would take longer).

_seen: dict = {}


def _remember(key, plan):
    if len(_seen) >= 4096:
        _seen.clear()
    _seen[key] = plan
    return plan


def _sig(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _need(t, name: str, dtype, shape=None):
    """t is a cuda tensor of the dtype and, with None for any, the shape."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a cuda tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None and (t.dim() != len(shape) or any(w is not None and w != g for w, g in zip(shape, t.shape))):
        raise ValueError(f"{name} must have shape {tuple('*' if w is None else w for w in shape)}, not {tuple(t.shape)}")


def _one_device(*tensors) -> torch.device:
    """The device of the tensors, which must be one."""
    devices = {t.device for t in tensors if t is not None}
    if len(devices) != 1:
        raise ValueError(f"every tensor must be on one device, not on {sorted(map(str, devices))}")
    return devices.pop()


def _contiguous(t, name: str):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _strides(t, name: str, dims) -> tuple:
    """Element strides of the dims (0 for one of at most one element); channels contiguous."""
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    shape, stride = t.shape, t.stride()
    return tuple(stride[i] if shape[i] > 1 else 0 for i in dims)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_HERE = contextlib.nullcontext()


def _enter(device, stream, *inputs):
    """(stream handle, context to allocate in): results and workspaces belong to the stream
    that the kernels run on, and inputs made on another one are marked as used there."""
    if torch.cuda.current_device() != device.index:
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{torch.cuda.current_device()}")
    current = _raw_stream(device.index)
    if stream is None:
        return current, _HERE
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    if stream.cuda_stream == current:
        return current, _HERE
    for t in inputs:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream, torch.cuda.stream(stream)


# ---------------------------------------------------------------- norms and rotation

def rope_freqs(rot_dim: int, base: float = 10000.0, inv_freq=None, device="cuda"):
    """The angle per position of each of the rot_dim / 2 pairs, in units of 2^-64 turns
    (int64, the bits of an unsigned number), as ``qk_norm_rope`` takes them:
    base ** (-2 i / rot_dim) radians, or ``inv_freq`` (radians per position)."""
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even and not negative")
    if inv_freq is None:
        inv_freq = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    else:
        inv_freq = [float(f) for f in (inv_freq.tolist() if hasattr(inv_freq, "tolist") else inv_freq)]
    if len(inv_freq) != rot_dim // 2 or not all(math.isfinite(f) for f in inv_freq):
        raise ValueError(f"inv_freq must be {rot_dim // 2} finite numbers")
    turns = [int(round(f / (2 * math.pi) * 2 ** 64)) % 2 ** 64 for f in inv_freq]
    return torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=device)


_BNH, _BHN = (0, 1, 2), (0, 2, 1)  # where batch, token and head stand in the two layouts


def _plan_qk(q, k, wq, wk, freqs, positions, eps, interleaved, heads_first, y, dx):
    """(C parameters, their address, device, shapes of q and k in the result's layout)."""
    dt = q.dtype
    if dt not in _CODES:
        raise TypeError(f"unsupported dtype {dt}")
    _need(q, "q", dt, (None, None, None, None))
    B, N, Hq, d = q.shape
    _need(k, "k", dt, (B, N, None, d))
    Hk, wt = k.shape[2], wq.dtype
    if wt != dt and wt != torch.float32:
        raise TypeError(f"the weights must be {dt} or torch.float32, not {wt}")
    for w, name in ((wq, "wq"), (wk, "wk")):
        _need(w, name, wt, (d,))
        _contiguous(w, name)
    _need(freqs, "freqs", torch.int64, (None,))
    _contiguous(freqs, "freqs")
    pos_stride = 0
    if positions is not None:
        _need(positions, "positions", torch.int32, (N,) if positions.dim() == 1 else (B, N))
        pos_stride = positions.stride(0) if positions.dim() == 2 and B > 1 else 0
        if N > 1 and positions.stride(-1) != 1:
            raise ValueError("positions must be contiguous in its last dimension")
    device = _one_device(q, k, wq, wk, freqs, positions, *y, *dx)
    names = ("dyq", "dyk") if dx else ("out[0]", "out[1]")
    ys, ds, shapes = [], [], []
    for i, h in enumerate((Hq, Hk)):
        shape = (B, h, N, d) if heads_first else (B, N, h, d)
        shapes.append(shape)
        if y[i] is None:  # a new tensor, contiguous
            st = (h * N * d, d if heads_first else h * d, N * d if heads_first else d)
            ys.append(tuple(s if size > 1 else 0 for s, size in zip(st, (B, N, h))))
        else:
            _need(y[i], names[i], dt, shape)
            ys.append(_strides(y[i], names[i], _BHN if heads_first else _BNH))
        if dx and dx[i] is not None:
            _need(dx[i], "dq" if i == 0 else "dk", dt, (B, N, h, d))
            ds.append(_strides(dx[i], "dq" if i == 0 else "dk", _BNH))
        else:
            ds.append(tuple(s if size > 1 else 0 for s, size in zip((N * h * d, h * d, d), (B, N, h))))
    p = FaQkParams(B, N, Hq, Hk, d, _CODES[dt], _CODES[wt], 2 * freqs.shape[0], int(bool(interleaved)), float(eps),
                   pos_stride, _I64x3(*_strides(q, "q", _BNH)), _I64x3(*_strides(k, "k", _BNH)), _I64x3(*ys[0]),
                   _I64x3(*ys[1]), _I64x3(*ds[0]), _I64x3(*ds[1]))
    ref = ctypes.byref(p)
    nbytes = int(load().fa_qk_norm_rope_bwd_workspace_size(ref)) if dx else 0
    return ref, device, shapes, nbytes


def qk_norm_rope(q, k, wq, wk, freqs, positions=None, eps: float = 1e-6, interleaved: bool = False,
                 heads_first: bool = True, out=None, stream=None):
    """(yq, yk): RMS norm of each head of q [B, N, Hq, d] and k [B, N, Hk, d] (any strides of
    whole 16-byte vectors, such as views of one packed projection), times wq, wk [d], then
    the rotation of the first 2 * len(freqs) channels by the positions (int32 [N] or
    [B, N]; None: 0 .. N - 1).  Results are [B, H, N, d] as ``attention_fwd`` takes them,
    or, with ``heads_first`` false, [B, N, H, d]; ``out`` (yq, yk) may be (q, k) there."""
    yq, yk = (None, None) if out is None else out
    key = ("qk", _sig(q), _sig(k), _sig(wq), _sig(wk), _sig(freqs), _sig(positions), _sig(yq), _sig(yk), eps,
           interleaved, heads_first)
    ref, device, shapes, _ = _seen.get(key) or _remember(
        key, _plan_qk(q, k, wq, wk, freqs, positions, eps, interleaved, heads_first, (yq, yk), ()))
    handle, alloc = _enter(device, stream, q, k, wq, wk, freqs, positions, yq, yk)
    if out is None:
        with alloc:
            yq = torch.empty(shapes[0], dtype=q.dtype, device=device)
            yk = torch.empty(shapes[1], dtype=q.dtype, device=device)
    _check(load().fa_qk_norm_rope(ref, q.data_ptr(), k.data_ptr(), wq.data_ptr(), wk.data_ptr(), freqs.data_ptr(),
                                  _ptr(positions), yq.data_ptr(), yk.data_ptr(), handle), "fa_qk_norm_rope")
    return yq, yk


def qk_norm_rope_bwd(q, k, dyq, dyk, wq, wk, freqs, positions=None, eps: float = 1e-6, interleaved: bool = False,
                     heads_first: bool = True, dq=None, dk=None, workspace=None, stream=None):
    """(dq, dk, dwq, dwk): gradients of ``qk_norm_rope`` for dyq, dyk at its results (in its
    layout); q and k are its inputs.  dq, dk are [B, N, H, d] in q's dtype (views of a
    packed gradient may be given), dwq, dwk fp32 [d]."""
    key = ("qk_bwd", _sig(q), _sig(k), _sig(dyq), _sig(dyk), _sig(wq), _sig(wk), _sig(freqs), _sig(positions),
           _sig(dq), _sig(dk), _sig(workspace), eps, interleaved, heads_first)
    plan = _seen.get(key)
    if plan is None:
        if workspace is not None:
            _need(workspace, "workspace", workspace.dtype)
            _contiguous(workspace, "workspace")
            _one_device(q, workspace)
        plan = _remember(key, _plan_qk(q, k, wq, wk, freqs, positions, eps, interleaved, heads_first, (dyq, dyk), (dq, dk)))
    ref, device, _, nbytes = plan
    handle, alloc = _enter(device, stream, q, k, dyq, dyk, wq, wk, freqs, positions, dq, dk, workspace)
    d = q.shape[3]
    with alloc:
        if dq is None:
            dq = torch.empty(q.shape, dtype=q.dtype, device=device)
        if dk is None:
            dk = torch.empty(k.shape, dtype=q.dtype, device=device)
        dwq = torch.empty(d, dtype=torch.float32, device=device)
        dwk = torch.empty(d, dtype=torch.float32, device=device)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _check(load().fa_qk_norm_rope_bwd(ref, q.data_ptr(), k.data_ptr(), dyq.data_ptr(), dyk.data_ptr(), wq.data_ptr(),
                                      wk.data_ptr(), freqs.data_ptr(), _ptr(positions), dq.data_ptr(), dk.data_ptr(),
                                      dwq.data_ptr(), dwk.data_ptr(), workspace.data_ptr(), workspace.nbytes, handle),
           "fa_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------- the 4-bit cache

def kv4_block_bytes(d: int) -> int:
    """Bytes of a 16-token block of one head (``fa_kv4_block_bytes``)."""
    return int(load().fa_kv4_block_bytes(int(d)))


def kv4_cache(num_pages: int, heads: int, d: int, page_size: int = 64, device="cuda"):
    """A zeroed cache: uint8 [num_pages, heads, page_size / 16, kv4_block_bytes(d)]."""
    if d not in (64, 128):
        raise ValueError("head size must be 64 or 128")
    if page_size < 16 or page_size > 4096 or page_size & (page_size - 1):
        raise ValueError("page_size must be a power of two from 16 to 4096")
    return torch.zeros((num_pages, heads, page_size // KV4_BLOCK, kv4_block_bytes(d)), dtype=torch.uint8, device=device)


def _cache_params(cache, d: int) -> FaKv4Cache:
    _need(cache, "cache", torch.uint8, (None, None, None, {64: 1280, 128: 2560}.get(d, -1)))
    P, H, n, b = cache.shape
    s = cache.stride()
    if s[3] != 1 or (n > 1 and s[2] != b) or (H > 1 and s[1] != n * b):
        raise ValueError("cache must be contiguous within a page")
    return FaKv4Cache(P, KV4_BLOCK * n, H, d, s[0] if P > 1 else H * n * b)


def _plan_rows(cache, slots, k, v, T, H, d, dtype, dims, names):
    """(cache parameters, row parameters, device)."""
    c = _cache_params(cache, d)
    if cache.shape[1] != H:
        raise ValueError(f"{names[0]} has {H} heads, the cache {cache.shape[1]}")
    _need(slots, "slots", torch.int32, (T,))
    _contiguous(slots, "slots")
    strides = []
    for x, name in zip((k, v), names):
        if x is None:  # new and contiguous
            strides.append(tuple(st if size > 1 else 0 for st, size in zip((H * d, d) if dims == (0, 1) else (d, T * d), (T, H))))
        else:
            _need(x, name, dtype, (T, H, d) if dims == (0, 1) else (H, T, d))
            strides.append(_strides(x, name, dims))
    device = _one_device(cache, slots, k, v)
    rows = FaKv4Rows(T, _CODES[dtype], _I64x2(*strides[0]), _I64x2(*strides[1]))
    return ctypes.byref(c), ctypes.byref(rows), device


def kv4_append(k, v, slots, cache, stream=None) -> None:
    """Quantise the keys and values [T, Hk, d] of T tokens into their slots (int32 [T];
    negative: left out; distinct otherwise) of the cache.  Values saturate at +-16384."""
    key = ("append", _sig(k), _sig(v), _sig(slots), _sig(cache))
    plan = _seen.get(key)
    if plan is None:
        if k.dtype not in _CODES:
            raise TypeError(f"unsupported dtype {k.dtype}")
        _need(k, "k", k.dtype, (None, None, None))
        T, H, d = k.shape
        plan = _remember(key, _plan_rows(cache, slots, k, v, T, H, d, k.dtype, (0, 1), ("k", "v")))
    c, rows, device = plan
    handle, _ = _enter(device, stream, k, v, slots, cache)
    _check(load().fa_kv4_append(c, rows, k.data_ptr(), v.data_ptr(), slots.data_ptr(), cache.data_ptr(), handle),
           "fa_kv4_append")


def kv4_gather(cache, slots, d: int, dtype=torch.bfloat16, heads_first: bool = False, out=None, stream=None):
    """(k, v): the cached keys and values of T slots (zeros for a negative one), rounded to
    ``dtype``: [T, Hk, d], or, ``heads_first``, [Hk, T, d] (with a leading batch of one,
    as ``attention_fwd`` takes them)."""
    k, v = (None, None) if out is None else out
    key = ("gather", _sig(cache), _sig(slots), d, dtype, heads_first, _sig(k), _sig(v))
    plan = _seen.get(key)
    if plan is None:
        if dtype not in _CODES:
            raise TypeError(f"unsupported dtype {dtype}")
        _need(cache, "cache", torch.uint8, (None, None, None, None))
        _need(slots, "slots", torch.int32, (None,))
        plan = _remember(key, _plan_rows(cache, slots, k, v, slots.shape[0], cache.shape[1], d, dtype,
                                         (1, 0) if heads_first else (0, 1), ("out[0]", "out[1]")))
    c, rows, device = plan
    handle, alloc = _enter(device, stream, slots, cache, k, v)
    if out is None:
        T, H = slots.shape[0], cache.shape[1]
        shape = (H, T, d) if heads_first else (T, H, d)
        with alloc:
            k = torch.empty(shape, dtype=dtype, device=device)
            v = torch.empty(shape, dtype=dtype, device=device)
    _check(load().fa_kv4_gather(c, rows, cache.data_ptr(), slots.data_ptr(), k.data_ptr(), v.data_ptr(), handle),
           "fa_kv4_gather")
    return k, v


def _plan_attention(q, cache, block_table, kv_lens, cu_q, max_q_len, scale, window, out, lse, workspace):
    """(cache parameters, parameters, workspace bytes, device)."""
    if q.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"q must be fp16 or bf16, not {q.dtype}")
    _need(q, "q", q.dtype, (None, None, None))
    T, Hq, d = q.shape
    c = _cache_params(cache, d)
    _need(block_table, "block_table", torch.int32, (None, None))
    R, width = block_table.shape
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table must be contiguous in its last dimension")
    _need(kv_lens, "kv_lens", torch.int32, (R,))
    _contiguous(kv_lens, "kv_lens")
    if cu_q is not None:
        _need(cu_q, "cu_q", torch.int32, (R + 1,))
        _contiguous(cu_q, "cu_q")
    elif T < R:
        raise ValueError(f"q has {T} rows for {R} requests")
    o_stride = tuple(st if size > 1 else 0 for st, size in zip((Hq * d, d), (T, Hq)))
    if out is not None:
        _need(out, "out", q.dtype, (T, Hq, d))
        o_stride = _strides(out, "out", (0, 1))
    if lse is not None:
        _need(lse, "lse", torch.float32, (T, Hq))
        _contiguous(lse, "lse")
    if workspace is not None:
        _need(workspace, "workspace", workspace.dtype)
        _contiguous(workspace, "workspace")
    device = _one_device(q, cache, block_table, kv_lens, cu_q, out, lse, workspace)
    p = FaKv4AttnParams(R, T, Hq, _CODES[q.dtype], int(max_q_len), int(window), width,
                        1.0 / math.sqrt(d) if scale is None else float(scale),
                        block_table.stride(0) if R > 1 else width, _I64x2(*_strides(q, "q", (0, 1))), _I64x2(*o_stride))
    cref, ref = ctypes.byref(c), ctypes.byref(p)
    return cref, ref, int(load().fa_kv4_attention_workspace_size(cref, ref)), device


def kv4_attention(q, cache, block_table, kv_lens, cu_q=None, max_q_len: int = 1, scale: Optional[float] = None,
                  window: int = 0, out=None, lse=None, workspace=None, stream=None):
    """(o, lse): attention of each request's newest tokens, q [T, Hq, d], over its cached
    tokens.  Request r has kv_lens[r] tokens (these queries' own among them) in the pages
    block_table[r]; its queries are rows cu_q[r] : cu_q[r + 1] (None: row r), the last of
    them at its last token; each sees the tokens up to its own, and with ``window`` > 0
    only the last ``window`` of those.  Rows without a token to see: o = 0, lse = -inf;
    rows outside every request are not written.  ``max_q_len``: the most rows of a request,
    a hint.  Lengths stay on the GPU: the call does not synchronise."""
    key = ("attention", _sig(q), _sig(cache), _sig(block_table), _sig(kv_lens), _sig(cu_q), max_q_len, scale, window,
           _sig(out), _sig(lse), _sig(workspace))
    c, p, nbytes, device = _seen.get(key) or _remember(
        key, _plan_attention(q, cache, block_table, kv_lens, cu_q, max_q_len, scale, window, out, lse, workspace))
    handle, alloc = _enter(device, stream, q, cache, block_table, kv_lens, cu_q, out, lse, workspace)
    with alloc:
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=device)
        if lse is None:
            lse = torch.empty(q.shape[:2], dtype=torch.float32, device=device)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _check(load().fa_kv4_attention(c, p, q.data_ptr(), cache.data_ptr(), block_table.data_ptr(), kv_lens.data_ptr(),
                                   _ptr(cu_q), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.nbytes,
                                   handle), "fa_kv4_attention")
    return out, lse


# ---------------------------------------------------------------- block tables and slot maps

_PLAN_OUT = ("kv_lens", "cu_q", "positions", "slots", "counts")


def _plan_plan(seq_lens, new_lens, block_table, free_pages, free_count, page_size, T, out):
    """(parameters, sizes of the results, device)."""
    i32 = torch.int32
    _need(block_table, "block_table", i32, (None, None))
    R, width = block_table.shape
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table must be contiguous in its last dimension")
    for t, name, n in ((seq_lens, "seq_lens", R), (new_lens, "new_lens", R), (free_pages, "free_pages", None),
                       (free_count, "free_count", None)):
        _need(t, name, i32, (n,))
        _contiguous(t, name)
    if free_count.shape[0] < 1:
        raise ValueError("free_count is empty")
    sizes = [R, R + 1, int(T), int(T), 3]
    if out is not None:
        for name, n in zip(_PLAN_OUT, sizes):
            _need(out[name], f"out[{name!r}]", i32, (n,))
            _contiguous(out[name], f"out[{name!r}]")
    device = _one_device(seq_lens, new_lens, block_table, free_pages, free_count, *(out[n] for n in _PLAN_OUT if out))
    p = FaPlanParams(R, int(T), int(page_size), free_pages.shape[0], width, block_table.stride(0) if R > 1 else width)
    return ctypes.byref(p), sizes, device


def paged_plan(seq_lens, new_lens, block_table, free_pages, free_count, page_size: int, T: int, out=None, stream=None):
    """One step's block tables and slot maps, from request lengths (``fa_paged_plan``; int32
    device tensors).  Request r holds seq_lens[r] tokens and gets new_lens[r] more (< 0: it
    has ended and its pages go back).  block_table [R, width] and the stack
    free_pages[: free_count] are updated in place.  Returns, or fills ``out`` with,
    kv_lens [R], cu_q [R + 1], positions [T], slots [T] and counts [3] (pages left, new
    tokens, pages missing).  A request whose pages are not there keeps its length and gets
    slots of -1.  out["kv_lens"] may be seq_lens, and out["counts"] the tensor whose first
    element is free_count."""
    given = () if out is None else tuple(out[name] for name in _PLAN_OUT)
    key = ("plan", _sig(seq_lens), _sig(new_lens), _sig(block_table), _sig(free_pages), _sig(free_count), page_size, T,
           *map(_sig, given))
    p, sizes, device = _seen.get(key) or _remember(
        key, _plan_plan(seq_lens, new_lens, block_table, free_pages, free_count, page_size, T, out))
    handle, alloc = _enter(device, stream, seq_lens, new_lens, block_table, free_pages, free_count, *given)
    if out is None:
        with alloc:
            given = [torch.empty(n, dtype=torch.int32, device=device) for n in sizes]
        out = dict(zip(_PLAN_OUT, given))
    kv, cu, pos, slots, counts = given
    _check(load().fa_paged_plan(p, seq_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(),
                                free_pages.data_ptr(), free_count.data_ptr(), kv.data_ptr(), cu.data_ptr(),
                                pos.data_ptr(), slots.data_ptr(), counts.data_ptr(), handle), "fa_paged_plan")
    return out
