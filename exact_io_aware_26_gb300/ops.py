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
as used there.  New results of up to 1 MB share a block of memory.
"""
from __future__ import annotations

import ctypes
import importlib
import math
from typing import Optional

import torch

from . import FA_BF16, FA_F16, FA_F32, _check, load
from ._abi import I64x2, I64x3, FaKv4AttnParams, FaKv4Cache, FaKv4Rows, FaPlanParams, FaQkParams

KV4_GROUP = 32    # channels that share a (scale, base) pair
KV4_BLOCK = 16    # tokens of a cache block
KV4_SATURATE = 16384.0
PLAN_MAX_REQUESTS = 8192

_CODES = {torch.float32: FA_F32, torch.float16: FA_F16, torch.bfloat16: FA_BF16}


# ---------------------------------------------------------------- checks and calls
# A call's checks and its C parameters depend on its arguments' sizes, strides, types and
# device alone.  They are done once for each such combination, which is then registered
# with the extension (csrc/launch.cpp) that repeats the call: a call on sixteen tokens
# takes the GPU a few microseconds, the checks would take several times that.

_QK, _QK_BWD, _APPEND, _GATHER, _ATTENTION, _PLAN = range(6)
_ENTRY = ("fa_qk_norm_rope", "fa_qk_norm_rope_bwd", "fa_kv4_append", "fa_kv4_gather", "fa_kv4_attention", "fa_paged_plan")
_STREAM = (3, 0)
_launch = None  # the extension, from the first call on


def _extension():
    global _launch
    try:
        _launch = importlib.import_module("._launch", __package__)
    except ImportError as e:
        raise ImportError(f"_launch.so is missing or does not load ({e}): run exact_io_aware_26_gb300.build() first") from e
    return _launch


def _in(i: int) -> tuple:
    return 0, i


def _const(value) -> tuple:
    """A number, or the address of a C struct."""
    return 2, ctypes.addressof(value) if isinstance(value, ctypes.Structure) else int(value)


class _Outputs(list):
    """The (sizes, dtype) of the tensors that a call allocates."""

    def new(self, sizes, dtype) -> tuple:
        self.append((tuple(int(n) for n in sizes), dtype))
        return 1, len(self) - 1

    def given(self, i: int, t, sizes, dtype) -> tuple:
        """Argument i where it is given, else a new tensor."""
        return self.new(sizes, dtype) if t is None else _in(i)


def _call(op: int, tensors: tuple, scalars: tuple, stream, plan):
    """Run an entry point: ``plan(*tensors, *scalars)``, once for each combination of sizes,
    strides, types and scalars, checks them and gives (device, arguments, outputs, results,
    what to keep alive).  Results and workspaces are allocated on the stream that the
    kernels run on, and inputs made on another one are marked as used there."""
    if stream is not None:
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
        if stream.cuda_stream != torch.cuda.current_stream().cuda_stream:
            for t in tensors:
                if isinstance(t, torch.Tensor) and t.is_cuda:
                    t.record_stream(stream)
            with torch.cuda.stream(stream):
                return _call(op, tensors, scalars, None, plan)
    launch = _launch or _extension()
    got = launch.run(op, tensors, scalars)
    while got is None:  # again where another thread empties the table before this one's plan has run
        device, args, outputs, results, keep = plan(*tensors, *scalars)
        entry = ctypes.cast(getattr(load(), _ENTRY[op]), ctypes.c_void_p).value
        launch.register(op, tensors, scalars, entry, device.index, args, outputs, results, keep)
        got = launch.run(op, tensors, scalars)
    if type(got) is int:
        _check(got, _ENTRY[op])
    return got


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


def _dense(sizes, strides) -> tuple:
    """Strides of a new tensor, 0 for a dimension of at most one element."""
    return tuple(st if n > 1 else 0 for st, n in zip(strides, sizes))


def _workspace(new: _Outputs, i: int, given, nbytes: int, device) -> tuple:
    """(where the workspace comes from, its bytes); 0 bytes wanted is a refusal of the
    parameters, which the call itself will put in words."""
    if given is None:
        return new.new((max(int(nbytes), 1),), torch.uint8), int(nbytes)
    _need(given, "workspace", given.dtype)
    _contiguous(given, "workspace")
    _one_device(given, torch.empty(0, device=device))
    return _in(i), given.numel() * given.element_size()


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


def _qk_checked(q, k, wq, wk, freqs, positions, eps, interleaved, heads_first, y, dx, names):
    """(C parameters, device, shapes in the result's layout) of a call; y: the results or
    their gradients, dx: the gradients to write, None for one that is still to be made."""
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
    ys, ds, shapes = [], [], []
    for i, h in enumerate((Hq, Hk)):
        shapes.append((B, h, N, d) if heads_first else (B, N, h, d))
        if y[i] is None:  # a new tensor, contiguous
            ys.append(_dense((B, N, h), (h * N * d, d, N * d) if heads_first else (h * N * d, h * d, d)))
        else:
            _need(y[i], names[i], dt, shapes[i])
            ys.append(_strides(y[i], names[i], _BHN if heads_first else _BNH))
        if dx and dx[i] is not None:
            _need(dx[i], names[2 + i], dt, (B, N, h, d))
            ds.append(_strides(dx[i], names[2 + i], _BNH))
        else:
            ds.append(_dense((B, N, h), (N * h * d, h * d, d)))
    p = FaQkParams(B, N, Hq, Hk, d, _CODES[dt], _CODES[wt], 2 * freqs.shape[0], int(bool(interleaved)), float(eps),
                   pos_stride, I64x3(*_strides(q, "q", _BNH)), I64x3(*_strides(k, "k", _BNH)), I64x3(*ys[0]),
                   I64x3(*ys[1]), I64x3(*ds[0]), I64x3(*ds[1]))
    return p, device, shapes


def _plan_qk(q, k, wq, wk, freqs, positions, yq, yk, eps, interleaved, heads_first):
    p, device, shapes = _qk_checked(q, k, wq, wk, freqs, positions, eps, interleaved, heads_first, (yq, yk), (),
                                    ("out[0]", "out[1]"))
    new = _Outputs()
    res = [new.given(6, yq, shapes[0], q.dtype), new.given(7, yk, shapes[1], q.dtype)]
    return device, [_const(p), *map(_in, range(6)), *res, _STREAM], new, res, p


def _plan_qk_bwd(q, k, dyq, dyk, wq, wk, freqs, positions, dq, dk, workspace, eps, interleaved, heads_first):
    p, device, shapes = _qk_checked(q, k, wq, wk, freqs, positions, eps, interleaved, heads_first, (dyq, dyk), (dq, dk),
                                    ("dyq", "dyk", "dq", "dk"))
    new = _Outputs()
    res = [new.given(8, dq, q.shape, q.dtype), new.given(9, dk, k.shape, q.dtype),
           new.new((q.shape[3],), torch.float32), new.new((q.shape[3],), torch.float32)]
    ws, nbytes = _workspace(new, 10, workspace, load().fa_qk_norm_rope_bwd_workspace_size(ctypes.byref(p)), device)
    return device, [_const(p), *map(_in, range(8)), *res, ws, _const(nbytes), _STREAM], new, res, p


def qk_norm_rope(q, k, wq, wk, freqs, positions=None, eps: float = 1e-6, interleaved: bool = False,
                 heads_first: bool = True, out=None, stream=None):
    """(yq, yk): RMS norm of each head of q [B, N, Hq, d] and k [B, N, Hk, d] (any strides of
    whole 16-byte vectors, such as views of one packed projection), times wq, wk [d], then
    the rotation of the first 2 * len(freqs) channels by the positions (int32 [N] or
    [B, N]; None: 0 .. N - 1).  Results are [B, H, N, d] as ``attention_fwd`` takes them
    (where Hq = Hk), or, with ``heads_first`` false, [B, N, H, d]; ``out`` (yq, yk) may be (q, k) there."""
    yq, yk = (None, None) if out is None else out
    return _call(_QK, (q, k, wq, wk, freqs, positions, yq, yk), (float(eps), bool(interleaved), bool(heads_first)),
                 stream, _plan_qk)


def qk_norm_rope_bwd(q, k, dyq, dyk, wq, wk, freqs, positions=None, eps: float = 1e-6, interleaved: bool = False,
                     heads_first: bool = True, dq=None, dk=None, workspace=None, stream=None):
    """(dq, dk, dwq, dwk): gradients of ``qk_norm_rope`` for dyq, dyk at its results (in its
    layout); q and k are its inputs.  dq, dk are [B, N, H, d] in q's dtype (views of a
    packed gradient may be given), dwq, dwk fp32 [d]."""
    return _call(_QK_BWD, (q, k, dyq, dyk, wq, wk, freqs, positions, dq, dk, workspace),
                 (float(eps), bool(interleaved), bool(heads_first)), stream, _plan_qk_bwd)


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


def _rows_checked(cache, slots, k, v, T, H, d, dtype, heads_first, names):
    """(cache parameters, row parameters, device)."""
    c = _cache_params(cache, d)
    if cache.shape[1] != H:
        raise ValueError(f"{names[0]} has {H} heads, the cache {cache.shape[1]}")
    _need(slots, "slots", torch.int32, (T,))
    _contiguous(slots, "slots")
    strides = []
    for x, name in zip((k, v), names):
        if x is None:  # new and contiguous
            strides.append(_dense((T, H), (d, T * d) if heads_first else (H * d, d)))
        else:
            _need(x, name, dtype, (H, T, d) if heads_first else (T, H, d))
            strides.append(_strides(x, name, (1, 0) if heads_first else (0, 1)))
    rows = FaKv4Rows(T, _CODES[dtype], I64x2(*strides[0]), I64x2(*strides[1]))
    return c, rows, _one_device(cache, slots, k, v)


def _plan_append(k, v, slots, cache):
    if k.dtype not in _CODES:
        raise TypeError(f"unsupported dtype {k.dtype}")
    _need(k, "k", k.dtype, (None, None, None))
    T, H, d = k.shape
    c, rows, device = _rows_checked(cache, slots, k, v, T, H, d, k.dtype, False, ("k", "v"))
    return device, [_const(c), _const(rows), *map(_in, range(4)), _STREAM], (), (), (c, rows)


def _plan_gather(cache, slots, k, v, d, dtype, heads_first):
    if dtype not in _CODES:
        raise TypeError(f"unsupported dtype {dtype}")
    _need(cache, "cache", torch.uint8, (None, None, None, None))
    _need(slots, "slots", torch.int32, (None,))
    T, H = slots.shape[0], cache.shape[1]
    c, rows, device = _rows_checked(cache, slots, k, v, T, H, d, dtype, heads_first, ("out[0]", "out[1]"))
    new, shape = _Outputs(), (H, T, d) if heads_first else (T, H, d)
    res = [new.given(2, k, shape, dtype), new.given(3, v, shape, dtype)]
    return device, [_const(c), _const(rows), _in(0), _in(1), *res, _STREAM], new, res, (c, rows)


def kv4_append(k, v, slots, cache, stream=None) -> None:
    """Quantise the keys and values [T, Hk, d] of T tokens into their slots (int32 [T];
    negative: left out; distinct otherwise) of the cache.  Values saturate at +-16384."""
    _call(_APPEND, (k, v, slots, cache), (), stream, _plan_append)


def kv4_gather(cache, slots, d: int, dtype=torch.bfloat16, heads_first: bool = False, out=None, stream=None):
    """(k, v): the cached keys and values of T slots (zeros for a negative one), rounded to
    ``dtype``: [T, Hk, d], or, ``heads_first``, [Hk, T, d]; with a leading batch of one
    ``attention_fwd`` takes these for the T queries of the same tokens and Hq = Hk."""
    k, v = (None, None) if out is None else out
    return _call(_GATHER, (cache, slots, k, v), (int(d), dtype, bool(heads_first)), stream, _plan_gather)


def _plan_attention(q, cache, block_table, kv_lens, cu_q, out, lse, workspace, max_q_len, scale, window):
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
    o_stride = _dense((T, Hq), (Hq * d, d))
    if out is not None:
        _need(out, "out", q.dtype, (T, Hq, d))
        o_stride = _strides(out, "out", (0, 1))
    if lse is not None:
        _need(lse, "lse", torch.float32, (T, Hq))
        _contiguous(lse, "lse")
    device = _one_device(q, cache, block_table, kv_lens, cu_q, out, lse)
    p = FaKv4AttnParams(R, T, Hq, _CODES[q.dtype], int(max_q_len), int(window), width,
                        1.0 / math.sqrt(d) if scale is None else float(scale),
                        block_table.stride(0) if R > 1 else width, I64x2(*_strides(q, "q", (0, 1))), I64x2(*o_stride))
    new = _Outputs()
    res = [new.given(5, out, (T, Hq, d), q.dtype), new.given(6, lse, (T, Hq), torch.float32)]
    ws, nbytes = _workspace(new, 7, workspace, load().fa_kv4_attention_workspace_size(ctypes.byref(c), ctypes.byref(p)), device)
    return device, [_const(c), _const(p), *map(_in, range(5)), *res, ws, _const(nbytes), _STREAM], new, res, (c, p)


def kv4_attention(q, cache, block_table, kv_lens, cu_q=None, max_q_len: int = 1, scale: Optional[float] = None,
                  window: int = 0, out=None, lse=None, workspace=None, stream=None):
    """(o, lse): attention of each request's newest tokens, q [T, Hq, d], over its cached
    tokens.  Request r has kv_lens[r] tokens (these queries' own among them) in the pages
    block_table[r]; its queries are rows cu_q[r] : cu_q[r + 1] (None: row r), the last of
    them at its last token; each sees the tokens up to its own, and with ``window`` > 0
    only the last ``window`` of those.  Rows without a token to see: o = 0, lse = -inf;
    rows outside every request are not written.  ``max_q_len``: the most rows of a request,
    a hint.  Lengths stay on the GPU: the call does not synchronise."""
    return _call(_ATTENTION, (q, cache, block_table, kv_lens, cu_q, out, lse, workspace),
                 (int(max_q_len), None if scale is None else float(scale), int(window)), stream, _plan_attention)


# ---------------------------------------------------------------- block tables and slot maps

_PLAN_OUT = ("kv_lens", "cu_q", "positions", "slots", "counts")


def _plan_plan(seq_lens, new_lens, block_table, free_pages, free_count, kv_lens, cu_q, positions, slots, counts,
               page_size, T):
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
    if T < 0:
        raise ValueError("T is negative")
    given, new, res = (kv_lens, cu_q, positions, slots, counts), _Outputs(), []
    for i, (t, name, n) in enumerate(zip(given, _PLAN_OUT, (R, R + 1, int(T), int(T), 3))):
        if t is not None:
            _need(t, f"out[{name!r}]", i32, (n,))
            _contiguous(t, f"out[{name!r}]")
        res.append(new.given(5 + i, t, (n,), i32))
    device = _one_device(seq_lens, new_lens, block_table, free_pages, free_count, *given)
    p = FaPlanParams(R, int(T), int(page_size), free_pages.shape[0], width, block_table.stride(0) if R > 1 else width)
    return device, [_const(p), *map(_in, range(5)), *res, _STREAM], new, res, p


def paged_plan(seq_lens, new_lens, block_table, free_pages, free_count, page_size: int, T: int, out=None, stream=None):
    """One step's block tables and slot maps, from request lengths (``fa_paged_plan``; int32
    device tensors).  Request r holds seq_lens[r] tokens and gets new_lens[r] more (< 0: it
    has ended and its pages go back).  block_table [R, width] and the stack
    free_pages[: free_count] are updated in place.  Returns, or fills ``out`` with,
    kv_lens [R], cu_q [R + 1], positions [T], slots [T] and counts [3] (pages left, new
    tokens, pages missing).  A request whose pages are not there keeps its length and gets
    slots of -1.  out["kv_lens"] may be seq_lens, and out["counts"] the tensor whose first
    element is free_count."""
    given = (None,) * 5 if out is None else tuple(out[name] for name in _PLAN_OUT)
    got = _call(_PLAN, (seq_lens, new_lens, block_table, free_pages, free_count, *given), (int(page_size), int(T)),
                stream, _plan_plan)
    return dict(zip(_PLAN_OUT, got))
