"""Binding of ``include/gemm_serving.h``: rotary positions with per-head norms, the same written
into a paged key/value cache, and attention over such a cache.

    table, scale = g.rope_table(128, base=1e6, scaling="yarn", factor=4, original=32768)
    q = g.kv_append(ctx, q, k, v, k_cache, v_cache, q_start, kv_lens, page_table, table.cuda(), rope_scale=scale)
    out = g.paged_attention(ctx, q, k_cache, v_cache, q_start, kv_lens, page_table, max_q=1)

Queries, keys and values are ``[tokens, heads, head_dim]``, caches ``[pages, kv_heads, page_size,
head_dim]`` (a token-major cache ``[pages, page_size, kv_heads, head_dim]`` is passed as
``cache.transpose(1, 2)``), all float16 or all bfloat16 with ``head_dim`` (64 or 128) contiguous
and the other strides free (multiples of 8). Lengths and tables are int32 tensors on the device.
Calls run on ``stream`` (None: torch's current one); what they allocate belongs to that stream.
Like the rest of the package this module only marshals arguments; the header says what each call
computes and refuses.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

_g = None   # the package (set by it: this module is part of its import)

_i64, _i32, _vp, _f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float

GEMM_F16, GEMM_BF16 = 0, 1
GEMM_ROPE_PLAIN, GEMM_ROPE_LINEAR, GEMM_ROPE_NTK, GEMM_ROPE_YARN = 0, 1, 2, 3
_SCALINGS = {None: GEMM_ROPE_PLAIN, "linear": GEMM_ROPE_LINEAR, "ntk": GEMM_ROPE_NTK, "yarn": GEMM_ROPE_YARN}


class Heads(ctypes.Structure):
    """``gemm_heads``"""
    _fields_ = [("data", _vp), ("heads", _i64), ("token_stride", _i64), ("head_stride", _i64)]


class KvCache(ctypes.Structure):
    """``gemm_kv_cache``"""
    _fields_ = [("k", _vp), ("v", _vp), ("num_pages", _i64), ("page_size", _i64), ("kv_heads", _i64),
                ("head_dim", _i64), ("page_stride", _i64), ("head_stride", _i64), ("row_stride", _i64), ("dtype", _i32)]


class KvBatch(ctypes.Structure):
    """``gemm_kv_batch``"""
    _fields_ = [("num_seqs", _i64), ("num_tokens", _i64), ("max_q", _i64), ("q_start", _vp), ("kv_lens", _vp),
                ("page_table", _vp), ("table_width", _i64), ("table_stride", _i64), ("prefix_pages", _vp),
                ("num_prefix_pages", _i64)]


class Rope(ctypes.Structure):
    """``gemm_rope``"""
    _fields_ = [("table", _vp), ("rotary_dim", _i64), ("q_norm", _vp), ("k_norm", _vp), ("eps", _f32), ("scale", _f32),
                ("interleaved", _i32)]


# The same structs as the calls below pack them (a bytes object costs a third of a Structure to make).
_HEADS, _CACHE = struct.Struct("@Pqqq"), struct.Struct("@PPqqqqqqqi4x")
_BATCH, _ROPE = struct.Struct("@qqqPPPqqPq"), struct.Struct("@PqPPffi4x")
_NO_HEADS = _HEADS.pack(0, 0, 0, 0)

# Every symbol include/gemm_serving.h declares (the CPU tests check the library exports them).
SERVING_EXPORTS = ("gemm_rope_table", "gemm_qk_rope", "gemm_kv_append", "gemm_paged_attention",
                   "gemm_paged_attention_workspace")


def _declare(L):
    """Argument types of the serving calls (from ``lib()``); structs go by address or as bytes."""
    L.gemm_rope_table.argtypes = [_i64, ctypes.c_double, ctypes.c_int, ctypes.c_double, ctypes.c_double, _vp,
                                  ctypes.POINTER(_f32)]
    L.gemm_qk_rope.argtypes = [_vp, ctypes.c_int, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
    L.gemm_kv_append.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
    L.gemm_paged_attention.argtypes = [_vp, _vp, _vp, _vp, _f32, _vp, _vp, _i64, _vp, _i64, _vp]
    L.gemm_paged_attention_workspace.argtypes = [_vp, _vp, _vp, _i64]
    for name in SERVING_EXPORTS:
        getattr(L, name).restype = ctypes.c_int
    L.gemm_paged_attention_workspace.restype = _i64


# ---------------------------------------------------------------------- from tensors to structs

def _lib():
    return _g._lib or _g.lib()


_CODES = {torch.float16: GEMM_F16, torch.bfloat16: GEMM_BF16}


def _dtype_code(dtype):
    code = _CODES.get(dtype)
    if code is None:
        raise ValueError(f"float16 or bfloat16 expected, got {dtype}")
    return code


def _heads(t, what, dtype, device, shape=None):
    """``gemm_heads`` of ``t`` [tokens, heads, head_dim] (the stride of a dimension of one element
    does not matter and may be odd: a plain one stands in for it)."""
    s = t.shape
    if len(s) != 3 or t.dtype != dtype or t.device != device:
        raise ValueError(f"{what}: a [tokens, heads, head_dim] tensor of {dtype} on {device} expected")
    if shape is not None and s != shape:
        raise ValueError(f"{what}: shape {tuple(shape)} expected, got {tuple(s)}")
    st, sh, sd = t.stride()
    n, h, d = s
    if sd != 1 and d > 1:
        raise ValueError(f"{what}: head_dim must be contiguous")
    return _HEADS.pack(t.data_ptr(), h, st if n > 1 else h * d, sh if h > 1 else d)


_int32 = torch.int32   # (a global: half of an attribute of torch to look up)


def _ints(t, what, shape, device):
    """The address of an int32 tensor of ``shape`` (entries None: any), its last dimension contiguous."""
    s = t.shape
    if t.dtype is not _int32 or t.device != device or len(s) != len(shape) or s[0] != shape[0] and shape[0] is not None:
        raise ValueError(f"{what}: an int32 tensor of shape {shape} on {device} expected")
    if s[-1] > 1 and t.stride()[-1] != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return t.data_ptr()


def _vector(t, what, n, device):
    """The address of a contiguous int32 vector of ``n`` entries."""
    if t.dtype is not _int32 or t.shape != (n,) or t.device != device:
        raise ValueError(f"{what}: an int32 tensor of shape {(n,)} on {device} expected")
    if n > 1 and t.stride() != (1,):
        raise ValueError(f"{what}: the entries must be contiguous")
    return t.data_ptr()


def _cache(k_cache, v_cache):
    """``gemm_kv_cache``, page size, heads and head_dim."""
    s = k_cache.shape
    if len(s) != 4 or s != v_cache.shape or k_cache.dtype != v_cache.dtype or k_cache.device != v_cache.device:
        raise ValueError("k_cache and v_cache: [pages, kv_heads, page_size, head_dim] of one shape, type and device expected")
    n, h, p, d = s
    strides = k_cache.stride()
    if strides != v_cache.stride() and any(m > 1 and a != b for m, a, b in zip(s, strides, v_cache.stride())):
        raise ValueError("k_cache and v_cache must have the same strides")
    sn, sh, sp, sd = strides
    if sd != 1 and d > 1:
        raise ValueError("k_cache and v_cache: head_dim must be contiguous")
    return _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), n, p, h, d, sn if n > 1 else d, sh if h > 1 else d,
                       sp if p > 1 else d, _dtype_code(k_cache.dtype)), p, h, d


def _batch(tokens, q_start, kv_lens, page_table, device, max_q=None, prefix_pages=None, num_prefix_pages=0):
    s = kv_lens.shape
    n = s[0] if s else -1
    ps = _vector(q_start, "q_start", n + 1, device)
    pk = _vector(kv_lens, "kv_lens", n, device)
    pt = _ints(page_table, "page_table", (n, None), device)
    pre = 0
    if prefix_pages is not None:
        pre = _ints(prefix_pages, "prefix_pages", (None,), device)
        num_prefix_pages = prefix_pages.shape[0]
    width = page_table.shape[1]
    return _BATCH.pack(n, tokens, 0 if max_q is None else int(max_q), ps, pk, pt, width,
                       page_table.stride(0) if n > 1 else width, pre, num_prefix_pages)


def _weights(w, what, d, dtype, device):
    if w is None:
        return 0
    if w.dtype != dtype or w.device != device or w.shape != (d,) or not w.is_contiguous():
        raise ValueError(f"{what}: {d} contiguous weights of {dtype} on {device} expected")
    return w.data_ptr()


def _lse(lse, shape, device):
    """Address and token stride of ``lse`` for queries of ``shape``; None: no address."""
    if lse is None:
        return None, 0
    if lse.dtype != torch.float32 or lse.device != device or lse.shape != shape[:2] or shape[1] > 1 and lse.stride(1) != 1:
        raise ValueError(f"lse: a float32 tensor of shape {tuple(shape[:2])} on {device}, heads contiguous, expected")
    return lse.data_ptr(), lse.stride(0) if shape[0] > 1 else shape[1]


def _rope(q_norm, k_norm, eps, table, interleaved, scale, d, dtype, device):
    words, half = 0, 0
    if table is not None:
        if table.dtype != torch.int64 and table.dtype != torch.uint64 or table.device != device or table.dim() != 1 or (
                not table.is_contiguous()):
            raise ValueError(f"table: a contiguous int64 vector on {device} expected")
        words, half = table.data_ptr(), table.shape[0]
    return _ROPE.pack(words, 2 * half, _weights(q_norm, "q_norm", d, dtype, device), _weights(k_norm, "k_norm", d, dtype, device),
                      eps, scale, 1 if interleaved else 0)


def _current(device):
    """The handle of torch's current stream of ``device``."""
    try:   # a fifth of current_stream()'s cost
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device.index is None else device.index)
    except AttributeError:
        return torch.cuda.current_stream(device).cuda_stream


def _on(stream, device):
    """The handle of ``stream``; None is the current stream of ``device``."""
    if stream is None:
        return _current(device)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


_torch_empty = torch.empty


def _empty(shape, dtype, device, stream):
    """A tensor for a kernel on ``stream`` (None: the current one) to write. The memory comes from what is free
    on that stream: a block that is free on the current one may still be in use by work queued there."""
    if stream is None or device.type != "cuda":   # (the library refuses host memory)
        return _torch_empty(shape, dtype=dtype, device=device)
    handle = _on(stream, device)
    if handle == _current(device):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=device)):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))   # the caller's, that goes on with it
    return t


# --------------------------------------------------------------------------------- the calls

def rope_table(rotary_dim, base=10000.0, scaling=None, factor=1.0, original=None):
    """``(table, scale)``: the frequencies of ``gemm_rope`` as an int64 CPU tensor of
    ``rotary_dim / 2`` words (turns a position in units of 2^-64) and the factor for
    ``rope_scale``. ``scaling``: None, "linear", "ntk" or "yarn" (with ``original``, the trained
    length; by the paper's formula, see the header), for contexts ``factor`` times as long. Frequencies
    ``f`` of any other rule, in radians a position, are a table as ``round(f / (2 pi) * 2**64)``."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling: one of {sorted(k for k in _SCALINGS if k)} or None expected, got {scaling!r}")
    if not 16 <= int(rotary_dim) <= 128:
        raise _g.GemmError(_g.GEMM_ERR_ARG, "gemm_rope_table")
    table = torch.empty(int(rotary_dim) // 2, dtype=torch.int64)
    scale = _f32(1.0)
    _g._check(_lib().gemm_rope_table(int(rotary_dim), float(base), _SCALINGS[scaling], float(factor),
                                     0.0 if original is None else float(original), table.data_ptr(), ctypes.byref(scale)),
             "gemm_rope_table")
    return table, float(scale.value)


def qk_rope(ctx, q, k, positions, table=None, interleaved=False, rope_scale=1.0, q_norm=None, k_norm=None, eps=1e-6,
            q_out=None, k_out=None, stream=None):
    """Norm (if there are weights) and rotation (if there is a table) of ``q`` and ``k`` at
    ``positions`` (int32, one per token) through ``gemm_qk_rope``. Returns ``(q_out, k_out)``,
    allocated contiguous when not given; an output may be its own input. ``k`` may be None."""
    shape, dtype, device = q.shape, q.dtype, q.device
    if q_out is None:
        q_out = _empty(shape, dtype, device, stream)
    hq, hqo = _heads(q, "q", dtype, device), _heads(q_out, "q_out", dtype, device, shape)
    hk = hko = _NO_HEADS
    if k is not None:
        if k_out is None:
            k_out = _empty(k.shape, dtype, device, stream)
        hk, hko = _heads(k, "k", dtype, device), _heads(k_out, "k_out", dtype, device, k.shape)
        if k.shape[0] != shape[0] or k.shape[2] != shape[2]:
            raise ValueError(f"k: {shape[0]} tokens of head_dim {shape[2]} expected, got {tuple(k.shape)}")
    elif k_out is not None:
        raise ValueError("k_out without k")
    pos = _ints(positions, "positions", (shape[0],), device)
    r = _rope(q_norm, k_norm, eps, table, interleaved, rope_scale, shape[2], dtype, device)
    _g._check(_lib().gemm_qk_rope(_g._h(ctx), _dtype_code(dtype), shape[0], shape[2], hq, hk, pos, r, hqo, hko,
                                  _on(stream, device)), "gemm_qk_rope")
    return q_out, k_out


def kv_append(ctx, q, k, v, k_cache, v_cache, q_start, kv_lens, page_table, table=None, prefix_len=0, interleaved=False,
              rope_scale=1.0, q_norm=None, k_norm=None, eps=1e-6, q_out=None, stream=None):
    """Norm and rotation of a ragged batch's new queries and keys, the keys and ``v`` written to
    their rows of the cache, through ``gemm_kv_append``. ``kv_lens`` counts each sequence's own
    keys with the new ones; ``prefix_len`` (whole pages) the keys of a shared prefix before them.
    Returns ``q_out`` (allocated when not given; may be ``q``; None if ``q`` is None)."""
    dtype, device = k_cache.dtype, k_cache.device
    c, page, kv_heads, d = _cache(k_cache, v_cache)
    if prefix_len < 0 or page == 0 or prefix_len % page:
        raise ValueError(f"prefix_len: whole pages of {page} expected, got {prefix_len}")
    hk, hv = _heads(k, "k", dtype, device), _heads(v, "v", dtype, device, k.shape)
    tokens = k.shape[0]
    if k.shape[1] != kv_heads or k.shape[2] != d:
        raise ValueError(f"k: [tokens, {kv_heads}, {d}] expected, got {tuple(k.shape)}")
    hq = hqo = _NO_HEADS
    if q is not None:
        if q_out is None:
            q_out = _empty(q.shape, dtype, device, stream)
        hq, hqo = _heads(q, "q", dtype, device), _heads(q_out, "q_out", dtype, device, q.shape)
        if q.shape[0] != tokens or q.shape[2] != d:
            raise ValueError(f"q: {tokens} tokens of head_dim {d} expected, got {tuple(q.shape)}")
    elif q_out is not None:
        raise ValueError("q_out without q")
    b = _batch(tokens, q_start, kv_lens, page_table, device, num_prefix_pages=prefix_len // page)
    r = _rope(q_norm, k_norm, eps, table, interleaved, rope_scale, d, dtype, device)
    _g._check(_lib().gemm_kv_append(_g._h(ctx), c, b, hq, hk, hv, r, hqo, _on(stream, device)), "gemm_kv_append")
    return q_out


def paged_attention(ctx, q, k_cache, v_cache, q_start, kv_lens, page_table, max_q=None, prefix_pages=None, scale=None,
                    out=None, lse=None, workspace=None, stream=None):
    """Causal attention of a ragged batch's new queries over the paged cache through
    ``gemm_paged_attention`` (``scale`` defaults to 1/sqrt(head_dim)). ``max_q``: the largest
    number of new tokens of a sequence, if known. ``prefix_pages``: the pages of a prefix that
    all sequences share, which ``kv_lens`` does not count. ``lse``: a float32 [tokens, q_heads]
    tensor to fill with the log of each row's sum of exponentials. ``workspace``: a uint8 tensor
    of at least ``paged_attention_workspace`` bytes, allocated for the call when not given.
    Returns ``out`` (allocated when not given)."""
    L, h = _lib(), _g._h(ctx)
    shape, dtype, device = q.shape, k_cache.dtype, k_cache.device
    c, _, _, d = _cache(k_cache, v_cache)
    if out is None:
        out = _empty(shape, dtype, device, stream)
    hq, ho = _heads(q, "q", dtype, device), _heads(out, "out", dtype, device, shape)
    tokens, heads, q_dim = shape
    if q_dim != d:
        raise ValueError(f"q: head_dim {d} expected, got {q_dim}")
    b = _batch(tokens, q_start, kv_lens, page_table, device, max_q, prefix_pages)
    lse_ptr, lse_stride = _lse(lse, shape, device)
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != device):
        raise ValueError(f"workspace: a contiguous uint8 tensor on {device} expected")
    if workspace is None:
        need = L.gemm_paged_attention_workspace(h, c, b, heads)
        if need < 0:
            raise _g.GemmError(int(need), "gemm_paged_attention_workspace")
        workspace = _empty((need,), torch.uint8, device, stream)
    if scale is None:
        scale = 1.0 / math.sqrt(d) if d else 1.0   # (a head_dim of 0 is the library's to refuse)
    _g._check(L.gemm_paged_attention(h, c, b, hq, scale, ho, lse_ptr, lse_stride,
                                    workspace.data_ptr(), workspace.numel(), _on(stream, device)), "gemm_paged_attention")
    return out


def paged_attention_workspace(ctx, q, k_cache, v_cache, q_start, kv_lens, page_table, max_q=None, prefix_pages=None):
    """Workspace bytes of ``paged_attention`` for these arguments (shapes are read, contents are not)."""
    c, _, _, _ = _cache(k_cache, v_cache)
    b = _batch(q.shape[0], q_start, kv_lens, page_table, k_cache.device, max_q, prefix_pages)
    need = _lib().gemm_paged_attention_workspace(_g._h(ctx), c, b, q.shape[1])
    if need < 0:
        raise _g.GemmError(int(need), "gemm_paged_attention_workspace")
    return int(need)
