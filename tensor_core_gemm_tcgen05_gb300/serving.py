"""Binding of ``include/gemm_serving.h``: rotary positions with per-head norms, the same written
into a paged key/value cache, and attention over such a cache.

    table, scale = g.rope_table(128, base=1e6, scaling="yarn", factor=4, original=32768)
    q = g.kv_append(ctx, q, k, v, k_cache, v_cache, q_start, kv_lens, page_table, table.cuda(), rope_scale=scale)
    out = g.paged_attention(ctx, q, k_cache, v_cache, q_start, kv_lens, page_table, max_q=1)

Queries, keys and values are ``[tokens, heads, head_dim]``, caches ``[pages, kv_heads, page_size,
head_dim]`` (a token-major cache ``[pages, page_size, kv_heads, head_dim]`` is passed as
``cache.transpose(1, 2)``), all float16 or all bfloat16 with ``head_dim`` (64 or 128) contiguous
and the other strides free (multiples of 8). Lengths and tables are int32 tensors on the device.
Like the rest of the package this module only marshals arguments; the header says what each call
computes and refuses.
"""
from __future__ import annotations

import ctypes
import math

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


# Every symbol include/gemm_serving.h declares (the CPU tests check the library exports them).
SERVING_EXPORTS = ("gemm_rope_table", "gemm_qk_rope", "gemm_kv_append", "gemm_paged_attention",
                   "gemm_paged_attention_workspace")


def _declare(L):
    """Argument types of the serving calls (from ``lib()``)."""
    ph, pc, pb, pr = (ctypes.POINTER(t) for t in (Heads, KvCache, KvBatch, Rope))
    L.gemm_rope_table.argtypes = [_i64, ctypes.c_double, ctypes.c_int, ctypes.c_double, ctypes.c_double, _vp,
                                  ctypes.POINTER(_f32)]
    L.gemm_qk_rope.argtypes = [_vp, ctypes.c_int, _i64, _i64, ph, ph, _vp, pr, ph, ph, _vp]
    L.gemm_kv_append.argtypes = [_vp, pc, pb, ph, ph, ph, pr, ph, _vp]
    L.gemm_paged_attention.argtypes = [_vp, pc, pb, ph, _f32, ph, _vp, _i64, _vp, _i64, _vp]
    L.gemm_paged_attention_workspace.argtypes = [_vp, pc, pb, _i64]
    for name in SERVING_EXPORTS:
        getattr(L, name).restype = ctypes.c_int
    L.gemm_paged_attention_workspace.restype = _i64


# ---------------------------------------------------------------------- from tensors to structs

def _pkg():
    import sys
    return sys.modules[__package__]


def _stride(t, dim, other):
    """The stride of ``dim``; that of a dimension of one element does not matter and may be odd."""
    return t.stride(dim) if t.shape[dim] > 1 else other


def _dtype_code(t):
    import torch
    if t.dtype == torch.float16:
        return GEMM_F16
    if t.dtype == torch.bfloat16:
        return GEMM_BF16
    raise ValueError(f"float16 or bfloat16 expected, got {t.dtype}")


def _heads(t, what, like):
    """``gemm_heads`` of ``t`` [tokens, heads, head_dim], of the dtype and device of ``like``."""
    if t is None:
        return Heads(None, 0, 0, 0)
    if t.dim() != 3 or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{what}: a [tokens, heads, head_dim] tensor of {like.dtype} on {like.device} expected")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{what}: head_dim must be contiguous")
    d = t.shape[2]
    return Heads(t.data_ptr(), t.shape[1], _stride(t, 0, t.shape[1] * d), _stride(t, 1, d))


def _same(a, b, what):
    if a.shape != b.shape:
        raise ValueError(f"{what}: shape {tuple(a.shape)} expected, got {tuple(b.shape)}")


def _ints(t, what, shape, device):
    """The address of an int32 tensor of ``shape`` (entries None: any), its last dimension contiguous."""
    import torch
    if t.dtype != torch.int32 or t.device != device or t.dim() != len(shape) or any(
            s is not None and s != n for s, n in zip(shape, t.shape)):
        raise ValueError(f"{what}: an int32 tensor of shape {shape} on {device} expected")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return t.data_ptr()


def _cache(k_cache, v_cache):
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype or (
            k_cache.device != v_cache.device):
        raise ValueError("k_cache and v_cache: [pages, kv_heads, page_size, head_dim] of one shape, type and device expected")
    n, h, p, d = k_cache.shape
    if any(k_cache.shape[i] > 1 and k_cache.stride(i) != v_cache.stride(i) for i in range(4)):
        raise ValueError("k_cache and v_cache must have the same strides")
    if d > 1 and k_cache.stride(3) != 1:
        raise ValueError("k_cache and v_cache: head_dim must be contiguous")
    return KvCache(k_cache.data_ptr(), v_cache.data_ptr(), n, p, h, d, _stride(k_cache, 0, d), _stride(k_cache, 1, d),
                   _stride(k_cache, 2, d), _dtype_code(k_cache))


def _batch(tokens, q_start, kv_lens, page_table, device, max_q=None, prefix_pages=None, num_prefix_pages=0):
    n = kv_lens.shape[0]
    ps = _ints(q_start, "q_start", (n + 1,), device)
    pk = _ints(kv_lens, "kv_lens", (n,), device)
    pt = _ints(page_table, "page_table", (n, None), device)
    pre = None
    if prefix_pages is not None:
        pre = _ints(prefix_pages, "prefix_pages", (None,), device)
        num_prefix_pages = prefix_pages.shape[0]
    width = page_table.shape[1]
    return KvBatch(n, tokens, 0 if max_q is None else int(max_q), ps, pk, pt, width, _stride(page_table, 0, width), pre,
                   num_prefix_pages)


def _rope(q_norm, k_norm, eps, table, interleaved, scale, like):
    import torch
    for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
        if w is not None and (w.dtype != like.dtype or w.device != like.device or w.shape != (like.shape[2],)
                              or not w.is_contiguous()):
            raise ValueError(f"{name}: {like.shape[2]} contiguous weights of {like.dtype} on {like.device} expected")
    if table is not None and (table.dtype not in (torch.int64, torch.uint64) or table.device != like.device
                              or table.dim() != 1 or not table.is_contiguous()):
        raise ValueError(f"table: a contiguous int64 vector on {like.device} expected")
    return Rope(None if table is None else table.data_ptr(), 0 if table is None else 2 * table.shape[0],
                None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(),
                float(eps), float(scale), int(bool(interleaved)))


def _on(stream, t):
    """The handle of ``stream``; None is the current stream of ``t``'s device."""
    import torch
    s = torch.cuda.current_stream(t.device) if stream is None else stream
    return int(s.cuda_stream) if hasattr(s, "cuda_stream") else int(s)


# --------------------------------------------------------------------------------- the calls

def rope_table(rotary_dim, base=10000.0, scaling=None, factor=1.0, original=None):
    """``(table, scale)``: the frequencies of ``gemm_rope`` as an int64 CPU tensor of
    ``rotary_dim / 2`` words (turns a position in units of 2^-64) and the factor for
    ``rope_scale``. ``scaling``: None, "linear", "ntk" or "yarn" (with ``original``, the trained
    length), for contexts ``factor`` times as long."""
    import torch
    g = _pkg()
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling: one of {sorted(k for k in _SCALINGS if k)} or None expected, got {scaling!r}")
    if not 16 <= int(rotary_dim) <= 128:
        raise g.GemmError(g.GEMM_ERR_ARG, "gemm_rope_table")
    table = torch.empty(int(rotary_dim) // 2, dtype=torch.int64)
    scale = _f32(1.0)
    g._check(g.lib().gemm_rope_table(int(rotary_dim), float(base), _SCALINGS[scaling], float(factor),
                                     0.0 if original is None else float(original), table.data_ptr(), ctypes.byref(scale)),
             "gemm_rope_table")
    return table, float(scale.value)


def qk_rope(ctx, q, k, positions, table=None, interleaved=False, rope_scale=1.0, q_norm=None, k_norm=None, eps=1e-6,
            q_out=None, k_out=None, stream=None):
    """Norm (if there are weights) and rotation (if there is a table) of ``q`` and ``k`` at
    ``positions`` (int32, one per token) through ``gemm_qk_rope``. Returns ``(q_out, k_out)``,
    allocated contiguous when not given; an output may be its own input. ``k`` may be None."""
    import torch
    g = _pkg()
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if k_out is None and k is not None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    if (k is None) != (k_out is None):
        raise ValueError("k_out without k")
    hq, hqo = _heads(q, "q", q), _heads(q_out, "q_out", q)
    hk, hko = _heads(k, "k", q), _heads(k_out, "k_out", q)
    _same(q, q_out, "q_out")
    if k is not None:
        _same(k, k_out, "k_out")
        if k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
            raise ValueError(f"k: {q.shape[0]} tokens of head_dim {q.shape[2]} expected, got {tuple(k.shape)}")
    pos = _ints(positions, "positions", (q.shape[0],), q.device)
    r = _rope(q_norm, k_norm, eps, table, interleaved, rope_scale, q)
    rc = g.lib().gemm_qk_rope(g._h(ctx), _dtype_code(q), q.shape[0], q.shape[2], hq, hk, pos, r, hqo, hko, _on(stream, q))
    g._check(rc, "gemm_qk_rope")
    return q_out, k_out


def kv_append(ctx, q, k, v, k_cache, v_cache, q_start, kv_lens, page_table, table=None, prefix_len=0, interleaved=False,
              rope_scale=1.0, q_norm=None, k_norm=None, eps=1e-6, q_out=None, stream=None):
    """Norm and rotation of a ragged batch's new queries and keys, the keys and ``v`` written to
    their rows of the cache, through ``gemm_kv_append``. ``kv_lens`` counts each sequence's own
    keys with the new ones; ``prefix_len`` (whole pages) the keys of a shared prefix before them.
    Returns ``q_out`` (allocated when not given; may be ``q``; None if ``q`` is None)."""
    import torch
    g = _pkg()
    c = _cache(k_cache, v_cache)
    if prefix_len < 0 or c.page_size == 0 or prefix_len % c.page_size:
        raise ValueError(f"prefix_len: whole pages of {c.page_size} expected, got {prefix_len}")
    if q_out is None and q is not None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if (q is None) != (q_out is None):
        raise ValueError("q_out without q")
    hk, hv = _heads(k, "k", k_cache), _heads(v, "v", k_cache)
    hq, hqo = _heads(q, "q", k_cache), _heads(q_out, "q_out", k_cache)
    _same(k, v, "v")
    if k.shape[1:] != (c.kv_heads, c.head_dim):
        raise ValueError(f"k: [tokens, {c.kv_heads}, {c.head_dim}] expected, got {tuple(k.shape)}")
    if q is not None:
        _same(q, q_out, "q_out")
        if q.shape[0] != k.shape[0] or q.shape[2] != c.head_dim:
            raise ValueError(f"q: {k.shape[0]} tokens of head_dim {c.head_dim} expected, got {tuple(q.shape)}")
    b = _batch(k.shape[0], q_start, kv_lens, page_table, k_cache.device, num_prefix_pages=prefix_len // c.page_size)
    r = _rope(q_norm, k_norm, eps, table, interleaved, rope_scale, k)
    rc = g.lib().gemm_kv_append(g._h(ctx), c, b, hq, hk, hv, r, hqo, _on(stream, k_cache))
    g._check(rc, "gemm_kv_append")
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
    import torch
    g = _pkg()
    c = _cache(k_cache, v_cache)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    hq, ho = _heads(q, "q", k_cache), _heads(out, "out", k_cache)
    _same(q, out, "out")
    if q.shape[2] != c.head_dim:
        raise ValueError(f"q: head_dim {c.head_dim} expected, got {q.shape[2]}")
    b = _batch(q.shape[0], q_start, kv_lens, page_table, q.device, max_q, prefix_pages)
    lse_ptr, lse_stride = None, 0
    if lse is not None:
        if lse.dtype != torch.float32 or lse.device != q.device or lse.shape != q.shape[:2] or (
                lse.shape[1] > 1 and lse.stride(1) != 1):
            raise ValueError(f"lse: a float32 tensor of shape {tuple(q.shape[:2])} on {q.device}, heads contiguous, expected")
        lse_ptr, lse_stride = lse.data_ptr(), _stride(lse, 0, lse.shape[1])
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()
                                  or workspace.device != q.device):
        raise ValueError(f"workspace: a contiguous uint8 tensor on {q.device} expected")
    handle = _on(stream, q)
    if workspace is None:
        need = g.lib().gemm_paged_attention_workspace(g._h(ctx), c, b, q.shape[1])
        if need < 0:
            raise g.GemmError(int(need), "gemm_paged_attention_workspace")
        if handle == torch.cuda.current_stream(q.device).cuda_stream:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:   # the allocator must know the stream that uses the memory
            with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=q.device)):
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    s = 1.0 / math.sqrt(c.head_dim) if scale is None else float(scale)
    rc = g.lib().gemm_paged_attention(g._h(ctx), c, b, hq, s, ho, lse_ptr, lse_stride, workspace.data_ptr(),
                                      workspace.numel(), handle)
    g._check(rc, "gemm_paged_attention")
    return out


def paged_attention_workspace(ctx, q, k_cache, v_cache, q_start, kv_lens, page_table, max_q=None, prefix_pages=None):
    """Workspace bytes of ``paged_attention`` for these arguments (shapes are read, contents are not)."""
    g = _pkg()
    c = _cache(k_cache, v_cache)
    b = _batch(q.shape[0], q_start, kv_lens, page_table, q.device, max_q, prefix_pages)
    need = g.lib().gemm_paged_attention_workspace(g._h(ctx), c, b, q.shape[1])
    if need < 0:
        raise g.GemmError(int(need), "gemm_paged_attention_workspace")
    return int(need)
