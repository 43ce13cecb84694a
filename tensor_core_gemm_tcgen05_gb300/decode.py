"""Binding of ``include/gemm_decode.h``: attention for trees of drafted tokens over a paged cache,
the cache held to a bounded size by the attention weight its keys have drawn, rows of it moved
up, and products with 4-bit weights for few rows.

    # drafted trees: parents[t] is the node before token t among its sequence's new tokens, or -1
    mask, positions = g.tree_mask(ctx, parents, q_start, kv_lens, max_nodes)
    q, k = g.qk_rope(ctx, q, k, positions, table)
    g.kv_append(ctx, None, k, v, k_cache, v_cache, q_start, kv_lens, page_table)
    out = g.tree_attention(ctx, q, k_cache, v_cache, q_start, kv_lens, page_table, mask, max_q=max_nodes)
    kv_lens = g.kv_compact(ctx, k_cache, v_cache, kv_lens, page_table, accepted, counts, start=lens_before)

    # a bounded cache: weights is a float32 tensor [pages, kv_heads, page_size]
    g.kv_weigh(ctx, q, k_cache, q_start, kv_lens, page_table, lse, weights)
    index, counts = g.kv_select(ctx, weights, kv_lens, page_table, keep=4096, first=4, recent=256)
    kv_lens = g.kv_compact(ctx, k_cache, v_cache, kv_lens, page_table, index, counts, weights=weights)

    y = g.w4_gemm(ctx, x, codes, scales, zeros, bias, g.EPI_GELU)

Tensors, streams and errors are as in ``serving``; the header says what each call computes and
refuses.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import serving as _s

_g = None   # the package (set by it: this module is part of its import)

_i64, _i32, _vp, _f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float

GEMM_TREE_MAX_WORDS = 64

_int32, _float32, _uint8 = torch.int32, torch.float32, torch.uint8


class Tree(ctypes.Structure):
    """``gemm_tree``"""
    _fields_ = [("mask", _vp), ("mask_words", _i64), ("mask_stride", _i64)]


class KvSeqs(ctypes.Structure):
    """``gemm_kv_seqs``"""
    _fields_ = [("num_seqs", _i64), ("kv_lens", _vp), ("page_table", _vp), ("table_width", _i64), ("table_stride", _i64)]


class KvWeights(ctypes.Structure):
    """``gemm_kv_weights``"""
    _fields_ = [("data", _vp), ("page_stride", _i64), ("head_stride", _i64)]


class W4(ctypes.Structure):
    """``gemm_w4``"""
    _fields_ = [("codes", _vp), ("scales", _vp), ("zeros", _vp), ("group", _i64)]


# The same structs as the calls below pack them.
_TREE, _SEQS, _WEIGHTS, _W4 = struct.Struct("@Pqq"), struct.Struct("@qPPqq"), struct.Struct("@Pqq"), struct.Struct("@PPPq")

# Every symbol include/gemm_decode.h declares (the CPU tests check the library exports them).
DECODE_EXPORTS = ("gemm_tree_mask", "gemm_tree_attention", "gemm_tree_attention_workspace", "gemm_kv_weigh", "gemm_kv_select",
                  "gemm_kv_compact", "gemm_w4_run")


def _declare(L):
    """Argument types of these calls (from ``lib()``); structs go by address or as bytes."""
    L.gemm_tree_mask.argtypes = [_vp, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp]
    L.gemm_tree_attention.argtypes = [_vp, _vp, _vp, _vp, _vp, _f32, _vp, _vp, _i64, _vp, _i64, _vp]
    L.gemm_tree_attention_workspace.argtypes = [_vp, _vp, _vp, _i64]
    L.gemm_kv_weigh.argtypes = [_vp, _vp, _vp, _vp, _f32, _vp, _i64, _i64, _f32, _vp, _vp]
    L.gemm_kv_select.argtypes = [_vp, _vp, _i64, _i64, _i64, _vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp]
    L.gemm_kv_compact.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp]
    L.gemm_w4_run.argtypes = [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _i64, ctypes.c_int, _vp]
    for name in DECODE_EXPORTS:
        getattr(L, name).restype = ctypes.c_int
    L.gemm_tree_attention_workspace.restype = _i64


# ---------------------------------------------------------------------- from tensors to structs

def _seqs(kv_lens, page_table, device):
    """``gemm_kv_seqs`` and the number of sequences."""
    s = kv_lens.shape
    n = s[0] if s else -1
    lens, table = _s._vector(kv_lens, "kv_lens", n, device), _s._ints(page_table, "page_table", (n, None), device)
    width = page_table.shape[1]
    return _SEQS.pack(n, lens, table, width, page_table.stride()[0] if n > 1 else width), n


def _weights(w, device, shape=None):
    """``gemm_kv_weights``"""
    s = w.shape
    if w.dtype is not _float32 or w.device != device or len(s) != 3 or (shape is not None and s != shape):
        raise ValueError(f"weights: a float32 tensor [pages, kv_heads, page_size]{'' if shape is None else f' = {tuple(shape)}'} on "
                         f"{device} expected")
    n, h, p = s
    sn, sh, sp = w.stride()
    if sp != 1 and p > 1:
        raise ValueError("weights: the rows of a page must be contiguous")
    return _WEIGHTS.pack(w.data_ptr(), sn if n > 1 else h * p, sh if h > 1 else p)


def _mask(mask, tokens, device):
    """Address, words and stride of a mask."""
    s = mask.shape
    if (mask.dtype is not _int32 and mask.dtype is not torch.uint32) or len(s) != 2 or s[0] != tokens or mask.device != device or (
            s[1] > 1 and mask.stride()[1] != 1):
        raise ValueError(f"mask: an int32 tensor [{tokens}, words] on {device}, words contiguous, expected")
    return mask.data_ptr(), s[1], mask.stride()[0] if tokens > 1 else s[1]


def _lists(index, n, heads, device):
    """Address, strides and length of index lists [seqs, most] or [seqs, kv_heads, most]."""
    s, strides = index.shape, index.stride()
    dims = len(s)
    if index.dtype is not _int32 or index.device != device or (dims != 2 and dims != 3) or s[0] != n or (
            dims == 3 and s[1] != heads) or (s[-1] > 1 and strides[-1] != 1):
        raise ValueError(f"index: an int32 tensor [{n}, most] or [{n}, {heads}, most] on {device}, the last dimension contiguous, expected")
    most = s[-1]
    return index.data_ptr(), strides[0] if n > 1 else most * heads, 0 if dims == 2 else strides[1] if heads > 1 else most, most


# --------------------------------------------------------------------------------- the calls

def tree_mask(ctx, parents, q_start, kv_lens, max_nodes, prefix_len=0, mask=None, positions=None, stream=None):
    """``(mask, positions)`` of drafted trees through ``gemm_tree_mask``: for each token the bits of
    the nodes that it sees (int32 [tokens, words], room for ``max_nodes`` nodes of a sequence) and
    its position (int32). ``kv_lens`` counts the new tokens, ``prefix_len`` the keys of a shared
    prefix before the sequence's own."""
    device, s = parents.device, parents.shape
    if len(s) != 1:
        raise ValueError("parents: one int32 per token expected")
    tokens = s[0]
    if mask is None:
        if not 0 <= max_nodes <= 32 * GEMM_TREE_MAX_WORDS:
            raise ValueError(f"max_nodes: up to {32 * GEMM_TREE_MAX_WORDS} expected, got {max_nodes}")
        mask = _s._empty((tokens, (max_nodes + 31) // 32 or 1), _int32, device, stream)
    if positions is None:
        positions = _s._empty((tokens,), _int32, device, stream)
    at, words, stride = _mask(mask, tokens, device)
    vector, s = _s._vector, kv_lens.shape
    n = s[0] if s else -1
    b = _s._BATCH.pack(n, tokens, 0, vector(q_start, "q_start", n + 1, device), vector(kv_lens, "kv_lens", n, device), 0, 0, 0, 0, 0)
    _g._check(_s._lib().gemm_tree_mask(_g._h(ctx), b, prefix_len, vector(parents, "parents", tokens, device), at, words, stride,
                                       vector(positions, "positions", tokens, device), _s._on(stream, device)), "gemm_tree_mask")
    return mask, positions


def tree_attention(ctx, q, k_cache, v_cache, q_start, kv_lens, page_table, mask, max_q=None, prefix_pages=None, scale=None,
                   out=None, lse=None, workspace=None, stream=None):
    """Attention of drafted tokens over the paged cache through ``gemm_tree_attention``: each sees
    the keys before its sequence's new ones and, of those, the ones that its row of ``mask`` names.
    All else is as in ``paged_attention``."""
    L, h = _s._lib(), _g._h(ctx)
    shape, dtype, device = q.shape, k_cache.dtype, k_cache.device
    c, _, _, d = _s._cache(k_cache, v_cache)
    if out is None:
        out = _s._empty(shape, dtype, device, stream)
    hq, ho = _s._heads(q, "q", dtype, device), _s._heads(out, "out", dtype, device, shape)
    tokens, heads, q_dim = shape
    if q_dim != d:
        raise ValueError(f"q: head_dim {d} expected, got {q_dim}")
    b = _s._batch(tokens, q_start, kv_lens, page_table, device, max_q, prefix_pages)
    tree = _TREE.pack(*_mask(mask, tokens, device))
    lse_ptr, lse_stride = _s._lse(lse, shape, device)
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != device):
        raise ValueError(f"workspace: a contiguous uint8 tensor on {device} expected")
    if workspace is None:
        need = L.gemm_tree_attention_workspace(h, c, b, heads)
        if need < 0:
            raise _g.GemmError(int(need), "gemm_tree_attention_workspace")
        workspace = _s._empty((need,), torch.uint8, device, stream)
    if scale is None:
        scale = 1.0 / math.sqrt(d) if d else 1.0
    _g._check(L.gemm_tree_attention(h, c, b, tree, hq, scale, ho, lse_ptr, lse_stride, workspace.data_ptr(), workspace.numel(),
                                    _s._on(stream, device)), "gemm_tree_attention")
    return out


def tree_attention_workspace(ctx, q, k_cache, v_cache, q_start, kv_lens, page_table, max_q=None, prefix_pages=None):
    """Workspace bytes of ``tree_attention`` for these arguments (shapes are read, contents are not)."""
    c, _, _, _ = _s._cache(k_cache, v_cache)
    b = _s._batch(q.shape[0], q_start, kv_lens, page_table, k_cache.device, max_q, prefix_pages)
    need = _s._lib().gemm_tree_attention_workspace(_g._h(ctx), c, b, q.shape[1])
    if need < 0:
        raise _g.GemmError(int(need), "gemm_tree_attention_workspace")
    return int(need)


def kv_weigh(ctx, q, k_cache, q_start, kv_lens, page_table, lse, weights, scale=None, window=0, decay=1.0, stream=None):
    """Adds to ``weights`` (float32 [pages, kv_heads, page_size], in place) the attention weight that
    the last ``window`` new tokens (0: all) give to each key, through ``gemm_kv_weigh``; the weights
    before are multiplied by ``decay``, those of the new tokens' keys start from 0. ``lse`` is what
    ``paged_attention`` filled for these queries. Returns ``weights``."""
    dtype, device = k_cache.dtype, k_cache.device
    c, page, heads, d = _s._cache(k_cache, k_cache)
    hq, s = _s._heads(q, "q", dtype, device), q.shape
    if s[2] != d:
        raise ValueError(f"q: head_dim {d} expected, got {s[2]}")
    b = _s._batch(s[0], q_start, kv_lens, page_table, device)
    w = _weights(weights, device, (k_cache.shape[0], heads, page))
    lse_ptr, lse_stride = _s._lse(lse, s, device)
    if scale is None:
        scale = 1.0 / math.sqrt(d) if d else 1.0
    _g._check(_s._lib().gemm_kv_weigh(_g._h(ctx), c, b, hq, scale, lse_ptr, lse_stride, window, decay, w, _s._on(stream, device)),
              "gemm_kv_weigh")
    return weights


def kv_select(ctx, weights, kv_lens, page_table, keep, first=0, recent=0, index=None, counts=None, stream=None):
    """``(index, counts)``: for each sequence and key head the ``keep`` keys to keep (all, if it has
    no more), ascending, -1 behind the last (int32 [seqs, kv_heads, keep]), and their number (int32
    [seqs]), through ``gemm_kv_select``: the first ``first``, the last ``recent`` and the heaviest of
    the others."""
    device = weights.device
    w = _weights(weights, device)
    pages, heads, page = weights.shape
    s, n = _seqs(kv_lens, page_table, device)
    if index is None:
        if keep < 0:
            raise ValueError(f"keep: at least 0 expected, got {keep}")
        index = _s._empty((n, heads, keep), _int32, device, stream)
    elif index.shape != (n, heads, keep):
        raise ValueError(f"index: shape {(n, heads, keep)} expected, got {tuple(index.shape)}")
    if counts is None:
        counts = _s._empty((n,), _int32, device, stream)
    at, seq_stride, head_stride, _ = _lists(index, n, heads, device)
    _g._check(_s._lib().gemm_kv_select(_g._h(ctx), s, pages, page, heads, w, keep, first, recent, at, seq_stride, head_stride,
                                       _s._vector(counts, "counts", n, device), _s._on(stream, device)), "gemm_kv_select")
    return index, counts


def kv_compact(ctx, k_cache, v_cache, kv_lens, page_table, index, counts, start=None, weights=None, new_lens=None, stream=None):
    """Moves rows of the cache up in place through ``gemm_kv_compact``: row ``start + index[j]`` of each
    sequence (and key head) to row ``start + j``, for ``j < counts``. ``index`` is int32 [seqs, kv_heads,
    most] or, for all heads alike, [seqs, most], ascending; ``start`` (None: 0) int32 [seqs];
    ``weights`` as in ``kv_weigh``, moved along if given. Returns the new lengths, ``start + counts``
    (allocated when not given)."""
    device = k_cache.device
    c, page, heads, _ = _s._cache(k_cache, v_cache)
    s, n = _seqs(kv_lens, page_table, device)
    at, seq_stride, head_stride, most = _lists(index, n, heads, device)
    w = None if weights is None else _weights(weights, device, (k_cache.shape[0], heads, page))
    if new_lens is None:
        new_lens = _s._empty((n,), _int32, device, stream)
    vector = _s._vector
    _g._check(_s._lib().gemm_kv_compact(_g._h(ctx), c, s, w, at, seq_stride, head_stride, most,
                                        None if start is None else vector(start, "start", n, device),
                                        vector(counts, "counts", n, device), vector(new_lens, "new_lens", n, device),
                                        _s._on(stream, device)), "gemm_kv_compact")
    return new_lens


def w4_gemm(ctx, a, codes, scales, zeros=None, bias=None, epilogue=0, out=None, stream=None):
    """``act(a @ W.T + bias)`` with 4-bit weights through ``gemm_w4_run``: ``a`` [rows, K] float16 or
    bfloat16, ``codes`` uint8 [N, K / 2] (even columns in the low half of a byte), ``scales`` [N, K /
    group] of ``a``'s type, ``zeros`` uint8 [N, K / group] or None (8): W = (code - zero) * scale, groups
    of 32, 64 or 128 columns. Returns ``out`` (allocated when not given)."""
    dtype, device = a.dtype, a.device
    size, wide = a.shape, scales.shape
    if len(size) != 2 or len(wide) != 2:
        raise ValueError("a [rows, K], codes [N, K / 2] and scales [N, K / group] expected")
    (m, k), (n, groups) = size, wide
    if codes.dtype is not _uint8 or codes.shape != (n, k // 2) or codes.device != device or not codes.is_contiguous():
        raise ValueError(f"codes: a contiguous uint8 tensor of shape {(n, k // 2)} on {device} expected")
    if scales.dtype is not dtype or scales.device != device or not scales.is_contiguous():
        raise ValueError(f"scales: a contiguous tensor of {dtype} on {device} expected")
    if zeros is None:
        zeros_ptr = 0
    elif zeros.dtype is not _uint8 or zeros.shape != wide or zeros.device != device or not zeros.is_contiguous():
        raise ValueError(f"zeros: a contiguous uint8 tensor of shape {(n, groups)} on {device} expected")
    else:
        zeros_ptr = zeros.data_ptr()
    if k and (not groups or k % groups):
        raise ValueError(f"scales: one for each group of the {k} columns expected, got {groups} a row")
    lda, ca = a.stride()
    if ca != 1 and k > 1:
        raise ValueError("a: the values of a row must be contiguous")
    if out is None:
        out, ldc = _s._empty((m, n), dtype, device, stream), n
    elif out.dtype is not dtype or out.shape != (m, n) or out.device != device or (n > 1 and out.stride()[1] != 1):
        raise ValueError(f"out: {m} rows of {n} contiguous values of {dtype} on {device} expected")
    else:
        ldc = out.stride()[0]
    if bias is not None and (bias.dtype is not dtype or bias.shape != (n,) or bias.device != device or not bias.is_contiguous()):
        raise ValueError(f"bias: {n} contiguous values of {dtype} on {device} expected")
    w = _W4.pack(codes.data_ptr(), scales.data_ptr(), zeros_ptr, k // groups if groups else 128)
    _g._check(_s._lib().gemm_w4_run(_g._h(ctx), _s._dtype_code(dtype), m, n, k, a.data_ptr(), lda if m > 1 else k, w,
                                    None if bias is None else bias.data_ptr(), out.data_ptr(), ldc if m > 1 else n, epilogue,
                                    _s._on(stream, device)), "gemm_w4_run")
    return out
