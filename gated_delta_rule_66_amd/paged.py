"""Paged cache operators of libkda.so (the "paged cache" of include/kda.h):
writing new tokens' keys and values into a paged cache, as they are or in 8
bits, reading them back, and the attention of new tokens over the cache.

Argument marshalling only, as in ``mixer.py``, whose conventions hold: bf16 or
fp32 tokens, sequences of one length ([N, T, ...]) or packed ([T_total, ...]
with ``cu_seqlens``), inputs that may be slices of wider projections.

Every call takes the cache as

    k_cache, v_cache   [pages, heads, page_size, D], the tokens' dtype,
                       float8_e4m3fn or int8; pages may be spaced (views of one
                       [pages, 2, heads, page_size, D] buffer)
    block_table        [N, blocks] int32: the page of positions
                       page_size * b .. of each sequence
    seq_lens           [N] int32: positions of each sequence, new tokens included
    k_scale, v_scale   [pages, heads, page_size] float8_e8m0fnu for 8-bit caches

Token t of a sequence's n is at position seq_lens - n + t.  Positions below
zero, and those on pages outside [0, pages), are not there: not written, read as
zeros, attended to by no token.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import kda as _k
from .kda import KDAError, PagedCache, _dtype_code
from .mixer import _INT_MAX, _call, _check, _device, _like, _p, _refuse, _rows, _size, _workspace

_KV = {torch.float32: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2, torch.int8: 3}
_SCALE = torch.float8_e8m0fnu


def _page_stride(t: torch.Tensor, name: str) -> int:
    """Elements between the pages of a cache whose strides are not simply nested."""
    P, H, S, D = t.shape
    st = t.stride()
    if (D != 1 and st[3] != 1) or (S != 1 and st[2] != D) or (H != 1 and st[1] != S * D):
        raise ValueError("%s must be contiguous within its pages" % name)
    return st[0] if P != 1 else H * S * D


def _cache(k_cache, v_cache, block_table, seq_lens, k_scale, v_scale, dev: int) -> PagedCache:
    """The C struct of a call's cache.  (As in the mixer operators, what is right passes by few host steps, which are
    what counts in one-token calls; what is not is named by the slower checks.)"""
    shape, ty = k_cache.shape, k_cache.dtype
    if len(shape) != 4:
        raise ValueError("k_cache is [pages, heads, page_size, D]")
    code = _KV.get(ty)
    if code is None:
        raise ValueError("a cache is bf16, fp32, float8_e4m3fn or int8, got %s" % ty)
    if k_cache.get_device() != dev or v_cache.get_device() != dev or v_cache.shape != shape or v_cache.dtype != ty:
        _refuse(k_cache, "k_cache", shape, ty, dev)
        _refuse(v_cache, "v_cache", shape, ty, dev)
    P, H, S, D = shape
    if P > _INT_MAX or H > _INT_MAX or S > _INT_MAX or D > _INT_MAX:
        raise KDAError(_k.KDA_ERR_UNSUPPORTED, "a cache of shape %s" % (tuple(shape),))
    kst, vst = k_cache.stride(), v_cache.stride()
    inner = (S * D, D, 1)
    ks = kst[0] if kst[1:] == inner else _page_stride(k_cache, "k_cache")
    vs = vst[0] if vst[1:] == inner else _page_stride(v_cache, "v_cache")
    if code >= 2:
        if k_scale is None or v_scale is None:
            raise ValueError("an 8-bit cache needs k_scale and v_scale")
        _check(k_scale, "k_scale", shape[:3], _SCALE, dev)
        _check(v_scale, "v_scale", shape[:3], _SCALE, dev)
        kp, vp = k_scale.data_ptr(), v_scale.data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale belong to 8-bit caches")
    else:
        kp = vp = None
    tshape = block_table.shape
    if len(tshape) != 2:
        raise ValueError("block_table is [N, blocks]")
    N, blocks = tshape
    if block_table.dtype != torch.int32 or block_table.get_device() != dev:
        _refuse(block_table, "block_table", tshape, torch.int32, dev)
    ts, one = block_table.stride()
    if (one != 1 and blocks > 1) or (ts < blocks and N > 1):
        raise ValueError("block_table must have contiguous rows of its own")
    _check(seq_lens, "seq_lens", (N,), torch.int32, dev)
    return PagedCache(code, P, H, S, D, blocks, k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, kp, vp,
                      block_table.data_ptr(), ts, seq_lens.data_ptr())


def _tokens(t: torch.Tensor, name: str, shape, lead: int, dtype, dev: int) -> int:
    """Elements between the token rows of a token tensor, as mixer._rows, which it leaves the unusual ones to."""
    if t.shape == shape and t.dtype == dtype and t.get_device() == dev and t.numel() <= _INT_MAX:
        st = t.stride()
        h, d = shape[lead:]
        if st[lead + 1] == 1 and st[lead] == d:
            if lead == 1:
                row = st[0]
            else:
                n, tokens = shape[:2]
                row = st[1] if tokens != 1 else st[0]
                if n != 1 and tokens != 1 and st[0] != row * tokens:
                    row = -1
            if row >= h * d:
                return row
    return _rows(t, name, shape, lead, dtype, dev)


def _batch(shape, seq_lens, cu_seqlens, dev: int, name: str):
    """(dimensions that count tokens, N, T) of token tensors [N, T, heads, D] or [T_total, heads, D]."""
    lead = 2 if cu_seqlens is None else 1
    if len(shape) != lead + 2:
        raise ValueError("%s is [N, T, heads, D], or [T_total, heads, D] with cu_seqlens" % name)
    N = seq_lens.numel()
    if cu_seqlens is None:
        if shape[0] != N:
            raise ValueError("%s has %d sequences, seq_lens %d" % (name, shape[0], N))
        return lead, N, shape[1]
    _check(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
    return lead, N, shape[0]


def kv_cache_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_table: torch.Tensor, seq_lens: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                   v_scale: Optional[torch.Tensor] = None, *, cu_seqlens: Optional[torch.Tensor] = None) -> None:
    """Writes the new tokens' keys and values, [N, T, heads, D] or packed
    [T_total, heads, D], to their positions in the cache through
    ``kda_kv_cache_write``.  8-bit caches get codes, rounded to nearest even,
    and the exponent of the smallest power of two that takes the row's largest
    magnitude to 448 (e4m3) or 127 (int8); a row with a NaN or an infinity gets
    a NaN scale.  Two tokens of a call must not share a position's row."""
    dev = _device(k)
    c = _cache(k_cache, v_cache, block_table, seq_lens, k_scale, v_scale, dev)
    lead, N, T = _batch(k.shape, seq_lens, cu_seqlens, dev, "k")
    shape = k.shape[:lead] + (c.heads, c.head_dim)
    ks = _tokens(k, "k", shape, lead, k.dtype, dev)
    vs = _tokens(v, "v", shape, lead, k.dtype, dev)
    _call("kda_kv_cache_write", dev, N, _p(cu_seqlens), T, _dtype_code(k.dtype), _p(k), ks, _p(v), vs,
          ctypes.byref(c))


def kv_cache_read(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  k_scale: Optional[torch.Tensor], v_scale: Optional[torch.Tensor], tokens: int, *,
                  dtype: torch.dtype = torch.bfloat16, cu_seqlens: Optional[torch.Tensor] = None,
                  k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None):
    """The last positions of every sequence through ``kda_kv_cache_read``: (k, v)
    [N, tokens, heads, D], or with ``cu_seqlens`` packed [tokens, heads, D], the
    last cu_seqlens[i + 1] - cu_seqlens[i] positions of sequence i.  ``dtype`` is
    bf16 or fp32 (the cache's own unless it has 8 bits); ``k`` and ``v`` may be
    given, and keep their rows behind the last sequence."""
    dev = _device(k_cache)
    c = _cache(k_cache, v_cache, block_table, seq_lens, k_scale, v_scale, dev)
    if not 0 <= tokens <= _INT_MAX:
        raise ValueError("tokens is a count, got %r" % (tokens,))
    shape = (tokens, c.heads, c.head_dim) if cu_seqlens is not None else (seq_lens.numel(), tokens, c.heads, c.head_dim)
    _, N, T = _batch(shape, seq_lens, cu_seqlens, dev, "k")
    code = _dtype_code(dtype)
    out = []
    for name, t in (("k", k), ("v", v)):
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
        else:
            _check(t, name, shape, dtype, dev)
        out.append(t)
    _call("kda_kv_cache_read", dev, N, _p(cu_seqlens), T, code, _p(out[0]), _p(out[1]), ctypes.byref(c))
    return out[0], out[1]


@functools.lru_cache(maxsize=1024)
def _attn_workspace(N, packed, T, H, code, *sizes) -> int:
    """The bytes of a call's workspace, which go by its sizes alone."""
    c = PagedCache(sizes[0], *sizes[1:])
    return _size("kda_paged_attn_workspace_size", N, int(packed), T, H, code, ctypes.byref(c))


def paged_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
               seq_lens: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
               v_scale: Optional[torch.Tensor] = None, *, scale: Optional[float] = None,
               gate: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Attention of new tokens over a paged cache that holds them already,
    through ``kda_paged_attn``:

        o_t = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q_t . k_j),  j up to t's own position

    q: [N, T, H, D], T from one token to whole prompts, or packed
    [T_total, H, D]; the cache's heads divide H.  ``scale`` is D ** -0.5 unless
    given; ``gate`` (like q): o times sigmoid(gate).  Returns o like q.  A token
    without a position to attend to gets zeros; rows of a packed ``out`` behind
    the last sequence are left as they are."""
    dev = _device(q)
    c = _cache(k_cache, v_cache, block_table, seq_lens, k_scale, v_scale, dev)
    lead, N, T = _batch(q.shape, seq_lens, cu_seqlens, dev, "q")
    H = q.shape[-2]
    shape = q.shape[:lead] + (H, c.head_dim)
    code = _dtype_code(q.dtype)
    qs = _tokens(q, "q", shape, lead, q.dtype, dev)
    zs = _tokens(gate, "gate", shape, lead, q.dtype, dev) if gate is not None else qs
    if out is None:
        out = _like(q)
    else:
        _check(out, "out", shape, q.dtype, dev)
    ref = ctypes.byref(c)
    need = _attn_workspace(N, cu_seqlens is not None, T, H, code, c.dt, c.pages, c.heads, c.page_size, c.head_dim,
                           c.blocks)
    workspace, have = _workspace(workspace, need, dev)
    _call("kda_paged_attn", dev, N, _p(cu_seqlens), T, H, code, c.head_dim ** -0.5 if scale is None else float(scale),
          _p(q), qs, _p(gate), zs, _p(out), ref, _p(workspace), have)
    return out
