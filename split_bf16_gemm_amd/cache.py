"""The attention part of a decode step: rotary positions, a paged 8-bit cache of keys and
values, attention over it and its pages, over the C ABI of include/lowm_cache.h.

As in ops.py, argument checks and marshalling only (in csrc/ops_binding.cpp); every step runs
in the HIP kernels of liblowm.so, on the caller's current stream (or ``stream``),
asynchronously, and lengths, tables and positions are read on the GPU, so that a captured step
may be replayed after they changed.  There is no fallback.

Sequences.  ``table`` [B, W] int32 lists the pages of each sequence in order, ``lens`` [B] int32
counts its tokens, those of the call itself included.  The rows of a call are those of its
sequences one after another: rows row_starts[b] to row_starts[b + 1] - 1 (int32 [B + 1]) for
sequence b, or as many for each where row_starts is None (one, in a decode step).  The last of a
sequence's rows stands at its last token.  Positions below 0 or past the table, and pages whose
number is not one (-1, say), are left out.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

import torch

from . import ops

PAGE = 64          # tokens of a page
ROTARY_INTERLEAVED, ROTARY_INVERSE = 1, 2

_vp, _i, _l, _f, _size = ops._vp, ops._i, ops._l, ops._f, ops._size


# The argument structs of lowm_cache.h.
class KvCacheArg(ctypes.Structure):
    _fields_ = ops._fields(("k v k_scale v_scale", _vp), ("P H D type layers", _i))


class SequencesArg(ctypes.Structure):
    _fields_ = ops._fields(("table lens row_starts", _vp), ("table_ld", _l), ("B W T", _i))


class RotaryArgs(ctypes.Structure):
    _fields_ = ops._fields(
        ("q k q_out k_out positions freqs", _vp),
        ("q_row q_head k_row k_head q_out_row q_out_head k_out_row k_out_head", _l),
        ("T Hq Hk D R first type positions_bytes flags", _i), ("scale", _f))


class CacheAppendArgs(ctypes.Structure):
    _fields_ = [("cache", KvCacheArg), ("seq", SequencesArg),
                *ops._fields(("k v", _vp), ("k_row k_head v_row v_head", _l), ("type", _i))]


class CacheReadArgs(ctypes.Structure):
    _fields_ = [("cache", KvCacheArg), ("seq", SequencesArg), *ops._fields(("k_out v_out", _vp))]


class CacheAttentionArgs(ctypes.Structure):
    _fields_ = [("cache", KvCacheArg), ("seq", SequencesArg),
                *ops._fields(("q out lse workspace", _vp), ("workspace_bytes", _size),
                             ("q_row q_head", _l), ("Hq window", _i), ("scale", _f))]


class ForkPagesArgs(ctypes.Structure):
    _fields_ = [("cache", KvCacheArg),
                *ops._fields(("table lens parents held table_out lens_out refs_out missing_out "
                              "workspace", _vp), ("workspace_bytes", _size),
                             ("R W reserve", _i))]


class CompactPagesArgs(ctypes.Structure):
    _fields_ = [("cache", KvCacheArg),
                *ops._fields(("table held table_out refs_out counts_out workspace", _vp),
                             ("workspace_bytes", _size), ("R W", _i))]


_lib = None


def library():
    """liblowm.so with the entry points of lowm_cache.h declared."""
    global _lib
    if _lib is None:
        lib = ops.library()
        c = lib.lib
        for name in ("rotary", "cache_append", "cache_read", "cache_attention", "fork_pages",
                     "compact_pages"):
            getattr(c, f"lowm_{name}").argtypes = [_vp, _vp]
        c.lowm_cache_attention_workspace_bytes.argtypes = [_i, _i, _i, _i]
        c.lowm_cache_attention_workspace_bytes.restype = _size
        c.lowm_pages_workspace_bytes.argtypes = [_i, _i, _i]
        c.lowm_pages_workspace_bytes.restype = _size
        _lib = lib
    return _lib


class KVCache(NamedTuple):
    """Keys and values of one layer, a byte an element (int8 or e4m3) with a scale, not negative,
    for each page of 64 tokens and head; or of several layers, with a first dimension more.

    Element d of token t of page p and head h is k[p, h, d // 16, t, d % 16] * k_scale[p, h]
    and v[p, h, t // 16, d, t % 16] * v_scale[p, h]."""
    k: torch.Tensor          # [P, H, D / 16, 64, 16]
    v: torch.Tensor          # [P, H, 4, D, 16]
    k_scale: torch.Tensor    # [P, H] fp32
    v_scale: torch.Tensor

    def layer(self, i: int) -> "KVCache":
        """Layer i of a cache of several."""
        return KVCache(*(x[i] for x in self))


def make_kv_cache(pages: int, heads: int, head_dim: int, *, layers: Optional[int] = None,
                  dtype: torch.dtype = torch.int8, device="cuda") -> KVCache:
    """A zeroed cache (head_dim a multiple of 16, at most 256; dtype int8 or float8_e4m3fn);
    with ``layers`` of that many, whose ``layer(i)`` the calls for one layer take."""
    if head_dim % 16 or not 16 <= head_dim <= 256:
        raise ValueError(f"head_dim must be a multiple of 16 up to 256, not {head_dim}")
    if dtype not in (torch.int8, torch.float8_e4m3fn):
        raise TypeError(f"a cache is int8 or float8_e4m3fn, not {dtype}")
    lead = ((layers,) if layers is not None else ()) + (pages, heads)

    def zeros(*shape):
        return torch.zeros(*lead, *shape, dtype=torch.int8, device=device).view(dtype)

    return KVCache(zeros(head_dim // 16, PAGE, 16), zeros(PAGE // 16, head_dim, 16),
                   torch.zeros(*lead, device=device), torch.zeros(*lead, device=device))


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str = "none",
                       factor: float = 1.0, original_length: int = 8192,
                       low: float = 1.0, high: float = 32.0, device="cuda") -> torch.Tensor:
    """Radians a position of each of a head's rotary_dim / 2 pairs, base^(-2i / rotary_dim), in
    fp64, for contexts ``factor`` times as long as ``original_length``:

    "none"      as they are
    "linear"    all slowed down by factor (positions interpolated)
    "base"      the base raised to base * factor^(R / (R - 2)), so that the slowest pair is
                slowed by factor and the fastest not at all
    "by_parts"  pairs that turn fewer than ``low`` times over original_length slowed by factor,
                those that turn more than ``high`` times kept, the others in between, linearly
                in their turns (a model's own low and high belong here: with a ramp in turns
                often 1 and 4; the defaults 1 and 32 are common with a ramp in the pair's index,
                which this is not)
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even and positive, not {rotary_dim}")
    if not (base > 0 and factor >= 1):
        raise ValueError("base must be positive and factor at least 1")
    if scaling == "base":
        if rotary_dim < 4:
            raise ValueError("scaling 'base' needs two pairs")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    at = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    freqs = base ** (-at / rotary_dim)
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "by_parts":
        if not 0 <= low < high:
            raise ValueError("by_parts needs 0 <= low < high")
        turns = original_length * freqs / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        freqs = freqs * (keep + (1 - keep) / factor)
    elif scaling not in ("none", "base"):
        raise ValueError(f"scaling must be 'none', 'linear', 'base' or 'by_parts', not {scaling!r}")
    return freqs.to(device)


def rotary(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor,
           freqs: torch.Tensor, *, layout: str = "half", first: int = 0, scale: float = 1.0,
           inverse: bool = False, q_out: Optional[torch.Tensor] = None,
           k_out: Optional[torch.Tensor] = None, stream=None):
    """(q', k'): q [T, Hq, D] and k [T, Hk, D] (or None) with the pairs of each head turned by
    positions[t] * freqs[i] and scaled.

    bf16 or fp32, any strides with contiguous rows (columns of a larger buffer).  The
    2 * len(freqs) elements from ``first`` on are turned, in pairs (i, i + len(freqs)) with layout
    "half" or (2i, 2i + 1) with "interleaved"; the others are copied.  positions int64 or int32
    [T]; freqs fp64 (rotary_frequencies), the angle being taken in fp64.  ``inverse`` turns back,
    as a gradient does.  q_out=q, k_out=k work in place."""
    if layout not in ("half", "interleaved"):
        raise ValueError(f"layout must be 'half' or 'interleaved', not {layout!r}")
    dev = q.device
    if q_out is None:
        q_out = ops._empty(q.shape, q.dtype, dev, stream)
    if k is None:
        k_out = None
    elif k_out is None:
        k_out = ops._empty(k.shape, k.dtype, dev, stream)
    rc = (ops._calls or ops._native()).rotary(
        q, q_out, k, k_out, positions, freqs, first,
        (ROTARY_INTERLEAVED if layout == "interleaved" else 0) | (ROTARY_INVERSE if inverse else 0),
        scale, ops._stream(stream, dev))
    if rc:
        library().check(rc)
    return q_out, k_out


def cache_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, table: torch.Tensor,
                 lens: torch.Tensor, *, row_starts: Optional[torch.Tensor] = None, stream=None):
    """Write k, v [T, H, D] (bf16 or fp32, any strides with contiguous rows) into the cache at
    the last positions of their sequences (``lens`` counts them already).

    A page's scale is its largest magnitude / 127 (int8) or / 448 (e4m3).  Where a page already
    holds earlier tokens its scale only grows, and those are then rounded again to the new step.
    A page must be one sequence's own (fork_pages).  Returns nothing."""
    rc = (ops._calls or ops._native()).cache_append(
        k, v, *cache, table, lens, row_starts, ops._stream(stream, k.device))
    if rc:
        library().check(rc)


def cache_read(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, *,
               row_starts: Optional[torch.Tensor] = None, rows: Optional[int] = None,
               k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
               stream=None):
    """(k, v) [T, H, D] bf16: the rows' keys and values as the cache holds them.  T is that of
    the outputs, or ``rows``; without row_starts one row a sequence where neither is given.  Rows
    that are left out are not written."""
    dev = cache.k.device
    if k_out is None:
        if v_out is not None:
            shape = v_out.shape
        else:
            if rows is None and row_starts is not None:
                raise ValueError("with row_starts, cache_read needs rows or outputs: how many "
                                 "rows there are is only known on the GPU")
            T = rows if rows is not None else table.shape[0]
            shape = (T, cache.k.shape[1], cache.v.shape[3])
        k_out = ops._empty(shape, torch.bfloat16, dev, stream)
    if v_out is None:
        v_out = ops._empty(k_out.shape, torch.bfloat16, dev, stream)
    rc = (ops._calls or ops._native()).cache_read(
        k_out, v_out, *cache, table, lens, row_starts, ops._stream(stream, dev))
    if rc:
        library().check(rc)
    return k_out, v_out


def make_cache_attention_workspace(T: int, q_heads: int, heads: int, head_dim: int,
                                   device="cuda") -> Optional[torch.Tensor]:
    """A zeroed workspace of cache_attention for T rows (None for sizes it rejects); it serves
    any sizes that need no more bytes, one call at a time, but no other operator."""
    n = library().lib.lowm_cache_attention_workspace_bytes(T, q_heads, heads, head_dim)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def cache_attention(q: torch.Tensor, cache: KVCache, table: torch.Tensor, lens: torch.Tensor, *,
                    row_starts: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                    window: int = 0, workspace: Optional[torch.Tensor],
                    out: Optional[torch.Tensor] = None, lse_out: Optional[torch.Tensor] = None,
                    stream=None):
    """(out [T, Hq, D], lse [T, Hq]) of the rows q [T, Hq, D] (bf16, any strides with contiguous
    rows) over their sequences' cache; query head h reads head h // (Hq // H).

    A row at position p sees tokens 0 to p, or with ``window`` the last ``window`` of them; scores
    are q . k * scale (default D ** -0.5).  out is bf16; lse, the logarithm of the sum of e^score
    in fp32, is written where lse_out is given (else None comes back).  A row that sees nothing
    has out 0 and lse -inf.  workspace: make_cache_attention_workspace."""
    dev = q.device
    if out is None:
        out = ops._empty(q.shape, torch.bfloat16, dev, stream)
    rc = (ops._calls or ops._native()).cache_attention(
        q, *cache, table, lens, row_starts, out, lse_out, workspace, window,
        q.shape[-1] ** -0.5 if scale is None else scale, ops._stream(stream, dev))
    if rc:
        library().check(rc)
    return out, lse_out


def make_pages_workspace(rows: int, width: int, pages: int,
                         device="cuda") -> Optional[torch.Tensor]:
    """A workspace of fork_pages and compact_pages for tables [rows, width] and caches of that
    many pages (None for sizes they reject); it needs no clearing and serves one call at a time."""
    n = library().lib.lowm_pages_workspace_bytes(rows, width, pages)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _ints(shape, dev, stream):
    return ops._empty(shape, torch.int32, dev, stream)


def fork_pages(cache: KVCache, table: torch.Tensor, lens: torch.Tensor,
               parents: Optional[torch.Tensor] = None, *, reserve: int = 0,
               held: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor],
               outs=None, stream=None):
    """(table', lens', refs, missing): the sequences of the next step.  Row r goes on as
    parents[r] (int32 [R]; None: itself), or ends, its pages freed, where that is -1.

    Rows share their parent's pages; of the rows that take over an unfinished last page one keeps
    it and the others get copies (in every layer of ``cache``), and a row that goes on gets pages
    for ``reserve`` more tokens.  New pages are the lowest that are in no row and not held (held
    int32 [P]: pages with a value > 0 are someone else's).  refs [P] counts the uses of each page.
    missing [1] counts the pages that were not to be had (-1 in the table); tokens appended there
    are lost, and as long as such a page is a row's unfinished last one every call counts it.  A
    row that ended has length 0, and begins anew from there: add a step's token to the lengths of
    those that go on only.  ``outs``: four tensors to write into, none of them an input."""
    dev = table.device
    if outs is None:
        outs = (_ints(table.shape, dev, stream), _ints(lens.shape, dev, stream),
                _ints(cache.k.shape[-5:-4], dev, stream), _ints((1,), dev, stream))
    rc = (ops._calls or ops._native()).fork_pages(
        *cache, table, lens, parents, held, *outs, workspace, reserve, ops._stream(stream, dev))
    if rc:
        library().check(rc)
    return tuple(outs)


def compact_pages(cache: KVCache, table: torch.Tensor, *, held: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor], outs=None, stream=None):
    """(table', refs, counts): the highest pages in use moved to the lowest free ones, in every
    layer of ``cache``, while those are lower; held pages stay.  counts [2]: pages moved, and one
    more than the highest page still in use.  ``outs``: three tensors to write into, none of them
    an input."""
    dev = table.device
    if outs is None:
        outs = (_ints(table.shape, dev, stream), _ints(cache.k.shape[-5:-4], dev, stream),
                _ints((2,), dev, stream))
    rc = (ops._calls or ops._native()).compact_pages(
        *cache, table, held, *outs, workspace, ops._stream(stream, dev))
    if rc:
        library().check(rc)
    return tuple(outs)
