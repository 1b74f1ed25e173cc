"""Binding of the serving operators: page operations, the 8-bit key/value cache with its
attention, and beam selection (``include/kda.h``).

Argument marshalling only, as in :mod:`chunked_kda_delta_gb300.kda`: every step runs in the
library's CUDA kernels, asynchronously on the given (or current) stream, and there is no
fallback.  What only a kernel can see (page numbers out of range, too few free pages, values
that are not finite) goes to the device status word: :func:`~.kda.kda_get_device_status`.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from .kda import KdaKvCache, KdaPageShape, KdaPool, _check, _ptr, load_library

_ACT_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_LOGIT_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device).cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    return ctypes.c_void_p(int(stream))


def _vector(name, t, dtypes, shape, device):
    """A contiguous tensor of one of these types and exactly this shape on `device`."""
    if not isinstance(dtypes, tuple):
        dtypes = (dtypes,)
    if t.dtype not in dtypes or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtypes[0]} tensor on {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _pages(tables, refs):
    if tables.device.type != "cuda":
        raise ValueError("tables must be on cuda")
    if tables.dim() != 2 or tables.shape[1] < 1:
        raise ValueError("tables must be [rows, width]")
    if refs.dim() != 1:
        raise ValueError("refs must be [pages]")
    _vector("tables", tables, torch.int32, tables.shape, tables.device)
    _vector("refs", refs, torch.int32, refs.shape, tables.device)
    return KdaPageShape(tables.shape[0], tables.shape[1], refs.shape[0])


def _results(tables, refs, new_tables, new_refs):
    for name, t, like in (("new_tables", new_tables, tables), ("new_refs", new_refs, refs)):
        if t is not None:
            _vector(name, t, torch.int32, like.shape, like.device)
    return (torch.empty_like(tables) if new_tables is None else new_tables,
            torch.empty_like(refs) if new_refs is None else new_refs)


def _pools(pools: Sequence[torch.Tensor], pages: int, device, layers_first: bool):
    """Pools as the ABI takes them: [pages, ...] tensors, or [layers, pages, ...] ones."""
    if isinstance(pools, torch.Tensor):
        raise ValueError("pools must be a sequence of tensors")
    lead = 1 if layers_first else 0
    table = (KdaPool * max(1, len(pools)))()
    for x, t in zip(table, pools):
        if t.device != device or t.dim() <= lead or t.shape[lead] != pages:
            raise ValueError(f"a pool must be a tensor on {device} with {pages} pages in dim {lead}")
        inner = 1
        for size, stride in zip(reversed(t.shape[lead + 1:]), reversed(t.stride()[lead + 1:])):
            if size != 1 and stride != inner:
                raise ValueError("the pages of a pool must be contiguous")
            inner *= size
        elem = t.element_size()
        x.base, x.page_bytes, x.page_stride = t.data_ptr(), inner * elem, t.stride(lead) * elem
        if pages <= 1:
            x.page_stride = max(x.page_stride, x.page_bytes)
        x.layers = t.shape[0] if layers_first else 1
        x.layer_stride = t.stride(0) * elem if layers_first else 0
    return table


def kda_pages_alloc(tables: torch.Tensor, refs: torch.Tensor, want: torch.Tensor,
                    new_tables: Optional[torch.Tensor] = None,
                    new_refs: Optional[torch.Tensor] = None, stream=None):
    """Gives row r at least ``want[r]`` pages; returns ``(new_tables, new_refs)``.

    ``tables``: int32 ``[rows, width]`` (-1: no page); ``refs``: int32 ``[pages]``, references
    to each page; ``want``: int32 ``[rows]``.  Free pages go out lowest first.  With too few of
    them entries stay -1 and the status word says ``KDA_ERR_NO_FREE_PAGE``.
    """
    lib = load_library()
    shape = _pages(tables, refs)
    _vector("want", want, torch.int32, (shape.rows,), tables.device)
    new_tables, new_refs = _results(tables, refs, new_tables, new_refs)
    with torch.cuda.device(tables.device):
        _check(lib, lib.kda_pages_alloc(ctypes.byref(shape), _ptr(tables), _ptr(refs), _ptr(want),
                                        _ptr(new_tables), _ptr(new_refs),
                                        _stream(stream, tables.device)))
    return new_tables, new_refs


def kda_pages_free(tables: torch.Tensor, refs: torch.Tensor, drop: torch.Tensor,
                   new_tables: Optional[torch.Tensor] = None,
                   new_refs: Optional[torch.Tensor] = None, stream=None):
    """Drops the rows where ``drop`` (bool or uint8 ``[rows]``) is set; returns
    ``(new_tables, new_refs)``."""
    lib = load_library()
    shape = _pages(tables, refs)
    _vector("drop", drop, (torch.bool, torch.uint8), (shape.rows,), tables.device)
    new_tables, new_refs = _results(tables, refs, new_tables, new_refs)
    with torch.cuda.device(tables.device):
        _check(lib, lib.kda_pages_free(ctypes.byref(shape), _ptr(tables), _ptr(refs), _ptr(drop),
                                       _ptr(new_tables), _ptr(new_refs),
                                       _stream(stream, tables.device)))
    return new_tables, new_refs


def kda_pages_fork(tables: torch.Tensor, refs: torch.Tensor, parents: torch.Tensor,
                   lens: Optional[torch.Tensor] = None, page_tokens: int = 0,
                   pools: Sequence[torch.Tensor] = (), layers_first: bool = False,
                   new_tables: Optional[torch.Tensor] = None,
                   new_refs: Optional[torch.Tensor] = None, stream=None):
    """Row r continues row ``parents[r]`` (-1: it ends); returns ``(new_tables, new_refs)``.

    Pages that ``lens[parent]`` tokens fill (``page_tokens`` each) are shared; the others
    become private to each row: its parent's page for the first row that continues it, the
    next free page with a copy of the contents in every pool for the others.  ``page_tokens``
    0 (recurrent states): every page is private.  ``pools``: tensors ``[pages, ...]``, or
    ``[layers, pages, ...]`` with ``layers_first``, of any type; their copies are made in place.
    """
    lib = load_library()
    shape = _pages(tables, refs)
    _vector("parents", parents, torch.int32, (shape.rows,), tables.device)
    if page_tokens > 0 and lens is None:
        raise ValueError("lens is needed with page_tokens")
    if lens is not None:
        _vector("lens", lens, torch.int32, (shape.rows,), tables.device)
    table = _pools(pools, shape.pages, tables.device, layers_first)
    new_tables, new_refs = _results(tables, refs, new_tables, new_refs)
    with torch.cuda.device(tables.device):
        _check(lib, lib.kda_pages_fork(ctypes.byref(shape), _ptr(tables), _ptr(refs),
                                       _ptr(parents), _ptr(lens), int(page_tokens), table,
                                       len(pools), _ptr(new_tables), _ptr(new_refs),
                                       _stream(stream, tables.device)))
    return new_tables, new_refs


def kda_pages_compact(tables: torch.Tensor, refs: torch.Tensor,
                      pools: Sequence[torch.Tensor] = (), layers_first: bool = False,
                      new_tables: Optional[torch.Tensor] = None,
                      new_refs: Optional[torch.Tensor] = None, stream=None):
    """Moves the pages in use to the front of the pools.

    Returns ``(new_tables, new_refs, page_map, num_live)``: ``page_map`` (int32 ``[pages]``) has
    each page's new number (-1: free), ``num_live`` (int32 ``[1]``) how many are in use.
    """
    lib = load_library()
    shape = _pages(tables, refs)
    table = _pools(pools, shape.pages, tables.device, layers_first)
    new_tables, new_refs = _results(tables, refs, new_tables, new_refs)
    page_map = torch.empty_like(refs)
    num_live = torch.empty(1, dtype=torch.int32, device=refs.device)
    with torch.cuda.device(tables.device):
        _check(lib, lib.kda_pages_compact(ctypes.byref(shape), _ptr(tables), _ptr(refs), table,
                                          len(pools), _ptr(new_tables), _ptr(new_refs),
                                          _ptr(page_map), _ptr(num_live),
                                          _stream(stream, tables.device)))
    return new_tables, new_refs, page_map, num_live


def kda_pages_copy(src: torch.Tensor, dst: torch.Tensor, pools: Sequence[torch.Tensor],
                   layers_first: bool = False, stream=None) -> None:
    """Copies page ``src[i]`` to page ``dst[i]`` (int32, negative: skipped) in every pool.

    No page may be the destination of two pairs, or of one and the source of another.
    """
    lib = load_library()
    if src.device.type != "cuda" or src.dim() != 1:
        raise ValueError("src must be [count] on cuda")
    _vector("src", src, torch.int32, src.shape, src.device)
    _vector("dst", dst, torch.int32, src.shape, src.device)
    if len(pools) == 0:
        return
    lead = 1 if layers_first else 0
    pages = pools[0].shape[lead] if pools[0].dim() > lead else -1
    table = _pools(pools, pages, src.device, layers_first)
    with torch.cuda.device(src.device):
        _check(lib, lib.kda_pages_copy(pages, src.shape[0], _ptr(src), _ptr(dst), table,
                                       len(pools), _stream(stream, src.device)))


def _cache(k_codes, v_codes, k_scale, v_scale, tables, lens, cu_tokens):
    device = k_codes.device
    if device.type != "cuda":
        raise ValueError("k_codes must be on cuda")
    if k_codes.dim() != 4:
        raise ValueError("k_codes must be [pages, heads, page_tokens, head_dim]")
    pages, heads, page_tokens, dim = k_codes.shape
    for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
        _vector(name, t, (torch.float8_e4m3fn, torch.uint8), k_codes.shape, device)
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        _vector(name, t, torch.float32, (pages, heads), device)
    if tables.dim() != 2 or tables.shape[1] < 1:
        raise ValueError("tables must be [rows, width]")
    _vector("tables", tables, torch.int32, tables.shape, device)
    rows, width = tables.shape
    _vector("lens", lens, torch.int32, (rows,), device)
    if cu_tokens is not None:
        _vector("cu_tokens", cu_tokens, torch.int32, (rows + 1,), device)
    p = lambda t: t.data_ptr()  # noqa: E731
    return KdaKvCache(p(k_codes), p(v_codes), p(k_scale), p(v_scale), pages, page_tokens, heads, dim,
                      p(tables), rows, width)


def _act(name, t, heads, dim, device):
    """[tokens, heads, head_dim] with contiguous heads; returns the token stride."""
    if t.dtype not in _ACT_DTYPES or t.device != device:
        raise ValueError(f"{name} must be bf16 or fp16 on {device}")
    if t.dim() != 3 or (heads is not None and t.shape[1] != heads) or t.shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, {heads if heads else 'heads'}, {dim}]")
    if t.numel() and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != dim)):
        raise ValueError(f"the heads of {name} must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * dim


def kda_kvcache_append(k: torch.Tensor, v: torch.Tensor, k_codes: torch.Tensor,
                       v_codes: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                       tables: torch.Tensor, lens: torch.Tensor,
                       cu_tokens: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantises new tokens into the paged 8-bit cache, in place.

    k, v: bf16 or fp16 ``[tokens, heads, head_dim]`` (any token stride that is a multiple of 8:
    slices of a fused projection are fine); k_codes, v_codes: ``float8_e4m3fn`` (or uint8)
    ``[pages, heads, page_tokens, head_dim]`` with one fp32 scale per page and head in
    k_scale, v_scale ``[pages, heads]``; tables: int32 ``[rows, width]``; lens: int32
    ``[rows]``, tokens each row holds before the call.  ``cu_tokens`` (int32 ``[rows + 1]``)
    gives each row's share of the new tokens; without it every row has one.
    """
    lib = load_library()
    cache = _cache(k_codes, v_codes, k_scale, v_scale, tables, lens, cu_tokens)
    if k.dtype != v.dtype or k.shape != v.shape:
        raise ValueError("k and v must have the same type and shape")
    ks = _act("k", k, cache.num_kv_heads, cache.head_dim, k_codes.device)
    vs = _act("v", v, cache.num_kv_heads, cache.head_dim, k_codes.device)
    with torch.cuda.device(k_codes.device):
        _check(lib, lib.kda_kvcache_append(ctypes.byref(cache), _ptr(k), _ptr(v),
                                           _ACT_DTYPES[k.dtype], ks, vs, k.shape[0], _ptr(lens),
                                           _ptr(cu_tokens), _stream(stream, k_codes.device)))


def kda_kvcache_attention(q: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor,
                          k_scale: torch.Tensor, v_scale: torch.Tensor, tables: torch.Tensor,
                          lens: torch.Tensor, cu_tokens: Optional[torch.Tensor] = None,
                          scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """Causal attention of each row's newest tokens over the paged 8-bit cache; returns ``out``.

    q: bf16 or fp16 ``[tokens, q_heads, head_dim]``, q_heads a multiple of the cache's heads;
    the cache as in :func:`kda_kvcache_append`, with the new tokens already appended: lens
    counts them too, and a row's n query tokens are its last n.  Tokens that see no key get
    zeros.  ``out`` may have a token stride of its own.
    """
    lib = load_library()
    cache = _cache(k_codes, v_codes, k_scale, v_scale, tables, lens, cu_tokens)
    qs = _act("q", q, None, cache.head_dim, k_codes.device)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    elif out.dtype != q.dtype or out.shape != q.shape:
        raise ValueError("out must have q's type and shape")
    os_ = _act("out", out, q.shape[1], cache.head_dim, k_codes.device)
    if scale is None:
        scale = cache.head_dim ** -0.5
    with torch.cuda.device(k_codes.device):
        _check(lib, lib.kda_kvcache_attention(ctypes.byref(cache), _ptr(q), q.shape[1],
                                              _ACT_DTYPES[q.dtype], qs, q.shape[0], _ptr(lens),
                                              _ptr(cu_tokens), ctypes.c_float(scale), _ptr(out),
                                              os_, _stream(stream, k_codes.device)))
    return out


def kda_beam_select(logits: torch.Tensor, scores: torch.Tensor, num_out: Optional[int] = None,
                    done: Optional[torch.Tensor] = None, eos: int = -1, stream=None):
    """One step of beam search; returns ``(scores, tokens, parents)``, with ``done`` given also
    the new ``done``.

    logits: fp32, bf16 or fp16 ``[batch, beams, vocab]`` (rows may be padded: any stride of the
    beams, the batch in steps of ``beams`` of them); scores: fp32 ``[batch, beams]``, -inf for
    a beam that is not there.  Each request's ``num_out`` (default: beams) best totals
    ``scores + log_softmax(logits)``, best first, ties in the order of beam and token; parents
    are rows ``b * beams + w`` (what :func:`kda_pages_fork` takes).  ``done`` (bool or uint8
    ``[batch, beams]``): finished beams, which continue only with ``eos`` at no cost.
    Places that no candidate is left for get -inf, -1, -1.
    """
    lib = load_library()
    if logits.device.type != "cuda" or logits.dim() != 3 or logits.dtype not in _LOGIT_DTYPES:
        raise ValueError("logits must be fp32, bf16 or fp16 [batch, beams, vocab] on cuda")
    batch, beams, vocab = logits.shape
    device = logits.device
    stride = logits.stride(1) if beams > 1 else logits.stride(0) if batch > 1 else vocab
    if logits.numel() and ((vocab > 1 and logits.stride(2) != 1) or
                           (batch > 1 and logits.stride(0) != beams * stride)):
        raise ValueError("logits must have contiguous rows at one stride")
    _vector("scores", scores, torch.float32, (batch, beams), device)
    if done is not None:
        _vector("done", done, (torch.bool, torch.uint8), (batch, beams), device)
    k = beams if num_out is None else int(num_out)
    if k < 1:
        raise ValueError("num_out must be at least 1")
    new_scores = torch.empty((batch, k), dtype=torch.float32, device=device)
    tokens, parents = (torch.empty((batch, k), dtype=torch.int32, device=device) for _ in range(2))
    new_done = None if done is None else torch.empty((batch, k), dtype=done.dtype, device=device)
    with torch.cuda.device(device):
        _check(lib, lib.kda_beam_select(batch, beams, vocab, k, _ptr(logits),
                                        _LOGIT_DTYPES[logits.dtype], stride, _ptr(scores),
                                        _ptr(done), int(eos), _ptr(new_scores), _ptr(tokens),
                                        _ptr(parents), _ptr(new_done), _stream(stream, device)))
    return (new_scores, tokens, parents) if done is None else (new_scores, tokens, parents, new_done)
