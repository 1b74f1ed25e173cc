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

from .kda import KdaKvCache, KdaPageShape, KdaPool, _check, load_library

_ACT_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_LOGIT_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_I32, _F32 = torch.int32, torch.float32
_BYTES = (torch.bool, torch.uint8)
_CODES = (torch.float8_e4m3fn, torch.uint8)

# These calls are shorter on the GPU than on the host in a decoding step, so the marshalling is
# kept lean: no context manager where the device is current already, the raw stream handle.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(device.index)
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _run(function, device, *args):
    """Calls `function` with `device` current."""
    if torch.cuda.current_device() == device.index:
        status = function(*args)
    else:
        with torch.cuda.device(device):
            status = function(*args)
    if status:
        _check(load_library(), status)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _vector(name, t, dtypes, shape, device):
    """A contiguous tensor of one of these types and exactly this shape on `device`."""
    if (t.dtype in dtypes if type(dtypes) is tuple else t.dtype is dtypes) and t.shape == shape \
            and t.device == device and t.is_contiguous():
        return
    if type(dtypes) is not tuple:
        dtypes = (dtypes,)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be a contiguous {dtypes[0]} tensor on {device}")


def _pages(tables, refs):
    shape, device = tables.shape, tables.device
    if device.type != "cuda":
        raise ValueError("tables must be on cuda")
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError("tables must be [rows, width]")
    pages = refs.shape
    if len(pages) != 1:
        raise ValueError("refs must be [pages]")
    _vector("tables", tables, _I32, shape, device)
    _vector("refs", refs, _I32, pages, device)
    return KdaPageShape(shape[0], shape[1], pages[0])


def _results(tables, refs, new_tables, new_refs):
    if new_tables is None:
        new_tables = torch.empty_like(tables)
    else:
        _vector("new_tables", new_tables, _I32, tables.shape, tables.device)
    if new_refs is None:
        new_refs = torch.empty_like(refs)
    else:
        _vector("new_refs", new_refs, _I32, refs.shape, refs.device)
    return new_tables, new_refs


def _pools(pools: Sequence[torch.Tensor], pages: int, device, layers_first: bool):
    """Pools as the ABI takes them: [pages, ...] tensors, or [layers, pages, ...] ones."""
    if isinstance(pools, torch.Tensor):
        raise ValueError("pools must be a sequence of tensors")
    lead = 1 if layers_first else 0
    table = (KdaPool * max(1, len(pools)))()
    for i, t in enumerate(pools):
        shape, stride = t.shape, t.stride()
        if t.device != device or len(shape) <= lead or shape[lead] != pages:
            raise ValueError(f"a pool must be a tensor on {device} with {pages} pages in dim {lead}")
        inner = 1
        for dim in range(len(shape) - 1, lead, -1):
            if shape[dim] != 1 and stride[dim] != inner:
                raise ValueError("the pages of a pool must be contiguous")
            inner *= shape[dim]
        elem = t.element_size()
        inner *= elem
        step = stride[lead] * elem
        table[i] = KdaPool(t.data_ptr(), inner, max(step, inner) if pages <= 1 else step,
                           stride[0] * elem if layers_first else 0, shape[0] if layers_first else 1)
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
    _vector("want", want, _I32, (shape.rows,), tables.device)
    new_tables, new_refs = _results(tables, refs, new_tables, new_refs)
    _run(lib.kda_pages_alloc, tables.device, ctypes.byref(shape), _ptr(tables), _ptr(refs),
         _ptr(want), _ptr(new_tables), _ptr(new_refs), _stream(stream, tables.device))
    return new_tables, new_refs


def kda_pages_free(tables: torch.Tensor, refs: torch.Tensor, drop: torch.Tensor,
                   new_tables: Optional[torch.Tensor] = None,
                   new_refs: Optional[torch.Tensor] = None, stream=None):
    """Drops the rows where ``drop`` (bool or uint8 ``[rows]``) is set; returns
    ``(new_tables, new_refs)``."""
    lib = load_library()
    shape = _pages(tables, refs)
    _vector("drop", drop, _BYTES, (shape.rows,), tables.device)
    new_tables, new_refs = _results(tables, refs, new_tables, new_refs)
    _run(lib.kda_pages_free, tables.device, ctypes.byref(shape), _ptr(tables), _ptr(refs),
         _ptr(drop), _ptr(new_tables), _ptr(new_refs), _stream(stream, tables.device))
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
    _vector("parents", parents, _I32, (shape.rows,), tables.device)
    if page_tokens > 0 and lens is None:
        raise ValueError("lens is needed with page_tokens")
    if lens is not None:
        _vector("lens", lens, _I32, (shape.rows,), tables.device)
    table = _pools(pools, shape.pages, tables.device, layers_first)
    new_tables, new_refs = _results(tables, refs, new_tables, new_refs)
    _run(lib.kda_pages_fork, tables.device, ctypes.byref(shape), _ptr(tables), _ptr(refs),
         _ptr(parents), _ptr(lens), int(page_tokens), table, len(pools), _ptr(new_tables),
         _ptr(new_refs), _stream(stream, tables.device))
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
    _run(lib.kda_pages_compact, tables.device, ctypes.byref(shape), _ptr(tables), _ptr(refs),
         table, len(pools), _ptr(new_tables), _ptr(new_refs), _ptr(page_map), _ptr(num_live),
         _stream(stream, tables.device))
    return new_tables, new_refs, page_map, num_live


def kda_pages_copy(src: torch.Tensor, dst: torch.Tensor, pools: Sequence[torch.Tensor],
                   layers_first: bool = False, stream=None) -> None:
    """Copies page ``src[i]`` to page ``dst[i]`` (int32, negative: skipped) in every pool.

    No page may be the destination of two pairs, or of one and the source of another.
    """
    lib = load_library()
    if src.device.type != "cuda" or src.dim() != 1:
        raise ValueError("src must be [count] on cuda")
    _vector("src", src, _I32, src.shape, src.device)
    _vector("dst", dst, _I32, src.shape, src.device)
    if len(pools) == 0:
        return
    lead = 1 if layers_first else 0
    pages = pools[0].shape[lead] if pools[0].dim() > lead else -1
    table = _pools(pools, pages, src.device, layers_first)
    _run(lib.kda_pages_copy, src.device, pages, src.shape[0], _ptr(src), _ptr(dst), table,
         len(pools), _stream(stream, src.device))


def _cache(k_codes, v_codes, k_scale, v_scale, tables, lens, cu_tokens):
    device, shape = k_codes.device, k_codes.shape
    if device.type != "cuda":
        raise ValueError("k_codes must be on cuda")
    if len(shape) != 4:
        raise ValueError("k_codes must be [pages, heads, page_tokens, head_dim]")
    pages, heads, page_tokens, dim = shape
    _vector("k_codes", k_codes, _CODES, shape, device)
    _vector("v_codes", v_codes, _CODES, shape, device)
    scales = (pages, heads)
    _vector("k_scale", k_scale, _F32, scales, device)
    _vector("v_scale", v_scale, _F32, scales, device)
    table = tables.shape
    if len(table) != 2 or table[1] < 1:
        raise ValueError("tables must be [rows, width]")
    _vector("tables", tables, _I32, table, device)
    rows, width = table
    _vector("lens", lens, _I32, (rows,), device)
    if cu_tokens is not None:
        _vector("cu_tokens", cu_tokens, _I32, (rows + 1,), device)
    return KdaKvCache(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                      pages, page_tokens, heads, dim, tables.data_ptr(), rows, width), device, heads, dim


def _act(name, t, heads, dim, device):
    """[tokens, heads, head_dim] with contiguous heads; returns tokens, heads, token stride."""
    shape = t.shape
    if t.dtype not in _ACT_DTYPES or t.device != device:
        raise ValueError(f"{name} must be bf16 or fp16 on {device}")
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, {heads if heads else 'heads'}, {dim}]")
    tokens, heads, _ = shape
    stride = t.stride()
    if tokens and heads and (stride[2] != 1 or (heads > 1 and stride[1] != dim)):
        raise ValueError(f"the heads of {name} must be contiguous")
    return tokens, heads, stride[0] if tokens > 1 else heads * dim


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
    cache, device, heads, dim = _cache(k_codes, v_codes, k_scale, v_scale, tables, lens, cu_tokens)
    if k.dtype is not v.dtype or k.shape != v.shape:
        raise ValueError("k and v must have the same type and shape")
    tokens, _, ks = _act("k", k, heads, dim, device)
    _, _, vs = _act("v", v, heads, dim, device)
    _run(lib.kda_kvcache_append, device, ctypes.byref(cache), k.data_ptr(), v.data_ptr(),
         _ACT_DTYPES[k.dtype], ks, vs, tokens, lens.data_ptr(), _ptr(cu_tokens),
         _stream(stream, device))


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
    cache, device, _, dim = _cache(k_codes, v_codes, k_scale, v_scale, tables, lens, cu_tokens)
    tokens, heads, qs = _act("q", q, None, dim, device)
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=q.dtype, device=device)
        os_ = heads * dim
    else:
        if out.dtype is not q.dtype or out.shape != q.shape:
            raise ValueError("out must have q's type and shape")
        os_ = _act("out", out, heads, dim, device)[2]
    _run(lib.kda_kvcache_attention, device, ctypes.byref(cache), q.data_ptr(), heads,
         _ACT_DTYPES[q.dtype], qs, tokens, lens.data_ptr(), _ptr(cu_tokens),
         dim ** -0.5 if scale is None else scale, out.data_ptr(), os_, _stream(stream, device))
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
    device, shape = logits.device, logits.shape
    if device.type != "cuda" or len(shape) != 3 or logits.dtype not in _LOGIT_DTYPES:
        raise ValueError("logits must be fp32, bf16 or fp16 [batch, beams, vocab] on cuda")
    batch, beams, vocab = shape
    steps = logits.stride()
    stride = steps[1] if beams > 1 else steps[0] if batch > 1 else vocab
    if batch and beams and ((vocab > 1 and steps[2] != 1) or (batch > 1 and steps[0] != beams * stride)):
        raise ValueError("logits must have contiguous rows at one stride")
    rows = (batch, beams)
    _vector("scores", scores, _F32, rows, device)
    if done is not None:
        _vector("done", done, _BYTES, rows, device)
    k = beams if num_out is None else int(num_out)
    if k < 1:
        raise ValueError("num_out must be at least 1")
    size = (batch, k)
    new_scores = torch.empty(size, dtype=_F32, device=device)
    tokens = torch.empty(size, dtype=_I32, device=device)
    parents = torch.empty(size, dtype=_I32, device=device)
    new_done = None if done is None else torch.empty(size, dtype=done.dtype, device=device)
    _run(lib.kda_beam_select, device, batch, beams, vocab, k, logits.data_ptr(),
         _LOGIT_DTYPES[logits.dtype], stride, scores.data_ptr(), _ptr(done), eos,
         new_scores.data_ptr(), tokens.data_ptr(), parents.data_ptr(), _ptr(new_done),
         _stream(stream, device))
    return (new_scores, tokens, parents) if done is None else (new_scores, tokens, parents, new_done)
