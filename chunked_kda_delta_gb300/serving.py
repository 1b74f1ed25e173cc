"""The serving operators: page operations, the 8-bit key/value cache with its attention, and
beam selection (``include/kda.h``).

Thin wrappers of the extension ``_build/_kda_serving.so``, which checks the tensors, allocates what
is returned and calls the C ABI, asynchronously on the given (or current) stream; every step runs
in the library's CUDA kernels and there is no fallback.  Calls in a row: appending one token to 256
rows 5.2 us, a selection of 4 from 4 beams 8.2, a fork of a cache's tables 14.7 (GB300); with this
marshalling in Python and ctypes, where the host was the bound, 13.0, 25.3 and 33.9.
Results and scratch are torch's memory of the call's stream: inside ``torch.cuda.graph`` they belong to
the graph, and no call is needed before it.  (A capture begun without torch has to keep to the C
ABI: torch does not hold memory for it.)
What only a kernel can see (page numbers out of range, too few free pages, values that are not
finite) goes to the device status word: :func:`~.kda.kda_get_device_status`.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os
import threading
from typing import Optional, Sequence

import torch

from . import build as _build
from .kda import KdaError, load_library

_ext = None
_lock = threading.Lock()


def _binding():
    """The extension, loaded at the first call (built by :mod:`chunked_kda_delta_gb300.build`)."""
    global _ext
    if _ext is not None:
        return _ext
    with _lock:
        if _ext is None:
            load_library()
            if not os.path.exists(_build.BINDING_PATH):
                raise KdaError(5, f"extension {_build.BINDING_PATH} is missing; build it with "
                                  "`python -m chunked_kda_delta_gb300.build`")
            loader = importlib.machinery.ExtensionFileLoader("_kda_serving", _build.BINDING_PATH)
            spec = importlib.util.spec_from_loader("_kda_serving", loader)
            module = importlib.util.module_from_spec(spec)
            loader.exec_module(module)
            _ext = module
    return _ext


def _handle(stream):
    """A raw stream handle; None is the current stream of the tensors' device."""
    if stream is None:
        return None
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def kda_pages_alloc(tables: torch.Tensor, refs: torch.Tensor, want: torch.Tensor,
                    new_tables: Optional[torch.Tensor] = None,
                    new_refs: Optional[torch.Tensor] = None, stream=None):
    """Gives row r at least ``want[r]`` pages; returns ``(new_tables, new_refs)``.

    ``tables``: int32 ``[rows, width]`` (-1: no page); ``refs``: int32 ``[pages]``, references
    to each page; ``want``: int32 ``[rows]``.  Free pages go out lowest first.  With too few of
    them entries stay -1 and the status word says ``KDA_ERR_NO_FREE_PAGE``.
    """
    return (_ext or _binding()).pages_alloc(tables, refs, want, new_tables, new_refs, _handle(stream))


def kda_pages_free(tables: torch.Tensor, refs: torch.Tensor, drop: torch.Tensor,
                   new_tables: Optional[torch.Tensor] = None,
                   new_refs: Optional[torch.Tensor] = None, stream=None):
    """Drops the rows where ``drop`` (bool or uint8 ``[rows]``) is set; returns
    ``(new_tables, new_refs)``."""
    return (_ext or _binding()).pages_free(tables, refs, drop, new_tables, new_refs, _handle(stream))


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
    return (_ext or _binding()).pages_fork(tables, refs, parents, lens, page_tokens, pools,
                                           bool(layers_first), new_tables, new_refs, _handle(stream))


def kda_pages_compact(tables: torch.Tensor, refs: torch.Tensor,
                      pools: Sequence[torch.Tensor] = (), layers_first: bool = False,
                      new_tables: Optional[torch.Tensor] = None,
                      new_refs: Optional[torch.Tensor] = None, stream=None):
    """Moves the pages in use to the front of the pools.

    Returns ``(new_tables, new_refs, page_map, num_live)``: ``page_map`` (int32 ``[pages]``) has
    each page's new number (-1: free), ``num_live`` (int32 ``[1]``) how many are in use.
    """
    return (_ext or _binding()).pages_compact(tables, refs, pools, bool(layers_first), new_tables,
                                              new_refs, _handle(stream))


def kda_pages_copy(src: torch.Tensor, dst: torch.Tensor, pools: Sequence[torch.Tensor],
                   layers_first: bool = False, stream=None) -> None:
    """Copies page ``src[i]`` to page ``dst[i]`` (int32, negative: skipped) in every pool.

    No page may be the destination of two pairs, or of one and the source of another.
    """
    (_ext or _binding()).pages_copy(src, dst, pools, bool(layers_first), _handle(stream))


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
    (_ext or _binding()).kvcache_append(k, v, k_codes, v_codes, k_scale, v_scale, tables, lens,
                                        cu_tokens, _handle(stream))


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
    return (_ext or _binding()).kvcache_attention(q, k_codes, v_codes, k_scale, v_scale, tables, lens,
                                                  cu_tokens, scale, out, _handle(stream))


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
    return (_ext or _binding()).beam_select(logits, scores, num_out, done, eos, _handle(stream))
