"""The serving operators: page operations, the 8-bit key/value cache with its attention, penalties on
logits and beam selection (``include/kda.h``).

Thin wrappers of the extension ``_build/_kda_serving.so``, which checks the tensors, allocates what
is returned and calls the C ABI, asynchronously on the given (or current) stream; every step runs
in the library's CUDA kernels and there is no fallback.  Calls in a row: appending one token to 256
rows 5.2 us, with rotation 7.5, a selection of 4 from 4 beams 8.2, a fork of a cache's tables 14.7 (GB300); with this
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


def kda_kvcache_append_rotary(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rotary: torch.Tensor,
                              k_codes: torch.Tensor, v_codes: torch.Tensor, k_scale: torch.Tensor,
                              v_scale: torch.Tensor, tables: torch.Tensor, lens: torch.Tensor,
                              cu_tokens: Optional[torch.Tensor] = None,
                              positions: Optional[torch.Tensor] = None, interleaved: bool = False,
                              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """:func:`kda_kvcache_append` with the rotation of positions on the way; returns the rotated q.

    q: ``[tokens, q_heads, head_dim]`` of k's type; ``rotary``: fp32 ``[positions, rotary_dim]``, a
    position's ``rotary_dim / 2`` cosines and then as many sines (any scaling of angles is in there);
    rotary_dim: a multiple of 16 up to head_dim, channels past it stay as they are.  Pairs lie
    rotary_dim / 2 apart, or side by side with ``interleaved``.  ``positions`` (int32 ``[tokens]``):
    each token's row of ``rotary``; without it its place in the cache.  ``out`` may be q itself, and
    may have a token stride of its own.
    """
    return (_ext or _binding()).kvcache_append_rotary(q, k, v, rotary, k_codes, v_codes, k_scale, v_scale, tables, lens,
                                                      cu_tokens, positions, interleaved, out, _handle(stream))


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


def kda_kvcache_attention_shared(q: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor,
                                 k_scale: torch.Tensor, v_scale: torch.Tensor, tables: torch.Tensor,
                                 lens: torch.Tensor, cu_rows: torch.Tensor,
                                 cu_tokens: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                                 out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """:func:`kda_kvcache_attention` for rows that share prefixes; returns ``out``.

    Rows ``cu_rows[g]`` to ``cu_rows[g + 1] - 1`` (int32 ``[groups + 1]``) are a group, a request's beams
    or the users of one system prompt: the keys that all of them have in the same pages (as
    :func:`kda_pages_fork` leaves them) are gone through once for the group.  The result is the same for
    any groups.  Where the sizes say that nothing is to be gained (tables with few places, as many groups as rows)
    nothing is shared, and ``cu_rows`` not read.  The tables' width counts there, not the rows' lengths: for short
    rows in wide tables :func:`kda_kvcache_attention` is faster (64 groups of 4 rows of 500 keys in tables for
    131072, 64 heads over 8: 74 us against 172).
    """
    return (_ext or _binding()).kvcache_attention_shared(q, k_codes, v_codes, k_scale, v_scale, tables, lens,
                                                         cu_tokens, scale, out, _handle(stream), cu_rows)


def kda_logits_penalize(logits: torch.Tensor, history: Optional[torch.Tensor] = None, lens: Optional[torch.Tensor] = None,
                        prompt_lens: Optional[torch.Tensor] = None, repetition: Optional[torch.Tensor] = None,
                        presence: Optional[torch.Tensor] = None, frequency: Optional[torch.Tensor] = None,
                        bias_tokens: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                        mask: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Penalties for repeated tokens, biases and a grammar's mask on logits; returns ``out``.

    logits: fp32, bf16 or fp16 ``[..., vocab]`` (what :func:`kda_beam_select` takes), R rows in all.  The
    others have R rows in one leading dimension, or logits' leading ones:
    ``history`` (int32 ``[R, width]``), each row's tokens, prompt first, ``lens`` of them (default: width)
    with ``prompt_lens`` of the prompt (default: 0; taken as the nearest of 0 to the row's length), negative
    tokens skipped; ``repetition`` (fp32 ``[R]``)
    divides positive and multiplies other logits of tokens in the history; ``frequency`` times how
    often, plus ``presence`` if, a token is in the history behind the prompt is taken off; ``bias`` (fp32
    ``[R, n]``) is added to the logits of ``bias_tokens`` (int32 ``[R, n]``), of one token several times
    too; ``mask`` (int32 ``[R, words]``): tokens whose bit ``t % 32`` of word ``t // 32`` is 0 get -inf.
    ``out`` may be logits itself: only what changes is written then.
    """
    return (_ext or _binding()).logits_penalize(logits, history, lens, prompt_lens, repetition, presence, frequency, bias_tokens,
                                                bias, mask, out, _handle(stream))


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
