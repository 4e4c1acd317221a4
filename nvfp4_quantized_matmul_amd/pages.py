"""Pages of the paged cache, kept on the device: which are free, which ones a
sequence has, and sequences that share theirs.

One table and one count serve the caches of all layers: ``table`` int32 [batch,
width] names the pages of each sequence in order (-1: none), ``refs`` int32
[pages] counts the entries that name a page.  A page whose count is not above 0
is free; the caller may count references of its own.  A new table is all -1
with counts 0.  A decode step::

    lens += 1
    nv.kv_free(table, lens, refs, page, keep=window, sinks=sinks)
    waits = nv.kv_reserve(caches, table, lens, refs) > 0
    step = torch.where(waits, 0, lens)
    for cache in caches:
        q = nv.kv_append(k, v, cache, table, step, q=q, inv_freq=inv_freq)
        o = nv.paged_attention(q, cache, table, step, window=window, sinks=sinks)
    lens -= waits.int()

A sequence that got no pages must not be appended to: its entry names no page,
or one that other sequences read too.  With length 0 its new tokens are written
nowhere and see nothing (their rows of o are zeros); its length is taken back,
and the same tokens come again with a later step.  Nothing is read on the host,
so a step can be captured in a graph.
"""

from __future__ import annotations

from typing import Optional, Sequence, Tuple, Union

import torch

from . import NVFP4Error, _check, _on_device, _stream, load_library
from .serving import _I32, _PAGES, _U8, KVCache, _CacheStruct


# As for the operators that a step calls beside these, a call's checks are one
# expression, and what is wrong is worked out only once it fails.

def _refuse(index: int, **tensors: torch.Tensor) -> None:
    """Raises for a tensor that is not contiguous int32 on device `index`, or else for a shape."""
    for name, t in tensors.items():
        if t.dtype is not _I32:
            raise TypeError(f"{name} must be int32, got {t.dtype}")
        if t.get_device() < 0:
            raise ValueError("all tensors must be on the GPU")
        if t.get_device() != index:
            raise ValueError(f"{name} must be on the same GPU as the others")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    raise ValueError("table must be [batch, width], lens [batch] and refs [pages]: got "
                     + ", ".join(f"{name} {tuple(t.shape)}" for name, t in tensors.items()))


def _table(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor) -> Tuple[int, int, int, int]:
    """(device index, batch, width, pages) of a table, lengths and counts, checked."""
    index, shape, pages = table.get_device(), table.shape, refs.shape
    if not (index >= 0 and len(shape) == 2 and len(pages) == 1 and lens.shape == (shape[0],) and table.dtype is _I32
            and lens.dtype is _I32 and refs.dtype is _I32 and lens.get_device() == index == refs.get_device()
            and table.is_contiguous() and lens.is_contiguous() and refs.is_contiguous()):
        _refuse(index, table=table, lens=lens, refs=refs)
    return index, shape[0], shape[1], pages[0]


def _layers(caches: Union[KVCache, Sequence[KVCache]], index: int, pages: int):
    """(first cache, their number, nvfp4_kv_cache_t array), checked."""
    if isinstance(caches, KVCache):
        caches = (caches,)
    count = len(caches)
    if count == 0:
        raise ValueError("there is no cache")
    first = caches[0]
    shape = first._k.shape
    for c in caches:
        if c._index != index or c._k.shape != shape:
            raise ValueError("the caches must be of one shape and on the table's GPU")
    if pages != first._pages:
        raise ValueError(f"refs must have one count for each of the {first._pages} pages, got {pages}")
    return first, count, (_CacheStruct * count)(*[c._struct for c in caches])


def kv_free(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page: int, keep: int = 0,
            sinks: int = 0) -> None:
    """Gives back the pages that hold nothing that is needed.

    table int32 [batch, width] and refs int32 [pages] are changed in place;
    lens int32 [batch]; page: the tokens of a page.  Entry i of a sequence stays
    if its page begins before the sequence's length, and with keep > 0 if
    besides it ends behind the last `keep` tokens' first one or begins before
    `sinks`.  Other entries that name a page become -1 and its count falls.  A
    sequence that has ended has length 0.  A window of w tokens with n new ones
    a step needs keep = w + n - 1.
    """
    index, batch, width, pages = _table(table, lens, refs)
    if page not in _PAGES:
        raise ValueError(f"page must be one of {_PAGES}, got {page}")
    _check("nvfp4_kv_free", _on_device(
        index, load_library().nvfp4_kv_free, table.data_ptr(), batch, width, lens.data_ptr(), page, keep, sinks,
        refs.data_ptr(), pages, _stream(table.device)))


# nvfp4_kv_reserve_workspace_size and nvfp4_kv_compact_workspace_size by call shape
_WS_CACHE: dict = {}


def _workspace(fn: str, *key: int) -> int:
    n = _WS_CACHE.get((fn, key))
    if n is None:
        n = int(getattr(load_library(), fn)(*key))
        if n < 0:
            raise NVFP4Error(fn, n)
        if len(_WS_CACHE) < 4096:
            _WS_CACHE[fn, key] = n
    return n


def kv_reserve(caches: Union[KVCache, Sequence[KVCache]], table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
               cu_q: Optional[torch.Tensor] = None, tokens: Optional[int] = None) -> torch.Tensor:
    """Pages for new tokens; int32 [batch]: 0, or the pages that a sequence lacks.

    caches: one KVCache or those of all layers; table and refs are changed in
    place; lens int32 [batch] with the new tokens, cu_q int32 [batch + 1] their
    rows and `tokens` how many rows there are (default: one token for each
    sequence).  An entry that new tokens reach gets a free page, the lowest
    first, where it names none or one that is named more than once: then its
    contents are copied in all caches if earlier tokens share the page.  Tokens
    behind the table's width have no entry and are left out.  A sequence whose
    pages, with those of the sequences before it, are more than are free keeps
    its entries as they are; no token may be appended to it before a later call
    has served it: give it length 0 in the calls that follow.
    """
    index, batch, width, pages = _table(table, lens, refs)
    first, count, structs = _layers(caches, index, pages)
    if cu_q is None:
        if tokens is not None and tokens != batch:
            raise ValueError(f"without cu_q every sequence has one new token: {tokens} tokens, {batch} sequences")
        tokens = batch
    else:
        if not (cu_q.shape == (batch + 1,) and cu_q.dtype is _I32 and cu_q.get_device() == index and cu_q.is_contiguous()):
            if cu_q.shape != (batch + 1,):
                raise ValueError(f"cu_q must be [{batch + 1}], got {tuple(cu_q.shape)}")
            _refuse(index, cu_q=cu_q)
        if tokens is None:
            raise ValueError("with cu_q, tokens says how many rows there are")
    ws_bytes = _workspace("nvfp4_kv_reserve_workspace_size", tokens, batch, first._page, pages)
    ws = torch.empty(ws_bytes, dtype=_U8, device=table.device)
    missing = torch.empty(batch, dtype=_I32, device=table.device)
    _check("nvfp4_kv_reserve", _on_device(
        index, load_library().nvfp4_kv_reserve, structs, count, table.data_ptr(), batch, width, lens.data_ptr(),
        None if cu_q is None else cu_q.data_ptr(), tokens, refs.data_ptr(), ws.data_ptr(), ws_bytes, missing.data_ptr(), _stream(table.device)))
    return missing


def kv_fork(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, parent: torch.Tensor,
            out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """A table and lengths whose row r is row parent[r]'s: sequences that go on
    from others and share their pages (samples of a prompt, beams of a search).

    table int32 [batch, width], lens int32 [batch], parent int32 [rows]; a
    parent outside [0, batch) gives a row without pages and tokens, and rows
    that are nobody's parent are dropped.  refs is changed in place, by the
    entries of the new table and those of the present one, which is not used
    any more.  out: the new table, int32 [rows, width], if given.
    """
    index, batch, width, pages = _table(table, lens, refs)
    if not (parent.dim() == 1 and parent.dtype is _I32 and parent.get_device() == index and parent.is_contiguous()):
        if parent.dim() != 1:
            raise ValueError("parent must be 1-D")
        _refuse(index, parent=parent)
    rows = parent.shape[0]
    if out is None:
        out = torch.empty(rows, width, dtype=_I32, device=table.device)
    elif not (out.shape == (rows, width) and out.dtype is _I32 and out.get_device() == index and out.is_contiguous()):
        if out.shape != (rows, width):
            raise ValueError(f"out must be {(rows, width)}, got {tuple(out.shape)}")
        _refuse(index, out=out)
    lens_out = torch.empty(rows, dtype=_I32, device=table.device)
    _check("nvfp4_kv_fork", _on_device(
        index, load_library().nvfp4_kv_fork, table.data_ptr(), batch, width, lens.data_ptr(), parent.data_ptr(), rows,
        refs.data_ptr(), pages, out.data_ptr(), lens_out.data_ptr(), _stream(table.device)))
    return out, lens_out


def kv_compact(caches: Union[KVCache, Sequence[KVCache]], table: torch.Tensor, refs: torch.Tensor
               ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Moves the pages in use to the front of the pool; (used, where).

    caches, table and refs as for kv_reserve, all changed in place.  used int32
    [1]: the pages in use, which are the first ones then; where int32 [pages]:
    the new place of each page that was in use, -1 for the others.  The k-th
    page in use at or behind `used` goes to the k-th free one before it.
    """
    index, shape = table.get_device(), table.shape
    if not (index >= 0 and len(shape) == 2 and refs.dim() == 1 and table.dtype is _I32 and refs.dtype is _I32
            and refs.get_device() == index and table.is_contiguous() and refs.is_contiguous()):
        _refuse(index, table=table, refs=refs)
    (batch, width), pages = shape, refs.shape[0]
    _, count, structs = _layers(caches, index, pages)
    ws_bytes = _workspace("nvfp4_kv_compact_workspace_size", pages)
    ws = torch.empty(ws_bytes, dtype=_U8, device=table.device)
    used = torch.empty(1, dtype=_I32, device=table.device)
    where = torch.empty(pages, dtype=_I32, device=table.device)
    _check("nvfp4_kv_compact", _on_device(
        index, load_library().nvfp4_kv_compact, structs, count, table.data_ptr(), batch, width, refs.data_ptr(), ws.data_ptr(),
        ws_bytes, used.data_ptr(), where.data_ptr(), _stream(table.device)))
    return used, where
