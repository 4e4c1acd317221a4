"""Serving operators around the quantized products: a paged key/value cache
held in 8 bits, attention over it, and the choice of the next token.

A decode step calls ``kv_append`` with the projections of its new tokens,
``paged_attention`` with the rotated queries, and ``sample`` with the logits::

    cache = nv.KVCache.empty(pages, kv_heads, page, dim)
    q = nv.kv_append(k, v, cache, table, lens, q=q, inv_freq=inv_freq)
    o = nv.paged_attention(q, cache, table, lens)
    token = nv.sample(logits, u, temperature=t, top_p=p)

As everywhere in the package the arguments' types, shapes and devices are
checked here, the work runs in the library's HIP kernels on the current
stream, and outputs and workspaces come from torch's allocator.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import NVFP4Error, _check, _dtype_code, _ptr, _stream, load_library

_PAGES = (16, 32, 64, 128, 256)
_DIMS = (64, 128, 192, 256)
_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8


class _CacheStruct(ctypes.Structure):
    """nvfp4_kv_cache_t"""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("page", ctypes.c_int64), ("dim", ctypes.c_int64)]


class KVCache:
    """A pool of pages of 8-bit keys and values.

    k uint8 [pages, heads, page, dim] and v uint8 [pages, heads, dim, page]
    hold E4M3 codes; k_scales and v_scales uint8 [pages, heads] the power of
    two (exponent + 127) that a page's codes of one head are multiplied by.
    page is 16, 32, 64, 128 or 256, dim 64, 128, 192 or 256.  The tensors are
    contiguous, on one GPU, and stay the caller's: the object only names them.
    """

    __slots__ = ("k", "v", "k_scales", "v_scales", "pages", "heads", "page", "dim", "device", "index", "_struct", "_ref")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor):
        if k.dim() != 4:
            raise ValueError("k must be [pages, heads, page, dim]")
        pages, heads, page, dim = k.shape
        if v.shape != (pages, heads, dim, page):
            raise ValueError(f"v {tuple(v.shape)} does not match k {tuple(k.shape)} (expected [pages, heads, dim, page])")
        if k_scales.shape != (pages, heads) or v_scales.shape != (pages, heads):
            raise ValueError("k_scales and v_scales must be [pages, heads]")
        if page not in _PAGES or dim not in _DIMS or heads < 1:
            raise ValueError(f"page must be one of {_PAGES}, dim one of {_DIMS} and heads at least 1, "
                             f"got {page}, {dim} and {heads}")
        index = k.get_device()
        for t in (k, v, k_scales, v_scales):
            if t.dtype is not _U8:
                raise TypeError(f"the cache's tensors must be uint8, got {t.dtype}")
            if not t.is_contiguous():
                raise ValueError("the cache's tensors must be contiguous")
            if t.get_device() != index:
                raise ValueError("the cache's tensors must be on the same device")
        if index < 0:
            raise ValueError("the cache's tensors must be on the GPU")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.pages, self.heads, self.page, self.dim = pages, heads, page, dim
        self.device, self.index = k.device, index
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                                    pages, heads, page, dim)
        self._ref = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, pages: int, heads: int, page: int, dim: int, device="cuda") -> "KVCache":
        """A cache of zeros, which kv_append fills."""
        z = lambda *shape: torch.zeros(shape, dtype=_U8, device=device)  # noqa: E731
        return cls(z(pages, heads, page, dim), z(pages, heads, dim, page), z(pages, heads), z(pages, heads))


def _tokens(name: str, x: torch.Tensor, cache: KVCache, heads: Optional[int], tokens: Optional[int], dtype) -> None:
    """x must be [tokens, heads, dim] on the cache's device with its last axis contiguous."""
    if x.dim() != 3 or x.shape[2] != cache.dim or (heads is not None and x.shape[1] != heads) or (
            tokens is not None and x.shape[0] != tokens):
        raise ValueError(f"{name} {tuple(x.shape)} must be [tokens, heads, dim] with dim {cache.dim}"
                         + (f", heads {heads}" if heads is not None else "")
                         + (f", tokens {tokens}" if tokens is not None else ""))
    if dtype is not None and x.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if x.get_device() != cache.index:
        raise ValueError(f"{name} must be on the cache's device")
    if x.stride(2) != 1:
        raise ValueError(f"{name}'s last axis must be contiguous")


def _plan(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, cu_q: Optional[torch.Tensor],
          max_q: Optional[int], tokens: int):
    """(batch, width, max_q) of the sequences' tensors, checked."""
    if table.dim() != 2 or lens.dim() != 1 or lens.shape[0] != table.shape[0]:
        raise ValueError("table must be [batch, width] and lens [batch]")
    batch, width = table.shape
    for name, t in (("table", table), ("lens", lens), ("cu_q", cu_q)):
        if t is None:
            continue
        if t.dtype is not _I32:
            raise TypeError(f"{name} must be int32, got {t.dtype}")
        if t.get_device() != cache.index:
            raise ValueError(f"{name} must be on the cache's device")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if cu_q is None:
        if tokens != batch:
            raise ValueError(f"without cu_q every sequence has one new token: {tokens} tokens, {batch} sequences")
        return batch, width, 1
    if cu_q.dim() != 1 or cu_q.shape[0] != batch + 1:
        raise ValueError("cu_q must be [batch + 1]")
    if max_q is None:
        return batch, width, tokens
    if max_q < 0 or (max_q == 0 and tokens > 0):
        raise ValueError("max_q must be at least the new tokens of the longest sequence")
    return batch, width, min(int(max_q), tokens)


def kv_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, table: torch.Tensor, lens: torch.Tensor,
              q: Optional[torch.Tensor] = None, cu_q: Optional[torch.Tensor] = None, max_q: Optional[int] = None,
              inv_freq: Optional[torch.Tensor] = None, interleaved: bool = False,
              out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Writes new keys and values into the cache; returns the rotated queries.

    k and v [tokens, kv heads, dim] and q [tokens, heads, dim] (float32,
    bfloat16 or float16, any strides of tokens and heads: the parts of one
    projection's rows serve as they are).  table int32 [batch, width]: the
    pages of each sequence, in order; lens int32 [batch]: its tokens, the new
    ones among them; cu_q int32 [batch + 1]: the rows of its new tokens
    (default: one each); max_q: an upper bound of a sequence's new tokens
    (default: all of them) that sizes the launch.

    inv_freq float32 [rot / 2]: channels [0, rot) of keys and queries turn by
    position * inv_freq[i], in the pairs (i, i + rot / 2) or, interleaved,
    (2i, 2i + 1).  A page's scale grows with its largest value, and the codes
    that it held are then rounded anew; the values of a page at one scale are
    off by at most half a step of their codes.
    """
    dtype = k.dtype
    code = _dtype_code(dtype)
    tokens = k.shape[0]
    _tokens("k", k, cache, cache.heads, None, None)
    _tokens("v", v, cache, cache.heads, tokens, dtype)
    batch, width, most = _plan(cache, table, lens, cu_q, max_q, tokens)
    rot = 0
    if inv_freq is not None:
        if inv_freq.dtype is not _F32 or inv_freq.dim() != 1:
            raise TypeError("inv_freq must be a 1-D float32 tensor")
        rot = 2 * inv_freq.shape[0]
        if rot > cache.dim:
            raise ValueError(f"inv_freq turns {rot} of {cache.dim} channels")
        if inv_freq.get_device() != cache.index or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be contiguous and on the cache's device")
        if rot == 0:
            inv_freq = None
    heads_q = 0
    if q is not None:
        _tokens("q", q, cache, None, tokens, dtype)
        heads_q = q.shape[1]
        if out is None:
            out = torch.empty(q.shape, dtype=dtype, device=cache.device)
        elif out.dtype is not dtype or out.shape != q.shape or not out.is_contiguous() or out.get_device() != cache.index:
            raise ValueError("out must be contiguous, of q's dtype, shape and device")
        q_args = (q.data_ptr(), q.stride(0), q.stride(1), heads_q, out.data_ptr())
    else:
        if out is not None:
            raise ValueError("out without q")
        q_args = (None, 0, 0, 0, None)
    if tokens and (q is None or heads_q):
        _check("nvfp4_kv_append", load_library().nvfp4_kv_append(
            cache._ref, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), *q_args, code,
            tokens, _ptr(cu_q), batch, most, table.data_ptr(), width, lens.data_ptr(), _ptr(inv_freq), rot,
            int(bool(interleaved)), _stream(cache.device)))
    return out


# nvfp4_paged_attention_workspace_size by call shape, as for qmm's workspace
_ATTENTION_WS_CACHE: dict = {}


def paged_attention(q: torch.Tensor, cache: KVCache, table: torch.Tensor, lens: torch.Tensor,
                    cu_q: Optional[torch.Tensor] = None, max_q: Optional[int] = None, window: int = 0,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention of the new tokens over their sequences' cached ones.

    q [tokens, heads, dim] (float32, bfloat16 or float16, any strides of
    tokens and heads), heads a multiple of the cache's; table, lens, cu_q and
    max_q as for kv_append, which has put the new tokens into the cache
    before.  window > 0: a query sees the last `window` tokens up to its own.
    scale defaults to dim ** -0.5.  Returns [tokens, heads, dim] in q's dtype,
    zeros for a query that sees nothing.
    """
    code = _dtype_code(q.dtype)
    _tokens("q", q, cache, None, None, None)
    tokens, heads_q, dim = q.shape
    if heads_q % cache.heads != 0:
        raise ValueError(f"{heads_q} query heads are not a multiple of the cache's {cache.heads}")
    batch, width, most = _plan(cache, table, lens, cu_q, max_q, tokens)
    window = int(window)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=cache.device)
    elif out.dtype is not q.dtype or out.shape != q.shape or not out.is_contiguous() or out.get_device() != cache.index:
        raise ValueError("out must be contiguous, of q's dtype, shape and device")
    lib = load_library()
    key = (tokens, heads_q, cache.heads, dim, cache.page, batch, most, width, window, code)
    ws_bytes = _ATTENTION_WS_CACHE.get(key)
    if ws_bytes is None:
        ws_bytes = int(lib.nvfp4_paged_attention_workspace_size(*key))
        if ws_bytes < 0:
            raise NVFP4Error("nvfp4_paged_attention_workspace_size", ws_bytes)
        if len(_ATTENTION_WS_CACHE) < 4096:
            _ATTENTION_WS_CACHE[key] = ws_bytes
    ws = torch.empty(ws_bytes, dtype=_U8, device=cache.device) if ws_bytes > 0 else None
    _check("nvfp4_paged_attention", lib.nvfp4_paged_attention(
        cache._ref, q.data_ptr(), q.stride(0), q.stride(1), heads_q, code, tokens, _ptr(cu_q), batch, most,
        table.data_ptr(), width, lens.data_ptr(), window, dim ** -0.5 if scale is None else float(scale), _ptr(ws),
        ws_bytes, out.data_ptr(), _stream(cache.device)))
    return out


def sample(logits: torch.Tensor, u: torch.Tensor, temperature: Optional[torch.Tensor] = None,
           top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
           min_p: Optional[torch.Tensor] = None, return_prob: bool = False):
    """The next token of each row of logits, from given random numbers.

    logits [batch, vocab] (float32, bfloat16 or float16, last axis
    contiguous); u float32 [batch] in [0, 1); temperature, top_p, min_p
    float32 [batch] and top_k int32 [batch], or None for 1, 1, 0 and 0 (all
    kept).  Tokens are ordered by falling logit, equal ones by index; weights
    are exp((logit - largest) / temperature).  top_k keeps the first k, top_p
    those of them with less than top_p of their sum before them, min_p those
    with at least min_p of the largest weight; the first one always stays.
    The token is the first kept one, by index, whose running sum of weights
    exceeds u times the whole.  Returns int32 [batch] (-1 for a row with
    nothing above -inf; NaN counts as -inf), with return_prob also its
    probability among the kept ones, float32 [batch].
    """
    code = _dtype_code(logits.dtype)
    if logits.dim() != 2:
        raise ValueError("logits must be [batch, vocab]")
    batch, vocab = logits.shape
    index = logits.get_device()
    if index < 0:
        raise ValueError("all tensors must be on the GPU")
    stride = logits.stride(0) if batch > 1 else vocab
    if vocab == 0 and batch > 0:
        raise ValueError("logits have no tokens")
    if vocab > 1 and logits.stride(1) != 1 or stride < vocab:
        raise ValueError("logits' last axis must be contiguous and rows must not overlap")
    for name, t, dtype in (("u", u, _F32), ("temperature", temperature, _F32), ("top_k", top_k, _I32),
                           ("top_p", top_p, _F32), ("min_p", min_p, _F32)):
        if t is None:
            continue
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.dim() != 1 or t.shape[0] != batch or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous with one value per row")
        if t.get_device() != index:
            raise ValueError("all tensors must be on the same device")
    device = logits.device
    token = torch.empty(batch, dtype=_I32, device=device)
    prob = torch.empty(batch, dtype=_F32, device=device) if return_prob else None
    lib = load_library()
    ws_bytes = int(lib.nvfp4_sample_workspace_size(batch, vocab, code))
    if ws_bytes < 0:
        raise NVFP4Error("nvfp4_sample_workspace_size", ws_bytes)
    ws = torch.empty(ws_bytes, dtype=_U8, device=device) if ws_bytes > 0 else None
    _check("nvfp4_sample", lib.nvfp4_sample(
        logits.data_ptr(), code, batch, vocab, stride, u.data_ptr(), _ptr(temperature), _ptr(top_k), _ptr(top_p),
        _ptr(min_p), _ptr(ws), ws_bytes, token.data_ptr(), _ptr(prob), _stream(device)))
    return (token, prob) if return_prob else token
