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

from . import NVFP4Error, _check, _dtype_code, _stream, load_library

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
    contiguous, on one GPU, and stay the caller's: the object only names them,
    by the addresses that they have when it is made, so its attributes cannot be
    assigned.
    """

    __slots__ = ("_k", "_v", "_k_scales", "_v_scales", "_pages", "_heads", "_page", "_dim", "_device", "_index",
                 "_struct", "_ref")

    k = property(lambda self: self._k, doc="codes of the keys")
    v = property(lambda self: self._v, doc="codes of the values")
    k_scales = property(lambda self: self._k_scales, doc="scales of the keys")
    v_scales = property(lambda self: self._v_scales, doc="scales of the values")
    pages = property(lambda self: self._pages, doc="pages of the pool")
    heads = property(lambda self: self._heads, doc="key/value heads")
    page = property(lambda self: self._page, doc="tokens of a page")
    dim = property(lambda self: self._dim, doc="channels of a head")
    device = property(lambda self: self._device, doc="the tensors' device")
    index = property(lambda self: self._index, doc="the device's index")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor):
        shape, index = k.shape, k.get_device()
        if len(shape) != 4:
            raise ValueError("k must be [pages, heads, page, dim]")
        pages, heads, page, dim = shape
        flat = (pages, heads)
        if v.shape != (pages, heads, dim, page):
            raise ValueError(f"v {tuple(v.shape)} does not match k {tuple(shape)} (expected [pages, heads, dim, page])")
        if k_scales.shape != flat or v_scales.shape != flat:
            raise ValueError("k_scales and v_scales must be [pages, heads]")
        if page not in _PAGES or dim not in _DIMS or heads < 1:
            raise ValueError(f"page must be one of {_PAGES}, dim one of {_DIMS} and heads at least 1, "
                             f"got {page}, {dim} and {heads}")
        if not (k.dtype is _U8 and v.dtype is _U8 and k_scales.dtype is _U8 and v_scales.dtype is _U8):
            raise TypeError("the cache's tensors must be uint8")
        if not (k.is_contiguous() and v.is_contiguous() and k_scales.is_contiguous() and v_scales.is_contiguous()):
            raise ValueError("the cache's tensors must be contiguous")
        if not index == v.get_device() == k_scales.get_device() == v_scales.get_device():
            raise ValueError("the cache's tensors must be on the same device")
        if index < 0:
            raise ValueError("the cache's tensors must be on the GPU")
        self._k, self._v, self._k_scales, self._v_scales = k, v, k_scales, v_scales
        self._pages, self._heads, self._page, self._dim, self._index = pages, heads, page, dim, index
        self._device = k.device
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                                    pages, heads, page, dim)
        self._ref = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, pages: int, heads: int, page: int, dim: int, device="cuda") -> "KVCache":
        """A cache of zeros, which kv_append fills."""
        z = lambda *shape: torch.zeros(shape, dtype=_U8, device=device)  # noqa: E731
        return cls(z(pages, heads, page, dim), z(pages, heads, dim, page), z(pages, heads), z(pages, heads))


# The checks run on every call of a decode step, so each is one comparison of
# what a call has at hand; what is wrong is worked out only once one fails.

def _refuse_tokens(name: str, x: torch.Tensor, cache: KVCache, tokens: int, heads: int, dtype) -> None:
    """Raises for a tensor of new tokens that is not [tokens, heads, dim]."""
    if x.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if x.shape != (tokens, heads, cache._dim):
        raise ValueError(f"{name} {tuple(x.shape)} must be {(tokens, heads, cache._dim)} ([tokens, heads, dim])")
    if x.get_device() != cache._index:
        raise ValueError(f"{name} must be on the cache's device")
    raise ValueError(f"{name}'s last axis must be contiguous")


def _refuse_sequences(cache: KVCache, **tensors: Optional[torch.Tensor]) -> None:
    for name, t in tensors.items():
        if t is None:
            continue
        if t.dtype is not _I32:
            raise TypeError(f"{name} must be int32, got {t.dtype}")
        if t.get_device() != cache._index:
            raise ValueError(f"{name} must be on the cache's device")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    raise ValueError("table must be [batch, width], lens [batch] and cu_q [batch + 1]")


def _sequences(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, cu_q: Optional[torch.Tensor],
               max_q: Optional[int], tokens: int):
    """(batch, width, max_q, address of cu_q) of the sequences' tensors, checked."""
    index, shape = cache._index, table.shape
    if not (len(shape) == 2 and lens.shape == (shape[0],) and table.dtype is _I32 and lens.dtype is _I32
            and table.get_device() == index == lens.get_device() and table.is_contiguous() and lens.is_contiguous()):
        _refuse_sequences(cache, table=table, lens=lens)
    batch, width = shape
    if cu_q is None:
        if tokens != batch:
            raise ValueError(f"without cu_q every sequence has one new token: {tokens} tokens, {batch} sequences")
        return batch, width, 1, None
    if not (cu_q.shape == (batch + 1,) and cu_q.dtype is _I32 and cu_q.get_device() == index and cu_q.is_contiguous()):
        _refuse_sequences(cache, cu_q=cu_q)
    if max_q is None or max_q > tokens:
        max_q = tokens
    elif max_q < 0 or (max_q == 0 and tokens > 0):
        raise ValueError("max_q must be at least the new tokens of the longest sequence")
    return batch, width, max_q, cu_q.data_ptr()


def _output(out: Optional[torch.Tensor], q: torch.Tensor, shape, cache: KVCache) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=q.dtype, device=cache._device)
    if out.dtype is not q.dtype or out.shape != shape or not out.is_contiguous() or out.get_device() != cache._index:
        raise ValueError("out must be contiguous, of q's dtype, shape and device")
    return out


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
    (default: all of them) that sizes the launch; a sequence's tokens past it
    are left out, and their rows of the result not written.

    inv_freq float32 [rot / 2]: channels [0, rot) of keys and queries turn by
    position * inv_freq[i], in the pairs (i, i + rot / 2) or, interleaved,
    (2i, 2i + 1).  A page's scale grows with its largest value, and the codes
    that it held are then rounded anew; the values of a page at one scale are
    off by at most half a step of their codes.
    """
    dtype, shape, index, dim = k.dtype, k.shape, cache._index, cache._dim
    code = _dtype_code(dtype)
    tokens = shape[0] if len(shape) else 0
    want = (tokens, cache._heads, dim)
    ks, vs = k.stride(), v.stride()
    if not (shape == want and k.get_device() == index and (ks[2] == 1 or tokens == 0)):
        _refuse_tokens("k", k, cache, tokens, cache._heads, dtype)
    if not (v.shape == want and v.dtype is dtype and v.get_device() == index and (vs[2] == 1 or tokens == 0)):
        _refuse_tokens("v", v, cache, tokens, cache._heads, dtype)
    batch, width, most, cu = _sequences(cache, table, lens, cu_q, max_q, tokens)
    rot, freq = 0, None
    if inv_freq is not None:
        if inv_freq.dtype is not _F32:
            raise TypeError(f"inv_freq must be float32, got {inv_freq.dtype}")
        if inv_freq.dim() != 1 or not inv_freq.is_contiguous() or inv_freq.get_device() != index:
            raise ValueError("inv_freq must be 1-D, contiguous and on the cache's device")
        rot = 2 * inv_freq.shape[0]
        if rot > dim:
            raise ValueError(f"inv_freq turns {rot} of {dim} channels")
        freq = inv_freq.data_ptr() if rot else None
    if q is not None:
        q_shape = q.shape
        qs, heads_q = q.stride(), q_shape[1] if len(q_shape) == 3 else 0
        if not (q_shape == (tokens, heads_q, dim) and q.dtype is dtype and q.get_device() == index
                and (qs[2] == 1 or tokens == 0 or heads_q == 0)):
            _refuse_tokens("q", q, cache, tokens, heads_q, dtype)
        out = _output(out, q, q_shape, cache)
        qp, q_token, q_head, qo = q.data_ptr(), qs[0], qs[1], out.data_ptr()
    else:
        if out is not None:
            raise ValueError("out without q")
        qp = qo = None
        q_token = q_head = heads_q = 0
    if tokens == 0:
        return out
    if heads_q == 0:
        qp = qo = None      # a tensor without heads has no address
    _check("nvfp4_kv_append", load_library().nvfp4_kv_append(
        cache._ref, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], qp, q_token, q_head, heads_q, qo, code,
        tokens, cu, batch, most, table.data_ptr(), width, lens.data_ptr(), freq, rot, 1 if interleaved else 0,
        _stream(cache._device)))
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
    shape, heads, dim = q.shape, cache._heads, cache._dim
    tokens, heads_q = (shape[0], shape[1]) if len(shape) == 3 else (0, 0)
    qs = q.stride()
    if not (shape == (tokens, heads_q, dim) and q.get_device() == cache._index
            and (qs[2] == 1 or tokens == 0 or heads_q == 0)):
        _refuse_tokens("q", q, cache, tokens, heads_q, q.dtype)
    if heads_q % heads != 0:
        raise ValueError(f"{heads_q} query heads are not a multiple of the cache's {heads}")
    batch, width, most, cu = _sequences(cache, table, lens, cu_q, max_q, tokens)
    out = _output(out, q, shape, cache)
    if tokens == 0 or heads_q == 0:
        return out
    lib = load_library()
    key = (tokens, heads_q, heads, dim, cache._page, batch, most, width, window, code)
    ws_bytes = _ATTENTION_WS_CACHE.get(key)
    if ws_bytes is None:
        ws_bytes = int(lib.nvfp4_paged_attention_workspace_size(*key))
        if ws_bytes < 0:
            raise NVFP4Error("nvfp4_paged_attention_workspace_size", ws_bytes)
        if len(_ATTENTION_WS_CACHE) < 4096:
            _ATTENTION_WS_CACHE[key] = ws_bytes
    ws = torch.empty(ws_bytes, dtype=_U8, device=cache._device) if ws_bytes else None
    _check("nvfp4_paged_attention", lib.nvfp4_paged_attention(
        cache._ref, q.data_ptr(), qs[0], qs[1], heads_q, code, tokens, cu, batch, most, table.data_ptr(), width,
        lens.data_ptr(), window, dim ** -0.5 if scale is None else scale, ws.data_ptr() if ws_bytes else None, ws_bytes,
        out.data_ptr(), _stream(cache._device)))
    return out


# nvfp4_sample_workspace_size by call shape
_SAMPLE_WS_CACHE: dict = {}


def _row_values(name: str, t: Optional[torch.Tensor], dtype, shape, index: int):
    """The address of a tensor of one value per row, checked; None for None."""
    if t is None:
        return None
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()):
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.get_device() != index:
            raise ValueError("all tensors must be on the same device")
        raise ValueError(f"{name} must be contiguous with one value per row")
    return t.data_ptr()


def sample(logits: torch.Tensor, u: torch.Tensor, temperature: Optional[torch.Tensor] = None,
           top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
           min_p: Optional[torch.Tensor] = None, return_prob: bool = False):
    """The next token of each row of logits, from given random numbers.

    logits [batch, vocab] (float32, bfloat16 or float16, last axis
    contiguous); u float32 [batch] in [0, 1); temperature, top_p, min_p
    float32 [batch] and top_k int32 [batch], or None for 1, 1, 0 and 0 (all
    kept).  Tokens are ordered by falling logit, equal ones by index; weights
    are exp((logit - largest) / temperature), at a temperature that is not above
    0 those of the largest alone.  top_k keeps the first k, top_p
    those of them with less than top_p of their sum before them, min_p those
    with at least min_p of the largest weight; the first one always stays.
    The token is the first kept one, by index, whose running sum of weights
    exceeds u times the whole.  Returns int32 [batch] (-1 for a row with
    nothing above -inf; NaN counts as -inf), with return_prob also its
    probability among the kept ones, float32 [batch].
    """
    code = _dtype_code(logits.dtype)
    shape, index = logits.shape, logits.get_device()
    if len(shape) != 2:
        raise ValueError("logits must be [batch, vocab]")
    if index < 0:
        raise ValueError("all tensors must be on the GPU")
    batch, vocab = shape
    if vocab == 0 and batch > 0:
        raise ValueError("logits have no tokens")
    row, last = logits.stride()
    if batch <= 1:
        row = vocab
    if (vocab > 1 and last != 1) or row < vocab:
        raise ValueError("logits' last axis must be contiguous and rows must not overlap")
    per_row = (batch,)
    up = _row_values("u", u, _F32, per_row, index)
    tp = _row_values("temperature", temperature, _F32, per_row, index)
    kp = _row_values("top_k", top_k, _I32, per_row, index)
    pp = _row_values("top_p", top_p, _F32, per_row, index)
    mp = _row_values("min_p", min_p, _F32, per_row, index)
    device = logits.device
    token = torch.empty(batch, dtype=_I32, device=device)
    prob = torch.empty(batch, dtype=_F32, device=device) if return_prob else None
    lib = load_library()
    key = (batch, vocab, code)
    ws_bytes = _SAMPLE_WS_CACHE.get(key)
    if ws_bytes is None:
        ws_bytes = int(lib.nvfp4_sample_workspace_size(*key))
        if ws_bytes < 0:
            raise NVFP4Error("nvfp4_sample_workspace_size", ws_bytes)
        if len(_SAMPLE_WS_CACHE) < 4096:
            _SAMPLE_WS_CACHE[key] = ws_bytes
    ws = torch.empty(ws_bytes, dtype=_U8, device=device) if ws_bytes else None
    _check("nvfp4_sample", lib.nvfp4_sample(
        logits.data_ptr(), code, batch, vocab, row, up, tp, kp, pp, mp, ws.data_ptr() if ws_bytes else None, ws_bytes,
        token.data_ptr(), prob.data_ptr() if return_prob else None, _stream(device)))
    return (token, prob) if return_prob else token
