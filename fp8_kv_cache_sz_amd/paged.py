"""The paged KV cache: writing new tokens' K and V into pages, reading them
back, and attention of new tokens over the pages (sz_cache_write,
sz_cache_read, sz_paged_attention in include/splitzip.h).

A ``PagedCache`` is one layer's ``[pages, 2, kv_heads, page_tokens, head_dim]``
tensor (keys, then values) of BF16, E5M2 or E4M3, with a scale byte for each
FP8 row.  E5M2 and BF16 pages are the codec's element types:
``encode(cache.data[first:last], codebook)`` compresses pages as they lie.

A ``PageBatch`` says which tokens a call is about: sequence i has
``kv_lens[i]`` tokens in the cache, the new ones included, and its new tokens
are ``starts[i]:starts[i + 1]`` of the packed axis of k, v, q and outputs.
The three arrays stay on the device; they may be changed in place between
calls and between replays of a captured graph.

Every call only enqueues unless ``check`` is true, which waits for the device
and raises ``SplitZipError`` if the batch was found wrong.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd import forward_ad

from . import _native
from ._native import SZ_BF16, SZ_FP8_E4M3, SZ_FP8_E5M2, SplitZipError

E4M3 = SZ_FP8_E4M3
ARRIVALS = 4096         # bytes of counters at the start of an attention workspace

# Looked up once: a small call is as short as the Python in front of its launch.
_bfloat16 = torch.bfloat16
_grad_enabled = torch.is_grad_enabled
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream

_BAD_BATCH = "paged cache (device check of the batch)"
_ELEMENT = {SZ_BF16: torch.bfloat16, SZ_FP8_E5M2: torch.float8_e5m2, SZ_FP8_E4M3: torch.float8_e4m3fn}


class _Fixed:
    """Attributes that the C structure of an object was made from are not
    reassigned: the kernels would go on with the tensors and bounds it had."""
    _made = False

    def __setattr__(self, name, value):
        if self._made and name in self._FIXED and value is not getattr(self, name):    # kv_lens += 1 assigns itself
            raise AttributeError("%s.%s is what its calls were made from: make another %s"
                                 % (type(self).__name__, name, type(self).__name__))
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        if name in self._FIXED:
            raise AttributeError("%s.%s is what its calls were made from" % (type(self).__name__, name))
        object.__delattr__(self, name)


class PagedCache(_Fixed):
    """One layer's pages.  ``data``: a contiguous device tensor ``[pages, 2,
    kv_heads, page_tokens, head_dim]`` of the element type (FP8 also as
    ``uint8``); ``scales``: ``uint8`` ``[pages, 2, kv_heads, page_tokens]``
    for FP8, None for BF16.  The tensors stay the caller's, and their memory
    where it is (no ``set_`` or ``resize_``); the attributes are not reassigned.
    ``status`` is the device int32 that the calls report into."""

    _FIXED = frozenset(("dtype", "data", "scales", "status", "device", "pages", "kv_heads", "page_tokens", "head_dim"))

    def __init__(self, dtype: int, data: torch.Tensor, scales: torch.Tensor | None = None,
                 status: torch.Tensor | None = None):
        if dtype not in _ELEMENT:
            raise ValueError("a paged cache holds BF16, E5M2 or E4M3, got dtype %r" % (dtype,))
        _plain("data", data)
        if data.dtype != _ELEMENT[dtype] and not (dtype != SZ_BF16 and data.dtype == torch.uint8):
            raise TypeError("data is %s, the cache's element type is %s" % (data.dtype, _ELEMENT[dtype]))
        if data.dim() != 5 or data.shape[1] != 2 or not data.is_contiguous():
            raise ValueError("data is a contiguous [pages, 2, kv_heads, page_tokens, head_dim] tensor")
        if dtype == SZ_BF16:
            if scales is not None:
                raise ValueError("a BF16 cache has no scales")
        else:
            if scales is None:
                raise ValueError("an FP8 cache needs scales")
            if scales.dtype != torch.uint8 or scales.shape != data.shape[:-1] or not scales.is_contiguous():
                raise ValueError("scales is a contiguous uint8 tensor of data's shape without the last axis")
            if scales.device != data.device:
                raise ValueError("data and scales are on different devices")
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=data.device)
        elif status.dtype != torch.int32 or status.numel() != 1 or status.device != data.device:
            raise ValueError("status is one int32 on the cache's device")
        pages, _, kv_heads, page_tokens, head_dim = data.shape
        c = _native.sz_cache(dtype, page_tokens, kv_heads, head_dim, pages, data.data_ptr(),
                             scales.data_ptr() if scales is not None else None)
        self.__dict__.update(                           # _index -1: not on a GPU
            dtype=dtype, data=data, scales=scales, status=status, device=data.device, _index=data.get_device(),
            pages=pages, kv_heads=kv_heads, page_tokens=page_tokens, head_dim=head_dim, _c=c, _ref=ctypes.byref(c),
            _status=status.data_ptr(), _made=True)

    def raise_status(self) -> None:
        """Waits for the current stream, raises if a call found its batch
        wrong, and clears the word."""
        status = int(self.status.item())
        if status != 0:
            self.status.zero_()
            torch.cuda.current_stream(self.device).synchronize()     # before a call on any stream reports again
            raise SplitZipError(_BAD_BATCH, status)


def paged_cache(pages: int, page_tokens: int, kv_heads: int, head_dim: int, dtype: int = SZ_BF16,
                device="cuda") -> PagedCache:
    """An empty cache; every row reads as zeros."""
    if dtype not in _ELEMENT:
        raise ValueError("a paged cache holds BF16, E5M2 or E4M3, got dtype %r" % (dtype,))
    shape = (pages, 2, kv_heads, page_tokens, head_dim)
    if dtype == SZ_BF16:
        return PagedCache(dtype, torch.zeros(shape, dtype=torch.bfloat16, device=device))
    data = torch.zeros(shape, dtype=torch.uint8, device=device).view(_ELEMENT[dtype])
    return PagedCache(dtype, data, torch.full(shape[:-1], 127, dtype=torch.uint8, device=device))


class PageBatch(_Fixed):
    """The tokens of a call.  ``page_table`` int32 ``[seqs, width]``,
    ``kv_lens`` int32 ``[seqs]``, ``starts`` int32 ``[seqs + 1]``, contiguous,
    on one device; ``tokens`` the length of the packed axis.  ``max_new`` and
    ``max_kv`` bound a sequence's new tokens and length; without them the
    launches are shaped for ``tokens`` and for full tables.  The tensors' values
    may change between calls; their memory stays where it is, and the attributes
    are not reassigned."""

    _FIXED = frozenset(("page_table", "kv_lens", "starts", "device", "seqs", "width", "tokens", "max_new", "max_kv"))

    def __init__(self, page_table: torch.Tensor, kv_lens: torch.Tensor, starts: torch.Tensor, tokens: int,
                 max_new: int | None = None, max_kv: int | None = None):
        if page_table.dim() != 2:
            raise ValueError("page_table is [seqs, width]")
        seqs, width = page_table.shape
        if kv_lens.shape != (seqs,) or starts.shape != (seqs + 1,):
            raise ValueError("kv_lens is [seqs] and starts [seqs + 1], with seqs = %d from page_table" % seqs)
        for name, t in (("page_table", page_table), ("kv_lens", kv_lens), ("starts", starts)):
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise TypeError("%s is a contiguous int32 tensor" % name)
            if t.device != page_table.device:
                raise ValueError("page_table, kv_lens and starts are on different devices")
        if tokens < 0 or (max_new is not None and max_new < 0) or (max_kv is not None and max_kv < 0):
            raise ValueError("tokens, max_new and max_kv count from 0")
        self.__dict__.update(
            page_table=page_table, kv_lens=kv_lens, starts=starts, device=page_table.device, seqs=seqs, width=width,
            tokens=tokens, _index=page_table.get_device(), max_new=tokens if max_new is None else max_new,
            max_kv=max_kv, _by_page={}, _made=True)

    def _ref(self, page_tokens: int):
        """The sz_batch for caches of this page size (max_kv defaults to a
        full table's tokens), or 0: for calls that look at no page."""
        ref = self._by_page.get(page_tokens)
        if ref is None:
            top = 2 ** 32 - 1
            max_kv = self.max_kv
            if max_kv is None:
                max_kv = min(self.width * page_tokens, 1 << 30) if page_tokens else 1 << 30
            if max(self.tokens, self.seqs, self.width, self.max_new, max_kv) > top:
                raise ValueError("the batch is too large")
            b = _native.sz_batch(self.page_table.data_ptr(), self.kv_lens.data_ptr(), self.starts.data_ptr(),
                                 self.seqs, self.width, self.tokens, self.max_new, max_kv)
            ref = self._by_page[page_tokens] = ctypes.byref(b)
        return ref


def _rows(name, t, tokens, heads, cache):
    if t.dtype is not _bfloat16:
        raise TypeError("%s is a bfloat16 tensor, got %s" % (name, t.dtype))
    if t.shape != (tokens, heads, cache.head_dim):
        raise ValueError("%s is [%d, %d, %d], got %s" % (name, tokens, heads, cache.head_dim, tuple(t.shape)))
    if t.get_device() != cache._index:
        raise ValueError("%s is on %s, the cache on %s" % (name, t.device, cache.device))
    token, head, last = t.stride()
    if last != 1 and tokens:
        raise ValueError("%s needs contiguous rows (a last stride of 1)" % name)
    if forward_ad._current_level >= 0 or (t.requires_grad and _grad_enabled()):
        _plain(name, t)
    return t.data_ptr(), token, head


def _plain(name, t):
    """Refuses tensors that autograd follows: the calls have no derivative."""
    if t.requires_grad and _grad_enabled():
        raise ValueError("%s requires a gradient, and the paged cache has none to give (torch.no_grad)" % name)
    if forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None:
        raise ValueError("%s has a tangent, and the paged cache has none to give" % name)


def _rows_meet(a, b, tokens, heads, dim):
    """Whether rows of two [tokens, heads, dim] tensors of 2-byte values, as
    _rows gives them, share memory.  Tensors that interleave (K and V of one
    tensor) have the same strides: then a row of one meets a row of the other
    where some (tokens, heads) apart is less than a row from their distance.
    Tensors that overlap with other strides are taken to."""
    (at, token, head), (bt, *strides) = a, b
    size = lambda token, head: 2 * ((tokens - 1) * token + (heads - 1) * head + dim)
    if at + size(token, head) <= bt or bt + size(*strides) <= at:
        return False
    token, head = token if tokens > 1 else 0, head if heads > 1 else 0
    if [token, head] != [strides[0] if tokens > 1 else 0, strides[1] if heads > 1 else 0]:
        return True
    apart = (bt - at) // 2
    block = (heads - 1) * head + dim                            # a token's rows
    if token and block <= apart % token <= token - block:       # side by side: K and V of [tokens, 2, heads, dim]
        return False
    for h in range(1 - heads, heads):
        rest = apart - h * head
        t = 0 if token == 0 else max(1 - tokens, min(tokens - 1, rest // token))
        if abs(rest - t * token) < dim or (t + 1 < tokens and abs(rest - (t + 1) * token) < dim):
            return True
    return False


def _run(name, call, cache, batch, args, stream, owned=(), status=None):
    """Launches a call on `stream` (None: the current one) with the cache's
    device current, reporting into `status` (None: the cache's word).  Memory
    that this layer took from the current stream's pool (`owned`) is handed
    over to a stream other than that."""
    index = cache._index
    if status is None:
        status = cache._status
    if batch._index != index:
        raise ValueError("the batch is on %s, the cache on %s" % (batch.device, cache.device))
    if index < 0:
        raise ValueError("the cache is on %s; its calls run on the GPU" % cache.device)
    if stream is None and _current_device() == index:            # the common case, without a Stream object
        rc = call(cache._ref, batch._by_page.get(cache.page_tokens) or batch._ref(cache.page_tokens), *args,
                  status, _current_stream(index))
        if rc:
            _native.check(name, rc)
        return
    device = cache.device
    if stream is not None and stream.device != device:
        raise ValueError("the stream is on %s, the cache on %s" % (stream.device, device))
    current = torch.cuda.current_stream(device)
    side = None if stream is None or stream == current else stream
    if side is not None and owned:
        side.wait_stream(current)
    with torch.cuda.device(device):
        rc = call(cache._ref, batch._ref(cache.page_tokens), *args, status, (side or current).cuda_stream)
    _native.check(name, rc)
    if side is not None:
        for t in owned:
            t.record_stream(side)


def _raise_status(cache, stream):
    if stream is not None:
        stream.synchronize()
    cache.raise_status()


def cache_check(cache: PagedCache, batch: PageBatch, stream=None) -> None:
    """Raises ``SplitZipError`` unless the batch fits the cache and no page is
    written from two places (sz_cache_check); waits for the device.  The check
    reports into a word of its own: what earlier calls put into the cache's
    stays there."""
    nbytes = _native.sz_cache_check_workspace_size(cache._ref)
    ws = torch.empty(nbytes // 4 + 1, dtype=torch.int32, device=cache.device)           # claims, then the word
    _run("sz_cache_check", _native.lib.sz_cache_check, cache, batch, (ws.data_ptr(), nbytes), stream, (ws,),
         ws.data_ptr() + nbytes)
    if stream is not None:
        stream.synchronize()
    found = int(ws[-1].item())
    if found != 0:
        raise SplitZipError(_BAD_BATCH, found)


def cache_write(cache: PagedCache, batch: PageBatch, k: torch.Tensor, v: torch.Tensor, stream=None,
                check: bool = True) -> None:
    """Writes the batch's tokens (bfloat16 ``[tokens, kv_heads, head_dim]``,
    any token and head strides that keep rows 16-byte aligned) into their
    pages, FP8 caches quantised with a power-of-two scale for each row
    (sz_cache_write).  With ``check`` the batch is checked first
    (``cache_check``) and nothing is written if it is wrong."""
    args = (*_rows("k", k, batch.tokens, cache.kv_heads, cache), *_rows("v", v, batch.tokens, cache.kv_heads, cache))
    if check:
        cache_check(cache, batch, stream)
    _run("sz_cache_write", _native.lib.sz_cache_write, cache, batch, args, stream)


def cache_read(cache: PagedCache, batch: PageBatch, out=None, stream=None, check: bool = True):
    """The batch's tokens out of their pages: bfloat16 ``(k, v)``, each
    ``[tokens, kv_heads, head_dim]`` (sz_cache_read).  ``out``: such a pair to
    read into.  Rows of tokens that belong to no sequence keep what they
    held."""
    tokens, heads, dim = batch.tokens, cache.kv_heads, cache.head_dim
    owned = ()
    if out is None:
        both = cache.data.new_empty((2, tokens, heads, dim), dtype=_bfloat16)
        owned = (both,)
        k, v = both.unbind(0)
        at, row = both.data_ptr(), heads * dim
        args = (at, row, dim, at + tokens * row * 2, row, dim)
    else:
        k, v = out
        args = (*_rows("out[0]", k, tokens, heads, cache), *_rows("out[1]", v, tokens, heads, cache))
        for token, head in (args[1:3], args[4:6]):
            (near, count), (far, more) = sorted([(token, tokens), (head, heads)])
            if (count > 1 and near < dim) or (more > 1 and far < (count - 1) * near + dim):
                raise ValueError("out has rows that share memory")
        if tokens and args[0] == args[3]:
            raise ValueError("out's two tensors are one")
        if tokens and _rows_meet(args[:3], args[3:], tokens, heads, dim):
            raise ValueError("out's two tensors share memory")
    _run("sz_cache_read", _native.lib.sz_cache_read, cache, batch, args, stream, owned)
    if check:
        _raise_status(cache, stream)
    return k, v


def attention_workspace(cache: PagedCache, batch: PageBatch, q_heads: int) -> torch.Tensor:
    """A workspace for ``paged_attention`` and ``tree_attention`` of this batch's
    bounds, with any window.  Its first ``ARRIVALS`` bytes are zero, as every call leaves them
    (they are cleared on the current stream, before any call that uses it)."""
    if q_heads <= 0 or q_heads % cache.kv_heads:
        raise ValueError("q_heads is a multiple of the cache's %d KV heads, got %d" % (cache.kv_heads, q_heads))
    n = _native.sz_paged_attention_workspace_size(cache._ref, batch._ref(cache.page_tokens), q_heads)
    ws = torch.empty(n, dtype=torch.uint8, device=cache.device)
    ws[:ARRIVALS].zero_()
    return ws


def paged_attention(q: torch.Tensor, cache: PagedCache, batch: PageBatch, scale: float | None = None,
                    window: int = 0, out: torch.Tensor | None = None, lse=False, ws: torch.Tensor | None = None,
                    stream=None, check: bool = True):
    """Causal attention of the batch's tokens over their sequences' cached
    keys and values, the tokens' own included (sz_paged_attention).  ``q``:
    bfloat16 ``[tokens, q_heads, head_dim]``; ``scale`` defaults to
    head_dim**-0.5; with ``window`` > 0 a token sees the last ``window``
    positions up to its own.  Returns bfloat16 ``out``, or ``(out, lse)`` with
    ``lse`` true or a float32 ``[tokens, q_heads]`` tensor to write into."""
    return _attend("sz_paged_attention", _native.lib.sz_paged_attention, (), q, cache, batch, scale, window, out, lse, ws,
                   stream, check)


def _attend(name, call, masks, q, cache, batch, scale, window, out, lse, ws, stream, check):
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q is [tokens, q_heads, head_dim]")
    q_heads = shape[1]
    qp, q_token, q_head = _rows("q", q, batch.tokens, q_heads, cache)
    if q_heads == 0 or q_heads % cache.kv_heads:
        raise ValueError("q has %d heads, not a multiple of the cache's %d KV heads" % (q_heads, cache.kv_heads))
    if window < 0:
        raise ValueError("window counts from 0 (0: none)")
    owned = []
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        owned.append(out)
    elif out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_contiguous() or out.device != cache.device:
        raise ValueError("out is a contiguous bfloat16 tensor of q's shape on the cache's device")
    elif out.requires_grad or forward_ad._current_level >= 0:
        _plain("out", out)
    if lse is True:
        lse = q.new_empty((batch.tokens, q_heads), dtype=torch.float32)
        owned.append(lse)
    elif lse is False:
        lse = None
    elif lse is not None and (lse.shape != q.shape[:2] or lse.dtype != torch.float32 or not lse.is_contiguous()
                              or lse.device != cache.device):
        raise ValueError("lse is a contiguous float32 [tokens, q_heads] tensor on the cache's device")
    elif lse is not None and (lse.requires_grad or forward_ad._current_level >= 0):
        _plain("lse", lse)
    if ws is None:
        ws = attention_workspace(cache, batch, q_heads)
        owned.append(ws)
    elif not ws.is_contiguous() or ws.get_device() != cache._index:
        raise ValueError("ws is a contiguous tensor on the cache's device (attention_workspace)")
    _run(name, call, cache, batch,
         (*masks, qp, q_heads, q_token, q_head, cache.head_dim ** -0.5 if scale is None else scale, min(window, 1 << 30),
          out.data_ptr(), None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.nbytes), stream, owned)
    if check:
        _raise_status(cache, stream)
    return out if lse is None else (out, lse)
