"""The rest of a serving step around the paged cache (paged.py): pages for
sequences from their lengths, trees of drafted tokens, rotary positions on the
way into the cache, attention of the trees, and the accepted tokens' rows moved
to where the next step expects them.  In the order of a step:

    pages_assign   -> page table, pages held, slots
    draft_tree     -> masks and positions of the trees
    rotary_write   -> turned queries; turned keys, and values, in their pages
    tree_attention -> the trees' attention over what is cached and themselves
    cache_keep     -> the accepted tokens' rows behind the sequences' pasts

Every call only enqueues unless ``check`` is true, which waits for the device
and raises ``SplitZipError`` if the batch was found wrong.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _native
from ._native import SZ_TREE_WORDS
from .paged import (PageBatch, PagedCache, SplitZipError, _attend, _BAD_BATCH, _current_device, _current_stream, _Fixed,
                    _plain, _raise_status, _rows, _rows_meet, _run)

_int32, _int64, _empty_like, _contiguous = torch.int32, torch.int64, torch.empty_like, torch.contiguous_format
COUNTERS = 256          # bytes at the start of an assignment's workspace
_NO_PAGE = 0            # the page size of calls that look at no page


def _ints(name, t, shape, index):
    """The address of a contiguous int32 tensor of this shape on the device."""
    if t.dtype is not _int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s is a contiguous int32 tensor %s, got %s %s" % (name, list(shape), t.dtype, list(t.shape)))
    if t.get_device() != index:
        raise ValueError("%s is on %s, not on the call's device" % (name, t.device))
    return t.data_ptr()


def _launch(name, call, index, device, args, stream, owned=()):
    """paged._run for calls without a cache: `args` and a stream, with device
    `index` current."""
    if index < 0:
        raise ValueError("the tensors are on %s; %s runs on the GPU" % (device, name))
    if stream is None and _current_device() == index:
        rc = call(*args, _current_stream(index))
        if rc:
            _native.check(name, rc)
        return
    if stream is not None and stream.device != device:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, device))
    current = torch.cuda.current_stream(device)
    side = None if stream is None or stream == current else stream
    if side is not None and owned:
        side.wait_stream(current)
    with torch.cuda.device(device):
        rc = call(*args, (side or current).cuda_stream)
    _native.check(name, rc)
    if side is not None:
        for t in owned:
            t.record_stream(side)


def _raise_word(status, stream):
    """Waits for the call, raises what it reported and clears the word."""
    if stream is not None:
        stream.synchronize()
    found = int(status.item())
    if found != 0:
        status.zero_()
        torch.cuda.current_stream(status.device).synchronize()
        raise SplitZipError(_BAD_BATCH, found)


class PagePool(_Fixed):
    """Free pages, as a ring in device memory: ``queue`` int32 ``[pages]``, of
    which the ``ends[1]`` entries from ``ends[0]`` on (modulo pages) are free
    page numbers; ``ends`` int32 ``[2]``.  ``status`` is the device int32 that
    calls report into.  The tensors' values change with every assignment; the
    attributes are not reassigned."""

    _FIXED = frozenset(("page_tokens", "queue", "ends", "status", "device", "pages"))

    def __init__(self, page_tokens: int, queue: torch.Tensor, ends: torch.Tensor, status: torch.Tensor | None = None):
        if queue.dim() != 1:
            raise ValueError("queue is [pages]")
        index = queue.get_device()
        _ints("queue", queue, queue.shape, index)
        _ints("ends", ends, (2,), index)
        if status is None:
            status = torch.zeros(1, dtype=_int32, device=queue.device)
        elif status.dtype != _int32 or status.numel() != 1 or status.device != queue.device:
            raise ValueError("status is one int32 on the pool's device")
        if not 0 < len(queue) <= 1 << 30:
            raise ValueError("a pool has 1 to 2**30 pages, got %d" % len(queue))
        if page_tokens not in (16, 32, 64, 128, 256, 512, 1024):
            raise ValueError("page_tokens is a power of two from 16 to 1024, got %r" % (page_tokens,))
        c = _native.sz_pool(page_tokens, len(queue), queue.data_ptr(), ends.data_ptr())
        self.__dict__.update(page_tokens=page_tokens, queue=queue, ends=ends, status=status, device=queue.device,
                             pages=len(queue), _index=index, _c=c, _ref=ctypes.byref(c), _made=True)

    def raise_status(self) -> None:
        """Waits for the current stream, raises if a call found its lengths
        wrong or the pool too small (``SZ_E_CAPACITY``), and clears the word."""
        _raise_word(self.status, None)


def page_pool(pages: int, page_tokens: int, device="cuda") -> PagePool:
    """A pool whose pages are all free."""
    return PagePool(page_tokens, torch.arange(pages, dtype=_int32, device=device),
                    torch.tensor([0, pages], dtype=_int32, device=device))


def assign_workspace(batch: PageBatch) -> torch.Tensor:
    """A workspace for ``pages_assign`` of batches of so many sequences.  Its
    first ``COUNTERS`` bytes are zero, as every call leaves them (they are
    cleared on the current stream, before any call that uses it)."""
    n = _native.sz_pages_assign_workspace_size(batch._ref(_NO_PAGE))
    ws = torch.empty(n, dtype=torch.uint8, device=batch.device)
    ws[:COUNTERS].zero_()
    return ws


def pages_assign(pool: PagePool, batch: PageBatch, held: torch.Tensor, held_out: torch.Tensor | None = None,
                 ends_out: torch.Tensor | None = None, slots=None, ws: torch.Tensor | None = None, stream=None,
                 check: bool = True):
    """Gives every sequence of the batch the pages that its length needs, and
    takes back those it no longer needs (sz_pages_assign).  ``held`` int32
    ``[seqs]``: how many entries of its row of ``batch.page_table`` a sequence
    holds; fresh entries are written behind them.  ``held`` and ``pool.ends``
    are updated, or with ``held_out`` and ``ends_out`` (int32 ``[2]``) left,
    and those written.  If the free pages do not reach for a sequence and all
    before it, it and those behind it that need more keep what they had, their
    fresh entries are -1 and the pool's status is ``SZ_E_CAPACITY``, unless
    something wrong was reported there.
    ``slots``: true, or an int64 ``[tokens]`` tensor, for the batch's tokens'
    page * page_tokens + row (-1: no place), which are returned."""
    index = pool._index
    if batch._index != index:
        raise ValueError("the batch is on %s, the pool on %s" % (batch.device, pool.device))
    shape = (batch.seqs,)
    at = _ints("held", held, shape, index)
    to = at if held_out is None else _ints("held_out", held_out, shape, index)
    ends = pool._c.ends if ends_out is None else _ints("ends_out", ends_out, (2,), index)
    if to != at and abs(to - at) < 4 * batch.seqs:
        raise ValueError("held_out shares memory with held")
    if ends != pool._c.ends and abs(ends - pool._c.ends) < 8:
        raise ValueError("ends_out shares memory with the pool's ends")
    owned = []
    if slots is True:
        slots = torch.empty(batch.tokens, dtype=torch.int64, device=pool.device)
        owned.append(slots)
    elif slots is False:
        slots = None
    elif slots is not None and (slots.dtype != _int64 or slots.shape != (batch.tokens,) or not slots.is_contiguous()
                                or slots.get_device() != index):
        raise ValueError("slots is a contiguous int64 [%d] tensor on the pool's device" % batch.tokens)
    if ws is None:
        ws = assign_workspace(batch)
        owned.append(ws)
    elif not ws.is_contiguous() or ws.get_device() != index:
        raise ValueError("ws is a contiguous tensor on the pool's device (assign_workspace)")
    page = pool.page_tokens
    _launch("sz_pages_assign", _native.lib.sz_pages_assign, index, pool.device,
            (pool._ref, batch._by_page.get(page) or batch._ref(page), at, to, ends,
             None if slots is None else slots.data_ptr(), ws.data_ptr(), ws.nbytes, pool.status.data_ptr()), stream, owned)
    if check:
        _raise_word(pool.status, stream)
    return slots


def tree_words(batch: PageBatch) -> int:
    """64-bit words of a token's mask in this batch."""
    words = batch.__dict__.get("_words")                # of fields that are not reassigned
    if words is None:
        words = batch.__dict__["_words"] = max(1, (min(batch.max_new, batch.tokens) + 63) // 64)
    return words


def draft_tree(batch: PageBatch, parents: torch.Tensor, out=None, status: torch.Tensor | None = None, stream=None,
               check: bool = True):
    """Trees of drafted tokens (sz_draft_tree): ``parents`` int32 ``[tokens]``
    has, for new token i of a sequence, the new token of the same sequence
    before it that it continues, or -1.  Returns ``(masks, positions)``: int64
    ``[tokens, words]``, bit j of the row's bits for new token j of the
    sequence and every token above, and int32 ``[tokens]``, the position that
    the token has in its line.  ``out``: such a pair to write into; rows of
    tokens that belong to no sequence keep what they held.  Parents that are
    none are reported into ``status`` (one int32, a cache's, say), without it
    only to ``check``."""
    index, tokens, words = batch._index, batch.tokens, tree_words(batch)
    if words > SZ_TREE_WORDS:
        raise ValueError("a tree has %d tokens at most, the batch's max_new is %d" % (64 * SZ_TREE_WORDS, batch.max_new))
    at = _ints("parents", parents, (tokens,), index)
    owned = []
    if out is None:
        masks = parents.new_empty((tokens, words), dtype=_int64)
        positions = _empty_like(parents)
        owned = [masks, positions]
    else:
        masks, positions = out
        words = _mask_words("out[0]", masks, batch, index)
        spans = sorted(((at, 4 * tokens), (_ints("out[1]", positions, (tokens,), index), 4 * tokens),
                        (masks.data_ptr(), 8 * tokens * words)))
        if spans[0][0] + spans[0][1] > spans[1][0] or spans[1][0] + spans[1][1] > spans[2][0]:
            raise ValueError("masks, positions and parents share memory")
    own = None
    if status is None:
        if check:
            own = torch.zeros(1, dtype=_int32, device=batch.device)
            owned.append(own)
    elif status.dtype != _int32 or status.numel() != 1 or status.get_device() != index:
        raise ValueError("status is one int32 on the batch's device")
    else:
        own = status
    _launch("sz_draft_tree", _native.lib.sz_draft_tree, index, batch.device,
            (batch._by_page.get(_NO_PAGE) or batch._ref(_NO_PAGE), at, masks.data_ptr(), words, positions.data_ptr(),
             None if own is None else own.data_ptr()), stream, owned)
    if check:
        _raise_word(own, stream)
    return masks, positions


def _mask_words(name, masks, batch, index):
    if masks.dtype is not _int64 or masks.dim() != 2 or masks.shape[0] != batch.tokens or not masks.is_contiguous():
        raise ValueError("%s is a contiguous int64 [%d, words] tensor" % (name, batch.tokens))
    if masks.get_device() != index:
        raise ValueError("%s is on %s, not on the call's device" % (name, masks.device))
    words = masks.shape[1]
    if not tree_words(batch) <= words <= SZ_TREE_WORDS:
        raise ValueError("%s has %d words a token; the batch's trees need %d, and %d are the most"
                         % (name, words, tree_words(batch), SZ_TREE_WORDS))
    return words


def tree_attention(q: torch.Tensor, cache: PagedCache, batch: PageBatch, masks: torch.Tensor, scale: float | None = None,
                   window: int = 0, out: torch.Tensor | None = None, lse=False, ws: torch.Tensor | None = None,
                   stream=None, check: bool = True):
    """``paged_attention`` for trees of drafted tokens (sz_tree_attention): a
    token sees what its sequence has cached before the new tokens, and of the
    new ones those that its row of ``masks`` (``draft_tree``; any masks will
    do) names.  With ``window`` > 0 a token that names c new ones sees the last
    window - max(c, 1) of the cached ones.  Where the
    batch's ``max_new`` times the query heads of a KV head is over 16,
    probabilities may be rounded to bfloat16, else they are held to 2^-15; its
    bounds (``max_kv`` too) decide, not its lengths."""
    words = _mask_words("masks", masks, batch, cache._index)
    return _attend("sz_tree_attention", _native.lib.sz_tree_attention, (masks.data_ptr(), words), q, cache, batch, scale,
                   window, out, lse, ws, stream, check)


def rotary_frequencies(dim: int, base: float = 10000.0, stretch: float = 1.0, original: int | None = None,
                       low: float = 1.0, high: float = 4.0) -> torch.Tensor:
    """float64 ``[dim / 2]`` frequencies base**(-2 i / dim), in radians a
    position.  ``stretch`` > 1 makes room for longer contexts: all frequencies
    divided by it (``original`` None), or by how often a context of
    ``original`` tokens holds a wavelength: ``high`` times or more, as it was;
    ``low`` times or less, divided; a linear blend of the two between."""
    if dim <= 0 or dim % 2 or not base > 0 or not stretch > 0:
        raise ValueError("dim is even and above 0, base and stretch above 0")
    f = float(base) ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    if original is None:
        return f / stretch
    if not high > low:
        raise ValueError("high is above low")
    keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
    return f * (keep + (1.0 - keep) / stretch)


# 2^160 / (2 pi), from pi to 50 places
_PER_TURN = 2 ** 160 * 10 ** 50 // (2 * 314159265358979323846264338327950288419716939937510)


def _turn(f: float) -> int:
    """f / 2 pi modulo 1, in units of 2^-64, as a signed 64-bit integer."""
    m, e = math.frexp(f)
    up = int(m * 2 ** 53) * _PER_TURN                    # f = m 2^e
    shift = 160 + 53 - 64 - e
    t = ((up + (1 << shift - 1) >> shift) if shift > 0 else up << -shift) % 2 ** 64
    return t - 2 ** 64 if t >= 2 ** 63 else t


class Rotary(_Fixed):
    """Rotary positions: ``frequencies`` (radians a position, one for each pair
    of the first ``2 * len(frequencies)`` values of a row; ``rotary_frequencies``),
    ``interleaved`` pairs (2d, 2d + 1) or else (d, d + dim / 2), and the factor
    ``amplitude`` of turned values.  Held on ``device`` (None: the frequencies'
    if that is a GPU, else the current GPU) as 64-bit fractions of a turn, so
    that angles are exact at any position."""

    _FIXED = frozenset(("turns", "dim", "interleaved", "amplitude", "device"))

    def __init__(self, frequencies: torch.Tensor, interleaved: bool = False, amplitude: float = 1.0, device=None):
        _plain("frequencies", frequencies)
        if frequencies.dim() != 1 or not frequencies.dtype.is_floating_point:
            raise ValueError("frequencies is one floating axis")
        dim = 2 * len(frequencies)
        if dim < 8 or dim % 8 or dim > 128:
            raise ValueError("4, 8, ... or 64 frequencies turn 8, 16, ... or 128 values, got %d" % len(frequencies))
        values = frequencies.double().tolist()
        if not all(map(math.isfinite, values)) or not abs(amplitude) < 2.0 ** 128 - 2.0 ** 103:
            raise ValueError("frequencies are finite, amplitude is in 32 bits")
        turns = torch.tensor([_turn(f) for f in values], dtype=torch.int64)
        if device is None:
            device = frequencies.device if frequencies.is_cuda else "cuda"
        turns = turns.to(device)
        c = _native.sz_rotary(turns.data_ptr(), dim, 1 if interleaved else 0, amplitude)
        self.__dict__.update(turns=turns, dim=dim, interleaved=bool(interleaved), amplitude=float(amplitude),
                             device=turns.device, _index=turns.get_device(), _c=c, _ref=ctypes.byref(c), _made=True)


def rotary_write(cache: PagedCache, batch: PageBatch, rotary: Rotary, q: torch.Tensor | None, k: torch.Tensor,
                 v: torch.Tensor, positions: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None,
                 check: bool = True):
    """``cache_write`` with rotary positions: turns the batch's queries and
    keys by their tokens' positions and writes keys and values into their pages
    (sz_rotary_write).  ``q`` (or None), ``k`` and ``v``: bfloat16 ``[tokens,
    heads, head_dim]`` with strides as in ``cache_write``.  ``positions`` int32
    ``[tokens]`` (a tree's, say) instead of the tokens' places.  Returns the
    turned queries, contiguous, or ``out``, which may be ``q`` itself; rows of
    tokens that belong to no sequence keep what they held.  With ``check`` the
    batch is looked at afterwards (a batch that writes a place twice is
    ``cache_check``'s to find)."""
    tokens = batch.tokens
    index = cache._index
    if rotary._index != index:
        raise ValueError("the rotary positions are on %s, the cache on %s" % (rotary.device, cache.device))
    if rotary.dim > cache.head_dim:
        raise ValueError("%d values of a row are turned, the cache's have %d" % (rotary.dim, cache.head_dim))
    at = None if positions is None else _ints("positions", positions, (tokens,), index)
    keys, values = _rows("k", k, tokens, cache.kv_heads, cache), _rows("v", v, tokens, cache.kv_heads, cache)
    owned = ()
    if q is None:
        if out is not None:
            raise ValueError("out is for queries, and there are none")
        args = (None, 0, 0, 0, None, 0, 0)
    else:
        if q.dim() != 3 or q.shape[1] == 0:
            raise ValueError("q is [tokens, q_heads, head_dim]")
        heads, dim = q.shape[1], cache.head_dim
        queries = _rows("q", q, tokens, heads, cache)
        if out is None:
            out = _empty_like(q, memory_format=_contiguous)
            owned = (out,)
            turned = (out.data_ptr(), heads * dim, dim)
        else:
            turned = _rows("out", out, tokens, heads, cache)
            _distinct(turned, tokens, heads, dim)
            if tokens and turned != queries and _rows_meet(turned, queries, tokens, heads, dim):
                raise ValueError("out shares memory with q without being q")
            for name, rows in (("k", keys), ("v", values)):
                if tokens and _spans_meet(turned, heads, rows, cache.kv_heads, tokens, dim):
                    raise ValueError("out shares memory with %s" % name)
        args = (queries[0], heads, *queries[1:], *turned)
    _run("sz_rotary_write", _native.lib.sz_rotary_write, cache, batch, (rotary._ref, at, *args, *keys, *values), stream,
         owned)
    if check:
        _raise_status(cache, stream)
    return out


def _distinct(rows, tokens, heads, dim):
    (near, count), (far, more) = sorted([(rows[1], tokens), (rows[2], heads)])
    if (count > 1 and near < dim) or (more > 1 and far < (count - 1) * near + dim):
        raise ValueError("out has rows that share memory")


def _spans_meet(out, heads, rows, row_heads, tokens, dim):
    """Whether rows of two tensors of different head counts share memory; with
    the same token stride each token's heads are looked at as one run."""
    (at, token, head), (bt, other, bhead) = out, rows
    run, brun = (heads - 1) * head + dim, (row_heads - 1) * bhead + dim          # a token's values, from its first row on
    if at + 2 * ((tokens - 1) * token + run) <= bt or bt + 2 * ((tokens - 1) * other + brun) <= at:
        return False
    if tokens > 1 and token != other:
        return True
    apart = (bt - at) // 2
    if tokens > 1:
        apart %= token
        return not (run <= apart and apart + brun <= token)
    return not (run <= apart or apart + brun <= 0)


class CacheLayers(_Fixed):
    """Caches of one shape, such as a model's layers, as one argument of
    ``cache_keep``.  ``status``: the first one's word, which calls on the layers
    report into."""

    _FIXED = frozenset(("caches", "status", "device"))

    def __init__(self, caches):
        caches = tuple(caches)
        if not caches or len(caches) > _native.SZ_KEEP_LAYERS:
            raise ValueError("1 to %d caches" % _native.SZ_KEEP_LAYERS)
        one = caches[0]
        shape = lambda c: (c.dtype, tuple(c.data.shape), c.device)
        if any(shape(c) != shape(one) for c in caches):
            raise ValueError("the caches differ in type, shape or device")
        spans = sorted((t.data_ptr(), t.nbytes) for c in caches for t in (c.data, c.scales) if t is not None)
        if any(a + n > b for (a, n), (b, _) in zip(spans, spans[1:])):
            raise ValueError("two of the caches share memory")
        c = (_native.sz_cache * len(caches))(*[c._c for c in caches])
        self.__dict__.update(caches=caches, status=one.status, device=one.device, _index=one._index, _c=c,
                             _ref=ctypes.cast(c, ctypes.POINTER(_native.sz_cache)), _made=True)


def cache_keep(caches, batch: PageBatch, kept: torch.Tensor, counts: torch.Tensor, stream=None, check: bool = True) -> None:
    """Moves the rows of the accepted new tokens to the places behind what their
    sequences had cached, in one cache or in ``CacheLayers`` (sz_cache_keep).
    ``kept`` int32 ``[seqs, width]``: the accepted tokens' indices among their
    sequence's new ones, ascending, ``counts`` int32 ``[seqs]`` how many.  The
    next lengths are kv_lens - n + counts."""
    layers = isinstance(caches, CacheLayers)
    one = caches.caches[0] if layers else caches
    index = one._index
    if batch._index != index:
        raise ValueError("the batch is on %s, the cache on %s" % (batch.device, one.device))
    if kept.dim() != 2:
        raise ValueError("kept is [seqs, width]")
    at = _ints("kept", kept, (batch.seqs, kept.shape[1]), index)
    many = _ints("counts", counts, (batch.seqs,), index)
    page = one.page_tokens
    _launch("sz_cache_keep", _native.lib.sz_cache_keep, index, one.device,
            (caches._ref, len(caches.caches) if layers else 1, batch._by_page.get(page) or batch._ref(page), at,
             kept.shape[1], many, one._status), stream)
    if check:
        _raise_status(one, stream)
