"""The least workspace that sz_paged_attention takes, found by bisection (the
null output is its last check, so nothing is launched), holds the counters and
the partials of as many chunks as the rule gives, worked out here on its own."""
import ctypes
import math

import pytest

from tests.test_library_abi import _native
from tests.test_paged_host import ARG, WORKSPACE, batch_of, cache_of, calls


def chunks(span, want):
    up = lambda x: -(-x // 128) * 128
    least = min(1024, up(-(-span // 64)))
    return max(1, -(-span // up(max(128, least, -(-span // max(1, want))))))


def rows_chunks(span, groups):
    return chunks(span, max(1024 // groups, min(3328 // groups, span // 1024)))


# seqs, tokens, max_new, max_kv, KV heads, query heads, head_dim, dtype, window, chunks by the rule
TOKENS = [(1, 1, 1, 65536, 4, 28, 128, 0), (64, 64, 1, 8192, 8, 32, 128, 2), (1, 1, 1, 1001, 8, 32, 128, 0),
          (3, 12, 4, 5000, 2, 8, 64, 1), (300, 300, 1, 700, 8, 8, 64, 0), (7, 7, 1, 129, 1, 1, 128, 0),
          (2, 2, 1, 128, 1, 16, 64, 0), (16, 80, 5, 6000, 2, 6, 64, 1)]


@pytest.mark.parametrize("shape", TOKENS)
@pytest.mark.parametrize("window", [0, 1000])
def test_single_tokens_and_drafts(shape, window):
    seqs, tokens, max_new, max_kv, heads, q_heads, dim, dtype = shape
    span = min(max_kv, window + max_new + 63) if window else max_kv
    check(shape, window, rows_chunks(span, seqs * heads))


# 4 waves of 32 rows each: slots of 128 rows, as many as tokens x group fill and one more a sequence
TILES = [(1, 512, 512, 16896, 8, 32, 128, 1), (1, 20, 20, 1500, 2, 8, 128, 0), (8, 512, 64, 1064, 8, 32, 64, 0),
         (2, 140, 70, 90000, 1, 4, 128, 0)]


@pytest.mark.parametrize("shape", TILES)
def test_prompts(shape):
    seqs, tokens, max_new, max_kv, heads, q_heads, dim, dtype = shape
    group = q_heads // heads
    assert not (dtype and tokens * group >= 256 * seqs and tokens * q_heads >= 256 * 256)       # four waves
    groups = (tokens * group // 128 + seqs) * heads
    want = min(2048 // 4 // groups, int(math.sqrt(12500 * max_kv / (tokens * q_heads * dim))))
    assert tokens == seqs * max_new or seqs == 1                # no sequence of few rows beside them
    check(shape, 0, chunks(max_kv, want))


def check(shape, window, splits):
    nat = _native()
    seqs, tokens, max_new, max_kv, heads, q_heads, dim, dtype = shape
    c = cache_of(nat, dtype=dtype, kv_heads=heads, head_dim=dim)
    b = batch_of(nat, seqs=seqs, tokens=tokens, max_new=max_new, max_kv=max_kv, table_width=-(-max_kv // 16))
    takes = lambda n: calls(nat, c, b, q_heads=q_heads, token=q_heads * dim, head=dim, window=window, ws_bytes=n, out=None)[2]
    size = nat.sz_paged_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), q_heads)
    assert takes(size) == ARG
    low, high = 0, size                                         # low is refused, high is taken
    while high - low > 1:
        mid = (low + high) // 2
        code = takes(mid)
        assert code in (ARG, WORKSPACE)
        low, high = (mid, high) if code == WORKSPACE else (low, mid)
    rows = tokens * q_heads
    partials = 0 if splits == 1 else splits * rows * (dim * 4 + 8)
    assert 4096 + partials <= high <= 4096 + partials + (512 if partials else 0), (splits, high)
    assert takes(high - 1) == WORKSPACE
