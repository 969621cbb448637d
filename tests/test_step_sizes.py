"""CPU checks of the sizes of workspaces: a caller asks for them before any call
has looked at its cache and batch, so no host field may end the process, and
what the calls refuse has no size."""
import ctypes
import itertools
import subprocess
import sys

from tests.conftest import ROOT
from tests.test_library_abi import _native
from tests.test_paged_host import ARG, BAD_CACHES, DTYPE, batch_of, cache_of, calls

TOP = 2 ** 32 - 1
ENDS = (0, 1, 2, 64, TOP)


def size_of(nat, c, b, q_heads):
    return nat.lib.sz_paged_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), q_heads)


def ask():
    """Sizes over the ends of every host field, of caches and batches that the
    calls refuse for most of them."""
    nat = _native()
    for kw, _ in BAD_CACHES:
        for b in ({}, dict(tokens=300, max_new=100, max_kv=100), dict(tokens=0), dict(seqs=0), dict(max_kv=0), dict(max_new=0)):
            size_of(nat, cache_of(nat, **kw), batch_of(nat, **b), 16)
    for dtype, dim, heads, group in itertools.product((0, 2, 7, TOP), ENDS + (96, 128), (1, 3, 1 << 16, 1 << 31), (1, 2, 1 << 16)):
        c = cache_of(nat, dtype=dtype, head_dim=dim, kv_heads=heads)
        for seqs, tokens, new, keys in itertools.product((0, 1, 1 << 24, 1 << 31, TOP), ENDS, (0, 1, 256, TOP), (0, 16, TOP)):
            b = batch_of(nat, seqs=seqs, tokens=tokens, max_new=new, max_kv=keys)
            size_of(nat, c, b, heads * group % 2 ** 32)
            nat.lib.sz_pages_assign_workspace_size(ctypes.byref(b))
        nat.lib.sz_cache_check_workspace_size(ctypes.byref(c))


def test_sizes_end_no_process():
    code = "import tests.test_step_sizes as t; t.ask()"
    assert subprocess.run([sys.executable, "-c", code], cwd=ROOT, timeout=600).returncode == 0


def test_what_the_calls_refuse_has_no_size():
    nat = _native()
    good = cache_of(nat), batch_of(nat)
    assert size_of(nat, *good, 16) >= 4096
    for kw in (dict(dtype=3), dict(dtype=TOP), dict(head_dim=0), dict(head_dim=96), dict(head_dim=256), dict(kv_heads=1025)):
        c = cache_of(nat, **kw)
        heads = 2 * c.kv_heads
        assert calls(nat, c, good[1], q_heads=heads)[2] in (ARG, DTYPE) and size_of(nat, c, good[1], heads) == 0, kw
    for kw in (dict(seqs=(1 << 24) + 1), dict(tokens=(1 << 30) + 1), dict(max_kv=(1 << 30) + 1, table_width=TOP)):
        b = batch_of(nat, **kw)
        assert calls(nat, good[0], b)[2] == ARG and size_of(nat, good[0], b, 16) == 0, kw
    assert calls(nat, *good, q_heads=1 << 16)[2] == ARG and size_of(nat, *good, 1 << 16) == 0
    # the ends of what they take have one
    c, b = cache_of(nat, kv_heads=1024, head_dim=64), batch_of(nat, seqs=1 << 24, tokens=1 << 30, max_new=1 << 30, max_kv=1 << 30)
    assert size_of(nat, c, b, 63 * 1024) >= 4096
