"""CPU checks of the calls of a serving step: every refusal of the C ABI and of
the Python layer (nothing is launched), the ends of what a tree's masks and
frequencies may be, and the test reference against hand-worked values."""
import ctypes
import itertools
import math

import pytest
import torch

import tests.stepref as step
from tests.test_library_abi import _native
from tests.test_paged_host import (ALIGN, ARG, BAD_BATCHES, BAD_CACHES, DTYPE, DUMMY, WORKSPACE, batch_of, cache_of)


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


def rotary_of(nat, **kw):
    f = dict(d_turns=DUMMY, dim=128, interleaved=0, amplitude=1.0)
    f.update(kw)
    return nat.sz_rotary(**f)


def pool_of(nat, **kw):
    f = dict(page_tokens=16, pages=10, queue=DUMMY, ends=DUMMY)
    f.update(kw)
    return nat.sz_pool(**f)


def write(nat, c, b, r, status=DUMMY, **kw):
    f = dict(positions=DUMMY, q=DUMMY, heads=16, q_token=4096, q_head=128, out=DUMMY, out_token=2048, out_head=128, k=DUMMY,
             k_token=1024, k_head=128, v=DUMMY, v_token=1024, v_head=128)
    f.update(kw)
    ref = lambda x: ctypes.byref(x) if x is not None else None
    return nat.lib.sz_rotary_write(ref(c), ref(b), ref(r), f["positions"], f["q"], f["heads"], f["q_token"], f["q_head"],
                                   f["out"], f["out_token"], f["out_head"], f["k"], f["k_token"], f["k_head"], f["v"],
                                   f["v_token"], f["v_head"], status, None)


def attend(nat, c, b, status=DUMMY, **kw):
    f = dict(masks=DUMMY, words=1, q=DUMMY, q_heads=16, token=2048, head=128, scale=1.0, window=0, out=DUMMY, lse=DUMMY,
             ws=DUMMY, ws_bytes=1 << 40)
    f.update(kw)
    ref = lambda x: ctypes.byref(x) if x is not None else None
    return nat.lib.sz_tree_attention(ref(c), ref(b), f["masks"], f["words"], f["q"], f["q_heads"], f["token"], f["head"],
                                     f["scale"], f["window"], f["out"], f["lse"], f["ws"], f["ws_bytes"], status, None)


def keep(nat, c, b, status=DUMMY, layers=1, **kw):
    f = dict(kept=DUMMY, width=4, counts=DUMMY)
    f.update(kw)
    many = (nat.sz_cache * max(len(c), 1))(*c) if c is not None else None
    return nat.lib.sz_cache_keep(many, layers, ctypes.byref(b) if b is not None else None, f["kept"], f["width"], f["counts"],
                                 status, None)


def tree(nat, b, status=DUMMY, **kw):
    f = dict(parents=DUMMY, masks=DUMMY, words=1, positions=DUMMY)
    f.update(kw)
    return nat.lib.sz_draft_tree(ctypes.byref(b) if b is not None else None, f["parents"], f["masks"], f["words"],
                                 f["positions"], status, None)


def assign(nat, p, b, status=DUMMY, **kw):
    f = dict(held=DUMMY, held_out=DUMMY, ends_out=DUMMY, slots=None, ws=DUMMY, ws_bytes=1 << 30)
    f.update(kw)
    ref = lambda x: ctypes.byref(x) if x is not None else None
    return nat.lib.sz_pages_assign(ref(p), ref(b), f["held"], f["held_out"], f["ends_out"], f["slots"], f["ws"],
                                   f["ws_bytes"], status, None)


def test_bad_caches_and_batches_are_refused():
    nat = _native()
    for kw, code in BAD_CACHES:
        c, b = cache_of(nat, **kw), batch_of(nat)
        if kw == dict(head_dim=256):
            continue
        assert write(nat, c, b, rotary_of(nat, dim=64)) == code, kw
        assert attend(nat, c, b) == code, kw
        assert keep(nat, [c], b) == code, kw
    for kw, code in BAD_BATCHES:
        c, b = cache_of(nat), batch_of(nat, **kw)
        assert write(nat, c, b, rotary_of(nat)) == code, kw
        assert attend(nat, c, b) == code, kw
        assert keep(nat, [c], b) == code, kw
        assert assign(nat, pool_of(nat), b) == code, kw
        if "max_kv" not in kw:
            assert tree(nat, b) == code, kw
    good = batch_of(nat)
    assert write(nat, None, good, rotary_of(nat)) == ARG and write(nat, cache_of(nat), None, rotary_of(nat)) == ARG
    assert attend(nat, None, good) == ARG and attend(nat, cache_of(nat), None) == ARG
    assert keep(nat, None, good) == ARG and keep(nat, [cache_of(nat)], None) == ARG
    assert assign(nat, None, good) == ARG and assign(nat, pool_of(nat), None) == ARG and tree(nat, None) == ARG
    for call in (lambda s: write(nat, cache_of(nat), good, rotary_of(nat), s), lambda s: attend(nat, cache_of(nat), good, s),
                 lambda s: keep(nat, [cache_of(nat)], good, s), lambda s: assign(nat, pool_of(nat), good, s)):
        assert call(None) == ARG and call(DUMMY + 2) == ALIGN
    assert tree(nat, good, DUMMY + 2) == ALIGN


def test_bad_rotary_writes_are_refused():
    nat = _native()
    c, b = cache_of(nat), batch_of(nat)
    assert write(nat, c, b, None) == ARG
    for kw in (dict(d_turns=None), dict(dim=0), dict(dim=4), dict(dim=12), dict(dim=136), dict(interleaved=2),
               dict(amplitude=math.nan), dict(amplitude=math.inf), dict(amplitude=1e39)):
        assert write(nat, c, b, rotary_of(nat, **kw)) == ARG, kw
    assert write(nat, cache_of(nat, head_dim=64), b, rotary_of(nat, dim=72)) == ARG
    assert write(nat, c, b, rotary_of(nat, d_turns=DUMMY + 4)) == ALIGN
    assert write(nat, c, b, rotary_of(nat), positions=DUMMY + 2) == ALIGN
    for name in ("q", "out", "k", "v"):
        assert write(nat, c, b, rotary_of(nat), **{name: None}) == ARG, name
        assert write(nat, c, b, rotary_of(nat), **{name: DUMMY + 8}) == ALIGN, name
        assert write(nat, c, b, rotary_of(nat), **{name + "_token": 1028}) == ALIGN, name
        assert write(nat, c, b, rotary_of(nat), **{name + "_head": 4}) == ALIGN, name
        assert write(nat, c, b, rotary_of(nat), **{name + "_head": 1 << 40}) == ARG, name
    assert write(nat, c, b, rotary_of(nat), heads=1 << 16) == ARG
    wide = batch_of(nat, tokens=1 << 30)                                 # more threads than a launch has
    assert write(nat, cache_of(nat, kv_heads=1024), wide, rotary_of(nat)) == ARG


def test_bad_tree_calls_are_refused():
    nat = _native()
    c, b = cache_of(nat), batch_of(nat)
    for kw in (dict(words=0), dict(words=17), dict(masks=None), dict(q=None), dict(q_heads=12), dict(q_heads=0),
               dict(scale=0.0), dict(scale=math.nan), dict(window=1 << 31), dict(out=None), dict(ws=None)):
        assert attend(nat, c, b, **kw) == ARG, kw
    for kw in (dict(masks=DUMMY + 4), dict(q=DUMMY + 8), dict(out=DUMMY + 8), dict(ws=DUMMY + 8), dict(lse=DUMMY + 2)):
        assert attend(nat, c, b, **kw) == ALIGN, kw
    assert attend(nat, c, b, ws_bytes=4095) == WORKSPACE
    many = batch_of(nat, tokens=65, max_new=65, table_width=8, max_kv=128)
    assert attend(nat, c, many) == ARG and tree(nat, many) == ARG          # 65 tokens do not fit a word
    for kw in (dict(words=0), dict(words=17), dict(parents=None), dict(masks=None), dict(positions=None)):
        assert tree(nat, b, **kw) == ARG, kw
    assert tree(nat, batch_of(nat, seqs=1 << 24, tokens=1 << 30, max_new=1000), words=16) == ARG   # more threads than a launch has
    for kw in (dict(parents=DUMMY + 2), dict(masks=DUMMY + 4), dict(positions=DUMMY + 1)):
        assert tree(nat, b, **kw) == ALIGN, kw


def test_bad_keeps_and_assignments_are_refused():
    nat = _native()
    c, b = cache_of(nat), batch_of(nat)
    assert keep(nat, [c], b, layers=0) == ARG and keep(nat, [c], b, layers=4097) == ARG
    for kw in (dict(kept=None), dict(counts=None), dict(width=(1 << 30) + 1)):
        assert keep(nat, [c], b, **kw) == ARG, kw
    for kw in (dict(kept=DUMMY + 2), dict(counts=DUMMY + 1)):
        assert keep(nat, [c], b, **kw) == ALIGN, kw
    for kw in (dict(dtype=1), dict(page_tokens=32), dict(kv_heads=4), dict(head_dim=64), dict(pages=11)):
        assert keep(nat, [c, cache_of(nat, **kw)], b, layers=2) == ARG, kw
    assert keep(nat, [c, cache_of(nat, data=None)], b, layers=2) == ARG
    wide = batch_of(nat, seqs=1 << 24)
    assert keep(nat, [cache_of(nat, kv_heads=1024)], wide) == ARG          # more threads than a launch has
    for kw in (dict(page_tokens=8), dict(page_tokens=48), dict(pages=0), dict(pages=(1 << 30) + 1), dict(queue=None),
               dict(ends=None)):
        assert assign(nat, pool_of(nat, **kw), b) == ARG, kw
    for kw in (dict(held=None), dict(held_out=None), dict(ends_out=None), dict(ws=None)):
        assert assign(nat, pool_of(nat), b, **kw) == ARG, kw
    for kw in (dict(held=DUMMY + 2), dict(held_out=DUMMY + 1), dict(ends_out=DUMMY + 2), dict(slots=DUMMY + 4),
               dict(ws=DUMMY + 8)):
        assert assign(nat, pool_of(nat), b, **kw) == ALIGN, kw
    for kw in (dict(queue=DUMMY + 2), dict(ends=DUMMY + 2)):
        assert assign(nat, pool_of(nat, **kw), b) == ALIGN, kw
    assert assign(nat, pool_of(nat), b, ws_bytes=nat.sz_pages_assign_workspace_size(ctypes.byref(b)) - 1) == WORKSPACE
    assert nat.lib.sz_pages_assign_workspace_size(None) == 0


def test_nothing_to_do_is_no_error():
    nat = _native()
    c = cache_of(nat)
    for b in (batch_of(nat, tokens=0, max_new=0), batch_of(nat, seqs=0, tokens=0, starts=None, kv_lens=None, page_table=None)):
        assert write(nat, c, b, rotary_of(nat), q=None, out=None, k=None, v=None) == 0
        assert attend(nat, c, b, masks=None, q=None, out=None, ws=None) == 0
        assert keep(nat, [c], b) == 0
        assert tree(nat, b, parents=None, masks=None, positions=None) == 0
    assert keep(nat, [c], batch_of(nat), width=0, kept=None, counts=None) == 0


def test_attention_workspace_covers_trees_of_many_shapes():
    """The size that attention_workspace reports is enough for a tree of any
    window, and a call says so where it is not."""
    import random
    nat = _native()
    rnd = random.Random(3)
    short = 0
    for _ in range(600):
        heads, dim, page = rnd.choice([1, 2, 3, 8]), rnd.choice([64, 128]), rnd.choice([16, 64])
        c = cache_of(nat, dtype=rnd.choice([0, 1, 2]), kv_heads=heads, head_dim=dim, page_tokens=page)
        seqs, new = int(2 ** rnd.uniform(0, 9)), int(2 ** rnd.uniform(0, 9))
        width = int(2 ** rnd.uniform(0, 12))
        max_kv = max(1, int(width * page * rnd.uniform(0.3, 1)))
        tokens = max(1, int(seqs * new * rnd.choice([1, rnd.random()])))
        q_heads = heads * rnd.choice([1, 2, 4, 7, 8])
        b = batch_of(nat, seqs=seqs, table_width=width, tokens=tokens, max_new=new, max_kv=max_kv)
        n = nat.lib.sz_paged_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), q_heads)
        kw = dict(words=8, q_heads=q_heads, token=q_heads * dim, head=dim, out=None)           # no output: the last refusal
        for window in (0, 1, rnd.randint(1, max_kv), (1 << 31) - 1):
            assert attend(nat, c, b, ws_bytes=n, window=window, **kw) == ARG
            least = attend(nat, c, b, ws_bytes=4096, window=window, **kw)
            assert least in (ARG, WORKSPACE)
            short += least == WORKSPACE
    assert short > 100                                       # shapes that are split are among them


def test_bounds_of_nothing_are_planned():
    """Bounds that leave no new token, no key or one of them: the size covers
    the call, which goes as far as its last refusal."""
    nat = _native()
    for dtype, heads, dim in itertools.product((0, 1, 2), (1, 1024), (64, 128)):
        c = cache_of(nat, dtype=dtype, kv_heads=heads, head_dim=dim)
        for seqs, tokens, new, max_kv, group in itertools.product((1, 3, 1 << 24), (1, 5), (0, 1), (0, 1, 16), (1, 63)):
            b = batch_of(nat, seqs=seqs, tokens=tokens, max_new=new, max_kv=max_kv)
            q_heads = heads * group
            n = nat.lib.sz_paged_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), q_heads)
            assert n >= 4096
            assert attend(nat, c, b, ws_bytes=n, q_heads=q_heads, token=q_heads * dim, head=dim, out=None) == ARG


def small():
    import fp8_kv_cache_sz_amd as sz
    table, kv, starts = torch.zeros(2, 2, dtype=torch.int32), ints([3, 4]), ints([0, 1, 2])
    return sz, sz.paged_cache(4, 16, 2, 64, sz.E5M2, device="cpu"), sz.PageBatch(table, kv, starts, 2)


def test_python_layer_refuses_trees():
    sz, cache, batch = small()
    parents = ints([-1, -1])
    for bad in (parents.long(), parents[:1], ints([[-1, -1]])):
        with pytest.raises(ValueError):
            sz.draft_tree(batch, bad, check=False)
    masks, positions = torch.zeros(2, 1, dtype=torch.int64), parents.clone()
    for out in ((masks.int(), positions), (masks[:1], positions), (masks[:, :0], positions), (masks, positions.long()),
                (torch.zeros(2, 17, dtype=torch.int64), positions), (masks.expand(2, 2), positions), (masks, parents)):
        with pytest.raises(ValueError):
            sz.draft_tree(batch, parents, out=out, check=False)
    eight = torch.zeros(8, dtype=torch.int32)
    for p, out in ((eight[:2], (masks, eight[1:3])), (eight[:2], (eight[:4].view(torch.int64).view(2, 1), positions)),
                   (parents, (eight[:4].view(torch.int64).view(2, 1), eight[3:5]))):
        with pytest.raises(ValueError, match="share memory"):
            sz.draft_tree(batch, p, out=out, check=False)
    with pytest.raises(ValueError, match="runs on the GPU"):             # side by side
        sz.draft_tree(batch, eight[:2], out=(eight[2:6].view(torch.int64).view(2, 1), eight[6:8]), check=False)
    for status in (torch.zeros(2, dtype=torch.int32), torch.zeros(1)):
        with pytest.raises(ValueError):
            sz.draft_tree(batch, parents, status=status, check=False)
    with pytest.raises(ValueError):                                      # nothing of this runs on the CPU
        sz.draft_tree(batch, parents, check=False)
    big = sz.PageBatch(torch.zeros(1, 1, dtype=torch.int32), ints([3]), ints([0, 2]), 2000)
    with pytest.raises(ValueError):
        sz.draft_tree(big, torch.zeros(2000, dtype=torch.int32), check=False)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for bad in (masks.int(), masks[:1], masks[0], torch.zeros(2, 17, dtype=torch.int64)):
        with pytest.raises(ValueError):
            sz.tree_attention(q, cache, batch, bad, check=False)
    for bad in (q.float(), q[:1], q[:, :3]):
        with pytest.raises((TypeError, ValueError)):
            sz.tree_attention(bad, cache, batch, masks, check=False)
    with pytest.raises(ValueError):
        sz.tree_attention(q, cache, batch, masks, window=-1, check=False)
    with pytest.raises(ValueError):
        sz.tree_attention(q.requires_grad_(), cache, batch, masks, check=False)
    assert sz.tree_words(batch) == 1
    assert sz.tree_words(sz.PageBatch(torch.zeros(1, 1, dtype=torch.int32), ints([3]), ints([0, 2]), 65)) == 2


def test_python_layer_refuses_rotary():
    sz, cache, batch = small()
    f = sz.rotary_frequencies(64)
    for bad in (f[:3], f[None], f.long(), torch.ones(68), torch.tensor([1.0, math.nan, 1.0, 1.0]), f[:0]):
        with pytest.raises(ValueError):
            sz.Rotary(bad, device="cpu")
    for bad in (math.inf, -math.inf, math.nan, 1e39):
        with pytest.raises(ValueError):
            sz.Rotary(f, amplitude=bad, device="cpu")
    with pytest.raises(ValueError):
        sz.Rotary(f.clone().requires_grad_(), device="cpu")
    for bad in (dict(dim=0), dict(dim=7), dict(dim=8, base=0.0), dict(dim=8, stretch=0.0),
                dict(dim=8, original=10, low=4.0, high=4.0)):
        with pytest.raises(ValueError):
            sz.rotary_frequencies(**bad)
    rotary = sz.Rotary(f, device="cpu")
    with pytest.raises(AttributeError):
        rotary.dim = 32
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    k = x[:, :2].contiguous()
    ok = lambda **kw: sz.rotary_write(cache, batch, rotary, **{**dict(q=x, k=k, v=k.clone(), check=False), **kw})
    for bad in (dict(q=x.float()), dict(q=x[:1]), dict(q=x[0]), dict(q=x[:, :0]), dict(k=x), dict(v=k[:1]), dict(k=k.float()),
                dict(positions=torch.zeros(2)), dict(positions=ints([0])), dict(out=x.float()), dict(out=x[:, :3]),
                dict(q=None, out=x), dict(out=torch.zeros(1, 4, 64, dtype=torch.bfloat16).expand(2, 4, 64)),
                dict(q=x.clone().requires_grad_()), dict(out=x.clone().requires_grad_())):
        with pytest.raises((TypeError, ValueError)):
            ok(**bad)
    wide = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="shares memory with q"):        # shifted by a head
        ok(q=wide[:, :4], out=wide[:, 1:5])
    with pytest.raises(ValueError, match="shares memory with k"):
        ok(q=wide[:, :4], k=wide[:, 6:], out=wide[:, 4:])
    with pytest.raises(ValueError, match="shares memory with v"):
        ok(q=wide[:, :4], v=wide[:, 2:4], out=wide[:, :4])
    with pytest.raises(ValueError, match="runs? on the GPU"):            # distinct, so only the device is wrong
        ok(q=wide[:, :4], k=wide[:, 4:6], v=wide[:, 6:], out=wide[:, :4])
    with pytest.raises(ValueError, match="runs? on the GPU"):
        ok()
    with pytest.raises(ValueError):
        sz.rotary_write(cache, batch, sz.Rotary(sz.rotary_frequencies(128), device="cpu"), x, k, k, check=False)


def test_python_layer_refuses_pools_and_keeps():
    sz, cache, batch = small()
    queue, ends, held = ints(range(4)), ints([0, 4]), ints([0, 0])
    for bad in ((16, queue.long(), ends), (16, queue[None], ends), (16, queue, ends[:1]), (16, queue, ends.long()),
                (24, queue, ends), (8, queue, ends), (16, queue[:0], ends), (16, queue, ends, torch.zeros(1))):
        with pytest.raises(ValueError):
            sz.PagePool(*bad)
    pool = sz.PagePool(16, queue, ends)
    with pytest.raises(AttributeError):
        pool.queue = queue.clone()
    ws = torch.zeros(1024, dtype=torch.uint8)
    ok = lambda **kw: sz.pages_assign(pool, batch, **{**dict(held=held, ws=ws, check=False), **kw})
    for bad in (dict(held=held.long()), dict(held=held[:1]), dict(held_out=held[:1]), dict(ends_out=held[:1]),
                dict(slots=torch.zeros(2, dtype=torch.int32)), dict(slots=torch.zeros(3, dtype=torch.int64)),
                dict(ws=ws[::2])):
        with pytest.raises(ValueError):
            ok(**bad)
    three = ints([0, 0, 0])
    with pytest.raises(ValueError, match="shares memory"):
        ok(held=three[:2], held_out=three[1:])
    with pytest.raises(ValueError, match="shares memory"):
        sz.pages_assign(sz.PagePool(16, queue, three[:2]), batch, held, ends_out=three[1:], ws=ws, check=False)
    with pytest.raises(ValueError, match="runs on the GPU"):
        ok()
    other = sz.paged_cache(4, 16, 2, 64, sz.E5M2, device="cpu")
    for bad in ((), (cache, cache), (cache, sz.paged_cache(5, 16, 2, 64, sz.E5M2, device="cpu")),
                (cache, sz.paged_cache(4, 16, 2, 64, sz.E4M3, device="cpu")),
                (cache, sz.PagedCache(sz.E5M2, other.data, cache.scales))):
        with pytest.raises(ValueError):
            sz.CacheLayers(bad)
    layers = sz.CacheLayers([cache, other])
    kept, counts = ints([[0], [0]]), ints([1, 1])
    for bad in ((kept.long(), counts), (kept[0], counts), (kept[:1], counts), (kept, counts[:1]), (kept, counts.long())):
        with pytest.raises(ValueError):
            sz.cache_keep(layers, batch, *bad, check=False)
    with pytest.raises(ValueError, match="runs on the GPU"):
        sz.cache_keep(layers, batch, kept, counts, check=False)


def test_turns_are_the_nearest_fractions():
    """2^64 f / 2 pi, by hand: a turn, a half, pi / 2^k and more than a turn."""
    import fp8_kv_cache_sz_amd as sz
    f = torch.tensor([math.pi, 2 * math.pi, 0.0, 1.0, -1.0, 8 * math.pi, 1e-30, 3.0], dtype=torch.float64)
    got = [int(t) % 2 ** 64 for t in sz.Rotary(f, device="cpu").turns]
    near = lambda x, y: min((x - y) % 2 ** 64, (y - x) % 2 ** 64)
    # math.pi is pi (1 - 3.9e-17): 2^63 (1 - 3.9e-17) is 359 short of 2^63
    assert near(got[0], 2 ** 63) == 360 or near(got[0], 2 ** 63) == 359
    assert near(got[1], 0) in (718, 719, 720) and got[2] == 0
    one = 2935890503282001226                               # 2^64 / (2 pi) = 2935890503282001226.39...
    assert near(got[3], one) <= 1 and near(got[4], -one) <= 1 and got[6] == 0
    assert near(got[5], 0) in range(2870, 2881) and near(got[7], 3 * one) <= 3


def test_references_by_hand():
    # two sequences: one grows from 1 page to 3, one gives one of 2 back; the ring wraps
    q, e, t, h, short, wrong = step.assign(16, ints([7, -9, -9, 5]), ints([3, 2]), ints([[2, -5, -5], [0, 1, -5]]),
                                           ints([33, 16]), ints([1, 2]), 3, 48)
    assert (q, e, t, h, short, wrong) == ([7, 1, -9, 5], [1, 1], [[2, 5, 7], [0, 1, -5]], [3, 1], False, False)
    assert step.slots(16, 8, t, [33, 16], [1, 3, 4], 5) == [-1, 5 * 16 + 15, 7 * 16, 15, -1]
    # 0 - 1 - 3, 0 - 2
    rows, wrong = step.tree([-1, 0, 0, 1], [10], [0, 4], 1)
    assert [rows[t] for t in range(4)] == [([1], 6), ([3], 7), ([5], 7), ([11], 8)] and not wrong
    cos, sin = step.angles([0, 1, 2 ** 31 - 1], [1.0])
    assert cos[0, 0] == 1.0 and sin[0, 0] == 0.0 and cos[1, 0] == math.cos(1.0)
    assert abs(float(cos[2, 0]) - math.cos(2 ** 31 - 1)) < 1e-9
    x = torch.zeros(3, 1, 4, dtype=torch.float64)
    x[1, 0] = torch.tensor([1.0, 2.0, 3.0, 4.0])
    a, size = step.turned(x, cos, sin, False, 2.0)
    c, s = math.cos(1.0), math.sin(1.0)
    assert torch.allclose(a[1, 0], torch.tensor([2 * (c - 2 * s), 2 * (2 * c + s), 3.0, 4.0], dtype=torch.float64))
    assert size[1, 0].tolist() == [6.0, 6.0, 0.0, 0.0]
