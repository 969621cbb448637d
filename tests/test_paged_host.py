"""CPU checks of the paged cache: every refusal of the C ABI and of the Python
layer (nothing is launched), workspace sizes, and the test reference against
hand-worked values."""
import ctypes
import math

import pytest
import torch

import tests.pagedref as ref
from tests.test_library_abi import _native

DUMMY = 1 << 20                # never dereferenced: every call below fails a host check first
ARG, DTYPE, ALIGN, WORKSPACE = -1, -2, -4, -7


def cache_of(nat, **kw):
    f = dict(dtype=0, page_tokens=16, kv_heads=8, head_dim=128, pages=10, data=DUMMY, scales=DUMMY)
    f.update(kw)
    return nat.sz_cache(**f)


def batch_of(nat, **kw):
    f = dict(page_table=DUMMY, kv_lens=DUMMY, starts=DUMMY, seqs=2, table_width=4, tokens=3, max_new=2, max_kv=64)
    f.update(kw)
    return nat.sz_batch(**f)


BAD_CACHES = [
    (dict(dtype=3), DTYPE), (dict(dtype=9), DTYPE), (dict(head_dim=96), ARG), (dict(head_dim=256), ARG),
    (dict(head_dim=0), ARG), (dict(page_tokens=8), ARG), (dict(page_tokens=24), ARG), (dict(page_tokens=2048), ARG),
    (dict(page_tokens=0), ARG), (dict(kv_heads=0), ARG), (dict(kv_heads=1025), ARG), (dict(pages=0), ARG),
    (dict(pages=1 << 31), ARG), (dict(data=None), ARG), (dict(data=DUMMY + 8), ALIGN),
    (dict(dtype=1, scales=None), ARG), (dict(dtype=2, scales=DUMMY + 4), ALIGN),
]
BAD_BATCHES = [
    (dict(starts=None), ARG), (dict(kv_lens=None), ARG), (dict(page_table=None), ARG), (dict(starts=DUMMY + 2), ALIGN),
    (dict(kv_lens=DUMMY + 1), ALIGN), (dict(page_table=DUMMY + 2), ALIGN), (dict(max_kv=65), ARG),
    (dict(max_kv=(1 << 30) + 1, table_width=1 << 31), ARG), (dict(tokens=(1 << 30) + 1), ARG),
    (dict(seqs=(1 << 24) + 1), ARG),
]


def calls(nat, c, b, status=DUMMY, **kw):
    """The three calls on one cache and batch, with good other arguments."""
    f = dict(k=DUMMY, q=DUMMY, token=1024, head=128, out=DUMMY, ws=DUMMY, ws_bytes=1 << 40, q_heads=16, scale=1.0,
             window=0, lse=DUMMY)
    f.update(kw)
    lib, c, b = nat.lib, ctypes.byref(c) if c is not None else None, ctypes.byref(b) if b is not None else None
    move = (c, b, f["k"], f["token"], f["head"], DUMMY, 1024, 128, status, None)
    return [lib.sz_cache_write(*move), lib.sz_cache_read(*move),
            lib.sz_paged_attention(c, b, f["q"], f["q_heads"], f["token"], f["head"], f["scale"], f["window"], f["out"],
                                   f["lse"], f["ws"], f["ws_bytes"], status, None)]


def test_bad_caches_and_batches_are_refused():
    nat = _native()
    for kw, code in BAD_CACHES:
        c, b = cache_of(nat, **kw), batch_of(nat)
        assert calls(nat, c, b) == [code] * 3, kw
        assert nat.lib.sz_cache_check(ctypes.byref(c), ctypes.byref(b), DUMMY, 1 << 40, DUMMY, None) == code, kw
    for kw, code in BAD_BATCHES:
        c, b = cache_of(nat), batch_of(nat, **kw)
        assert calls(nat, c, b) == [code] * 3, kw
        assert nat.lib.sz_cache_check(ctypes.byref(c), ctypes.byref(b), DUMMY, 1 << 40, DUMMY, None) == code, kw
    c, b = cache_of(nat), batch_of(nat)
    assert calls(nat, None, b) == [ARG] * 3 and calls(nat, c, None) == [ARG] * 3
    assert calls(nat, c, b, status=None) == [ARG] * 3
    assert calls(nat, c, b, status=DUMMY + 2) == [ALIGN] * 3


def test_bad_tensors_and_parameters_are_refused():
    nat = _native()
    c, b = cache_of(nat), batch_of(nat)
    assert calls(nat, c, b, k=None, q=None) == [ARG] * 3
    assert calls(nat, c, b, k=DUMMY + 2, q=DUMMY + 2) == [ALIGN] * 3
    assert calls(nat, c, b, token=1020) == [ALIGN] * 3 and calls(nat, c, b, head=129) == [ALIGN] * 3
    assert calls(nat, c, b, token=1 << 40) == [ARG] * 3
    attend = lambda **kw: calls(nat, c, b, **dict(dict(k=None), **kw))[2]
    for kw, code in [(dict(q_heads=0), ARG), (dict(q_heads=12), ARG), (dict(q_heads=1 << 16), ARG), (dict(scale=0.0), ARG),
                     (dict(scale=-1.0), ARG), (dict(scale=math.nan), ARG), (dict(scale=math.inf), ARG),
                     (dict(window=1 << 31), ARG), (dict(out=None), ARG), (dict(out=DUMMY + 8), ALIGN),
                     (dict(lse=DUMMY + 2), ALIGN), (dict(ws=None), ARG), (dict(ws=DUMMY + 8), ALIGN)]:
        assert attend(**kw) == code, kw
    # more workgroups than a launch takes
    huge = batch_of(nat, seqs=1 << 24, table_width=1 << 20, max_kv=1 << 24)
    assert calls(nat, cache_of(nat, kv_heads=1024), huge, q_heads=1024)[2] == ARG
    check = lambda ws, n: nat.lib.sz_cache_check(ctypes.byref(c), ctypes.byref(b), ws, n, DUMMY, None)
    assert nat.sz_cache_check_workspace_size(ctypes.byref(c)) == 256
    assert check(None, 256) == ARG and check(DUMMY + 4, 256) == ALIGN and check(DUMMY, 255) == WORKSPACE


def test_attention_workspace_is_checked_and_covers_every_window():
    """The size that the library asks for is enough for any window, and the
    calls refuse one byte less than they use."""
    nat = _native()
    for c, b, heads in [(cache_of(nat), batch_of(nat, seqs=1, tokens=1, max_new=1, max_kv=65536, table_width=4096), 32),
                        (cache_of(nat), batch_of(nat, seqs=3, tokens=90, max_new=60, max_kv=5000, table_width=400), 16),
                        (cache_of(nat, dtype=2), batch_of(nat, seqs=64, tokens=64, max_new=1, max_kv=8192,
                                                          table_width=512), 32)]:
        size = nat.sz_paged_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), heads)
        assert size >= 4096 and size % 256 == 0
        for window in (0, 1, 16, 100, 129, 1000, 4096, 70000):
            assert calls(nat, c, b, q_heads=heads, window=window, ws_bytes=4095)[2] == WORKSPACE
            # a call that fails its very last check would have passed the
            # workspace's: the pointer is never reached on this machine
            assert calls(nat, c, b, q_heads=heads, window=window, ws_bytes=size, out=None)[2] == ARG
    c, b = cache_of(nat), batch_of(nat)
    assert nat.sz_paged_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), 12) == 0
    assert nat.sz_paged_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), 0) == 0


def test_nothing_to_do_is_no_error():
    nat = _native()
    c = cache_of(nat)
    for kw in (dict(tokens=0, max_new=0), dict(seqs=0, starts=None, kv_lens=None, page_table=None)):
        b = batch_of(nat, **kw)
        assert calls(nat, c, b) == [0] * 3, kw


def test_python_layer_refuses():
    import fp8_kv_cache_sz_amd as sz
    H, D, P = 2, 64, 16
    data = torch.zeros(4, 2, H, P, D, dtype=torch.bfloat16)
    byte = torch.zeros(4, 2, H, P, D, dtype=torch.uint8)
    scales = torch.zeros(4, 2, H, P, dtype=torch.uint8)
    with pytest.raises(ValueError):
        sz.PagedCache(7, data)
    with pytest.raises(TypeError):
        sz.PagedCache(sz.BF16, byte)
    with pytest.raises(TypeError):
        sz.PagedCache(sz.E4M3, data, scales)
    with pytest.raises(TypeError):
        sz.PagedCache(sz.E4M3, byte.view(torch.float8_e5m2), scales)
    with pytest.raises(ValueError):
        sz.PagedCache(sz.BF16, data[:, :1])
    with pytest.raises(ValueError):
        sz.PagedCache(sz.BF16, data.transpose(2, 3))
    with pytest.raises(ValueError):
        sz.PagedCache(sz.BF16, data, scales)
    with pytest.raises(ValueError):
        sz.PagedCache(sz.E5M2, byte)
    with pytest.raises(ValueError):
        sz.PagedCache(sz.E5M2, byte, scales[:3])
    with pytest.raises(ValueError):
        sz.PagedCache(sz.E5M2, byte, scales, status=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        sz.paged_cache(4, P, H, D, 5, device="cpu")
    cache = sz.paged_cache(4, P, H, D, sz.E5M2, device="cpu")
    assert bool((cache.scales == 127).all()) and not bool(cache.data.float().any())
    table, kv, starts = (torch.zeros(2, 2, dtype=torch.int32), torch.tensor([3, 4], dtype=torch.int32),
                         torch.tensor([0, 1, 2], dtype=torch.int32))
    for bad in [(table[0], kv, starts), (table, kv[:1], starts), (table, kv, starts[:2]), (table, kv[None], starts)]:
        with pytest.raises(ValueError):
            sz.PageBatch(*bad, 2)
    for bad in [(table.long(), kv, starts), (table, kv.long(), starts), (table, kv, starts.float()),
                (table.T, kv, starts)]:
        with pytest.raises((TypeError, ValueError)):
            sz.PageBatch(*bad, 2)
    with pytest.raises(ValueError):
        sz.PageBatch(table, kv, starts, -1)
    batch = sz.PageBatch(table, kv, starts, 2)
    x = torch.zeros(2, H, D, dtype=torch.bfloat16)
    for bad in (x.float(), x[:1], x[:, :1], torch.zeros(2, H, 2 * D, dtype=torch.bfloat16)[:, :, ::2]):
        with pytest.raises((TypeError, ValueError)):
            sz.cache_write(cache, batch, bad, x, check=False)
        with pytest.raises((TypeError, ValueError)):
            sz.cache_read(cache, batch, out=(x, bad), check=False)
        with pytest.raises((TypeError, ValueError)):
            sz.paged_attention(bad[:, :, :] if bad.dim() == 3 else bad, cache, batch, check=False, ws=scales)
    with pytest.raises(ValueError):                        # nothing of this runs on the CPU
        sz.cache_write(cache, batch, x, x, check=False)
    with pytest.raises(ValueError):
        sz.paged_attention(torch.zeros(2, 3, D, dtype=torch.bfloat16), cache, batch, check=False)
    with pytest.raises(ValueError):
        sz.paged_attention(x, cache, batch, window=-1, check=False)
    with pytest.raises(ValueError):
        sz.paged_attention(x, cache, batch, out=x.float(), check=False)
    with pytest.raises(ValueError):
        sz.paged_attention(x, cache, batch, lse=torch.zeros(2, H, dtype=torch.float64), check=False)
    with pytest.raises(ValueError):
        sz.attention_workspace(cache, batch, 3)
    with pytest.raises(ValueError):                        # rows that share memory cannot be read into
        sz.cache_read(cache, batch, out=(x[:1].expand(2, H, D), x), check=False)


def test_reference_rounding_by_hand():
    """The oracle's quantisation against values worked out by hand."""
    x = torch.zeros(6, 64, dtype=torch.float64)
    x[0, :4] = torch.tensor([448.0, 1.0, -17.0, 19.0])          # k = 0: 17 ties to 16, 19 to 20
    x[1, :2] = torch.tensor([448.0 * 1.01, 3.0])                # just over the largest: k = 1
    x[2, :3] = torch.tensor([2.0 ** -133, 0.0, -0.0])           # smallest BF16: k is held at -126
    x[3, :3] = torch.tensor([math.inf, 2.0, math.nan])          # the finite values alone give the scale
    x[4, 0] = 3.3895313892515355e38                             # the largest BF16, 255 2^120: k = 120
    q, s = ref.quantise(x, ref.E4M3)
    assert s.tolist() == [127, 128, 1, 127 - 7, 247, 1]
    q = q.float()
    assert q[0, :4].tolist() == [448.0, 1.0, -16.0, 20.0] and q[1, :2].tolist() == [224.0, 1.5]
    assert q[2, 0] == 2.0 ** -7 and q[3, 1] == 256.0 and bool(q[3, :3].isnan()[[0, 2]].all()) and q[4, 0] == 256.0
    q, s = ref.quantise(x[3:4], ref.E5M2)
    assert s.tolist() == [127 - 14] and q.float()[0, 0] == math.inf and q.float()[0, 1] == 32768.0


def test_launches_that_no_grid_holds_are_refused():
    nat = _native()
    wide = cache_of(nat, kv_heads=1024)
    many = batch_of(nat, tokens=1 << 30, max_new=1 << 30)
    assert calls(nat, wide, many, q_heads=1024, token=1 << 17) == [ARG] * 3
    # 2^24 workgroups of 256 threads are one launch too many, in either kernel
    for kw in (dict(max_new=1), dict(max_new=100)):
        b = batch_of(nat, seqs=1 << 24, table_width=16, max_kv=128, tokens=1 << 20, **kw)
        assert calls(nat, cache_of(nat, kv_heads=1), b, q_heads=1)[2] == ARG


def test_scale_is_finite_in_powers_of_two():
    nat = _native()
    c, b = cache_of(nat), batch_of(nat)
    for scale in (3e38, 2.4e38, float("inf"), float("nan"), 0.0, -1.0):
        assert calls(nat, c, b, scale=scale)[2] == ARG, scale
    # the largest that is passes this check and fails the next
    assert calls(nat, c, b, scale=2.3e38, ws_bytes=0)[2] == WORKSPACE


def test_python_layer_refuses_shared_rows_and_gradients():
    import fp8_kv_cache_sz_amd as sz
    H, D, P = 2, 64, 16
    cache = sz.paged_cache(4, P, H, D, device="cpu")
    batch = sz.PageBatch(torch.zeros(2, 2, dtype=torch.int32), torch.tensor([3, 4], dtype=torch.int32),
                         torch.tensor([0, 1, 2], dtype=torch.int32), 2)
    x = torch.zeros(2, H, D, dtype=torch.bfloat16)
    store = torch.zeros(8 * D, dtype=torch.bfloat16)
    view = lambda token, head: store.as_strided((2, H, D), (token, head, 1))
    # the fourth: the second token starts inside the first's last row
    for bad in (view(D, D), view(0, D), view(D, 0), view(2 * D, D + 8), view(D, 2 * D - 8)):
        with pytest.raises(ValueError, match="share memory"):
            sz.cache_read(cache, batch, out=(bad, x), check=False)
    with pytest.raises(ValueError, match="are one"):
        sz.cache_read(cache, batch, out=(x, x), check=False)
    for good in (view(2 * D, D), view(D, 2 * D)):          # these fail only at the device
        with pytest.raises(ValueError, match="run on the GPU"):
            sz.cache_read(cache, batch, out=(good, x), check=False)
    g = x.clone().requires_grad_()
    for call in (lambda: sz.cache_write(cache, batch, g, x, check=False),
                 lambda: sz.cache_write(cache, batch, x, g, check=False),
                 lambda: sz.paged_attention(g, cache, batch, ws=store, check=False)):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="run on the GPU"):
            call()


def test_attention_workspace_covers_every_window_of_many_shapes():
    """As above over random shapes: the null output is the last check, so a
    call that reaches it has passed the workspace's."""
    import random
    nat = _native()
    rng = random.Random(5)
    for _ in range(400):
        heads, group = rng.choice([1, 2, 3, 8, 40]), rng.choice([1, 2, 4, 7, 16, 20, 32, 64])
        seqs, page = rng.choice([1, 2, 5, 16, 64, 300, 1100]), rng.choice([16, 64, 1024])
        max_kv = int(2 ** rng.uniform(0, 18))
        max_new = rng.choice([1, 1, 2, 5, 17, 64, 500, 5000])
        tokens = rng.choice([seqs * max_new, max(1, seqs * max_new // 3), seqs * max_new + 7])
        c = cache_of(nat, dtype=rng.randrange(3), kv_heads=heads, head_dim=rng.choice([64, 128]), page_tokens=page)
        b = batch_of(nat, seqs=seqs, tokens=tokens, max_new=max_new, max_kv=max_kv, table_width=-(-max_kv // page))
        size = nat.sz_paged_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), heads * group)
        for window in [0, 1, 16, 127, 1000, max_kv // 2, max_kv, 2 * max_kv + 5]:
            got = calls(nat, c, b, q_heads=heads * group, window=window, ws_bytes=size, out=None)[2]
            assert got == ARG, (heads, group, seqs, max_kv, max_new, tokens, window)
