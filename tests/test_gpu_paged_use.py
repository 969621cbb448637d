"""The paged cache as programs use it: captured graphs whose lengths change,
workspaces that calls share, other streams, padded batches, caches past 4
GiB, defaults and layouts of the Python layer."""
import math

import pytest
import torch

import tests.pagedref as ref
from tests.test_gpu_paged import BF16, E4M3, E5M2, batch_of, bits, filled, gen, on_gpu, sz

pytestmark = pytest.mark.gpu


def expected(q, cache, batch, window=0):
    """The eager result of a fresh call, and its 64-bit check."""
    out, lse = sz().paged_attention(q, cache, batch, window=window, lse=True)
    return out.clone(), lse.clone()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("shape", ["tokens", "one", "prompts", "mixed"])
def test_graph_replays_with_changing_lengths(dtype, shape):
    """Write and attention captured once; each replay sees other lengths,
    pages and inputs, with eager work between, and equals the eager calls."""
    m = sz()
    H, G, D, P = 2, 4, 128, 16
    new, most = {"tokens": ([1] * 9, 600), "one": ([1], 700), "prompts": ([70, 33], 200),
                 "mixed": ([1, 50, 1, 2], 400)}[shape]
    B, T, W = len(new), sum(new), -(-most // P)
    pages = B * W + 1
    data, scales = filled(dtype, pages, H, P, D, 17)
    cache = on_gpu(dtype, data, scales)
    twin = on_gpu(dtype, data, scales)                         # the eager calls' cache
    table = torch.zeros(B, W, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0] + [sum(new[:i + 1]) for i in range(B)], dtype=torch.int32, device="cuda")
    q = torch.zeros(T, H * G, D, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    batch = m.PageBatch(table, lens, starts, T, max_new=max(new), max_kv=most)
    ws = m.attention_workspace(cache, batch, H * G)
    out, lse = torch.empty_like(q), torch.empty(T, H * G, device="cuda")

    def step():
        m.cache_write(cache, batch, k, v, check=False)
        m.paged_attention(q, cache, batch, out=out, lse=lse, ws=ws, check=False)

    g = gen(3)
    def change(rep):
        table.copy_(torch.randperm(pages, generator=g)[:B * W].to(torch.int32).view(B, W))
        lens.copy_(torch.tensor([min(most, n + (37 * (i + 1) * (rep + 1)) % (most - n + 1)) for i, n in enumerate(new)],
                                dtype=torch.int32))
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g).to(torch.bfloat16))

    change(0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()                                                 # warm up
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    twin.data.view(torch.uint8).copy_(cache.data.view(torch.uint8))
    if scales is not None:
        twin.scales.copy_(cache.scales)
    for rep in range(5):
        print("graph replay", shape, rep, flush=True)
        change(rep)
        torch.cuda.synchronize()
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        m.cache_write(twin, batch, k, v)
        a, b = expected(q, twin, batch)                        # eager, with a workspace of its own
        assert torch.equal(bits(cache.data), bits(twin.data)), rep
        assert torch.equal(out, a) and torch.equal(lse, b), rep
        assert int(cache.status.item()) == 0


def test_graphs_and_calls_of_other_shapes_share_a_workspace():
    """One workspace, sized for the largest, under two captured graphs and
    eager calls of other shapes in between: each finds it as it needs it."""
    m = sz()
    H, G, D, P = 4, 2, 64, 16
    shapes = [([1000], [1]), ([30] * 40, [1] * 40), ([300, 200], [90, 60]), ([2000, 40], [5, 1])]
    made = []
    size = 0
    for i, (lens, new) in enumerate(shapes):
        table, kv, starts, T, pages = ref.layout(lens, new, P, seed=i)
        data, scales = filled(E5M2, pages, H, P, D, i)
        cache = on_gpu(E5M2, data, scales)
        batch = batch_of(table, kv, starts, T, max_new=max(new), max_kv=max(lens))
        q = torch.randn(T, H * G, D, generator=gen(i)).to(torch.bfloat16).cuda()
        made.append((q, cache, batch, m.paged_attention(q, cache, batch)))
        size = max(size, m.attention_workspace(cache, batch, H * G).numel())
    ws = torch.randint(0, 256, (size,), dtype=torch.uint8, device="cuda")
    ws[:4096].zero_()
    stream = torch.cuda.Stream()
    graphs = []
    for q, cache, batch, _ in made[:3]:
        out = torch.empty_like(q)
        with torch.cuda.stream(stream):
            m.paged_attention(q, cache, batch, out=out, ws=ws, check=False)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            m.paged_attention(q, cache, batch, out=out, ws=ws, check=False)
        graphs.append((graph, out))
    for rep in range(4):
        for i in (0, 2, 1, 0):
            graphs[i][1].zero_()
            graphs[i][0].replay()
            torch.cuda.synchronize()
            assert torch.equal(graphs[i][1], made[i][3]), (rep, i)
            q, cache, batch, want = made[3]
            assert torch.equal(m.paged_attention(q, cache, batch, ws=ws), want), (rep, i)
            torch.cuda.synchronize()


def test_other_streams():
    """Calls on a stream that is not the current one, one after another
    without waiting, and two streams at once with their own workspaces."""
    m = sz()
    H, G, D, P = 2, 4, 128, 32
    lens, new = [500, 900], [500, 1]
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=8)
    data, scales = filled(E4M3, pages, H, P, D, 8)
    x = torch.randn(T, H, D, generator=gen(1)).to(torch.bfloat16).cuda()
    q = torch.randn(T, H * G, D, generator=gen(2)).to(torch.bfloat16).cuda()
    batch = batch_of(table, kv, starts, T)
    plain = on_gpu(E4M3, data, scales)
    m.cache_write(plain, batch, x, x)
    want = m.paged_attention(q, plain, batch)
    want_k, want_v = m.cache_read(plain, batch)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    caches = [on_gpu(E4M3, data, scales) for _ in streams]
    torch.cuda.synchronize()
    for rep in range(3):
        got = []
        for s, cache in zip(streams, caches):
            m.cache_write(cache, batch, x, x, stream=s, check=rep == 0)
            got.append((m.paged_attention(q, cache, batch, stream=s, check=False),
                        m.cache_read(cache, batch, stream=s, check=False)))
        for s in streams:
            s.synchronize()
        for out, (k, v) in got:
            assert torch.equal(out, want) and torch.equal(k, want_k) and torch.equal(v, want_v)


def test_padded_batches():
    """A batch padded to a fixed size, as captured steps are: sequences
    without tokens, tokens that belong to none, table rows of no use."""
    m = sz()
    H, G, D, P = 2, 4, 128, 16
    lens, new = [100, 40, 0, 0], [1, 1, 0, 0]
    table, kv, starts, _, pages = ref.layout(lens, new, P, seed=5)
    data, scales = filled(BF16, pages, H, P, D, 6)
    cache = on_gpu(BF16, data, None)
    T = 8
    q = torch.randn(T, H * G, D, generator=gen(2)).to(torch.bfloat16)
    q[2:] = math.nan
    batch = batch_of(table, kv, starts, T, max_new=1, max_kv=128 if table.shape[1] * P >= 128 else 100)
    out = torch.full((T, H * G, D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H * G), 5.0, device="cuda")
    m.paged_attention(q.cuda(), cache, batch, out=out, lse=lse)
    want, want_l, tol, tol_l = ref.attention(q[:2], data, None, table, kv, starts, P, D ** -0.5, 0)
    assert not ref.close(out[:2], want, tol) and not ref.close(lse[:2], want_l, tol_l)
    assert bool((out[2:] == 5.0).all()) and bool((lse[2:] == 5.0).all())
    before = bits(cache.data)
    x = torch.full((T, H, D), 9.0, dtype=torch.bfloat16, device="cuda")
    m.cache_write(cache, batch, x, x)
    after = cache.data.cpu()
    changed = (bits(after) != before).view(pages, 2, H, P, 2 * D).any(-1).any(1).any(1)     # [pages, P]
    places = {(int(table[i, (n - 1) // P]), (n - 1) % P) for i, n in enumerate(lens[:2])}
    assert {tuple(p) for p in changed.nonzero().tolist()} == places
    out[2:] = 1.0
    k = torch.full((T, H, D), 4.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    m.cache_read(cache, batch, out=(k, v))
    assert bool((k[:2] == 9.0).all()) and bool((k[2:] == 4.0).all()) and bool((v[2:] == 4.0).all())
    # no tokens at all, and no sequences at all
    none = m.PageBatch(table[:0].cuda(), kv[:0].cuda(), starts[:1].cuda(), T)
    m.paged_attention(q.cuda(), cache, none, out=out)
    assert bool((out[2:] == 1.0).all())
    empty = batch_of(table, kv, torch.zeros_like(starts), 0)
    assert m.paged_attention(q[:0].cuda(), cache, empty).shape == (0, H * G, D)
    k, v = m.cache_read(cache, empty)
    assert k.shape == (0, H, D)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_pages_past_four_gib(dtype):
    """A cache of over 2^32 bytes (and, FP8, 2^32 values): pages at its end
    are as good as those at its beginning."""
    m = sz()
    H, D, P = 8, 128, 64
    page_bytes = 2 * H * P * D * (2 if dtype == BF16 else 1)
    pages = (1 << 32) // page_bytes + 40
    cache = m.paged_cache(pages, P, H, D, dtype)
    assert cache.data.nbytes > 1 << 32
    n, new = 700, [700]
    order = [pages - 1 - 3 * i for i in range(6)] + [2, 0, 5, 9, 7]
    table = torch.tensor([order], dtype=torch.int32)
    low = torch.tensor([list(range(20, 31))], dtype=torch.int32)
    starts, lens = torch.tensor([0, n], dtype=torch.int32), torch.tensor([n], dtype=torch.int32)
    g = gen(2)
    k, v = (torch.randn(n, H, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(n, H * 2, D, generator=g).to(torch.bfloat16).cuda()
    results = []
    for t in (table, low):
        batch = batch_of(t, lens, starts, n)
        m.cache_write(cache, batch, k, v)
        results.append((m.paged_attention(q, cache, batch), *m.cache_read(cache, batch)))
        last = m.PageBatch(t.cuda(), lens.cuda(), torch.tensor([0, 1], dtype=torch.int32).cuda(), 1)
        results[-1] += (m.paged_attention(q[-1:], cache, last),)
    for a, b in zip(*results):
        assert torch.equal(a, b)
    if dtype == BF16:
        assert torch.equal(results[0][1], k) and torch.equal(results[0][2], v)


def test_layouts_and_defaults():
    """q, k and v as slices of one projection, transposed tensors with
    aligned rows, scale and window defaults, lse and out given or not."""
    m = sz()
    H, G, D, P = 3, 2, 64, 16
    lens, new = [40, 21], [40, 3]
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=2)
    g = gen(4)
    qkv = torch.randn(T, (G + 2) * H, D, generator=g).to(torch.bfloat16).cuda()
    q, k, v = qkv[:, :G * H], qkv[:, G * H:(G + 1) * H], qkv[:, (G + 1) * H:]
    batch = batch_of(table, kv, starts, T)
    caches = [m.paged_cache(pages, P, H, D, m.E5M2) for _ in range(2)]
    m.cache_write(caches[0], batch, k, v)
    turned = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]          # head-major memory
    m.cache_write(caches[1], batch, turned[1], turned[2])
    for i in (1,):
        assert torch.equal(bits(caches[0].data), bits(caches[i].data))
        assert torch.equal(caches[0].scales, caches[i].scales)
    a = m.paged_attention(q, caches[0], batch)
    b, lse = m.paged_attention(turned[0], caches[1], batch, scale=D ** -0.5, window=0, lse=True)
    c = m.paged_attention(q, caches[0], batch, window=1 << 40)
    assert torch.equal(a, b) and torch.equal(a, c) and lse.shape == (T, G * H) and lse.dtype == torch.float32
    raw = m.PagedCache(m.E5M2, caches[0].data.view(torch.uint8), caches[0].scales)        # FP8 as plain bytes
    assert torch.equal(m.paged_attention(q, raw, batch), a)
    # misaligned rows are refused by the library
    odd = torch.zeros(T * G * H * D + 4, dtype=torch.bfloat16, device="cuda")[4:].view(T, G * H, D)
    with pytest.raises(m.SplitZipError):
        m.paged_attention(odd, caches[0], batch)
    # read into head-major memory
    k2 = torch.zeros(H, T, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    v2 = torch.zeros_like(k2)
    m.cache_read(caches[0], batch, out=(k2, v2))
    k1, v1 = m.cache_read(caches[0], batch)
    assert torch.equal(k1, k2) and torch.equal(v1, v2)


def test_instrumentation_names_the_launches():
    m = sz()
    H, D, P = 2, 128, 16
    table, kv, starts, T, pages = ref.layout([3000, 50], [1, 40], P, seed=1)
    cache = m.paged_cache(pages, P, H, D)
    batch = batch_of(table, kv, starts, T)
    x = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    m.profile_enable(True)
    try:
        m.cache_write(cache, batch, x, x)
        m.cache_read(cache, batch)
        m.paged_attention(torch.zeros(T, 8, D, dtype=torch.bfloat16, device="cuda"), cache, batch)
        got = m.profile_collect()
    finally:
        m.profile_enable(False)
    assert {"sz_cache_check_clear", "sz_cache_check_walk", "sz_cache_write", "sz_cache_read", "sz_attn_rows",
            "sz_attn_tiles", "sz_attn_join"} == set(got)


def test_streams_of_another_device_are_refused():
    import types
    cache = sz().paged_cache(2, 16, 1, 64)
    index = torch.zeros(1, dtype=torch.int32, device="cuda")
    batch = sz().PageBatch(index.view(1, 1), index + 1, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1)
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    other = types.SimpleNamespace(device=torch.device("cuda", cache.device.index + 1), cuda_stream=0)
    for call in (lambda: sz().cache_write(cache, batch, x, x, stream=other),
                 lambda: sz().cache_read(cache, batch, stream=other),
                 lambda: sz().paged_attention(x, cache, batch, stream=other)):
        with pytest.raises(ValueError, match="stream is on"):
            call()


@pytest.mark.parametrize("seqs", [62, 63, 64, 126, 127])
def test_tokens_behind_the_last_sequence_belong_to_none(seqs):
    """What lies in memory behind the batch's arrays, a sequence by its looks,
    is not read: the tokens behind the last one are nobody's."""
    m = sz()
    H, D, P = 1, 64, 16
    table = torch.arange(seqs + 1, dtype=torch.int32, device="cuda").view(-1, 1)
    lens = torch.ones(seqs + 1, dtype=torch.int32, device="cuda")
    starts = torch.arange(seqs + 2, dtype=torch.int32, device="cuda")
    T = seqs + 1
    cache = m.paged_cache(seqs + 1, P, H, D)
    batch = m.PageBatch(table[:seqs], lens[:seqs], starts[:seqs + 1], T)
    x = torch.ones(T, H, D, dtype=torch.bfloat16, device="cuda")
    m.cache_write(cache, batch, x, x)
    assert bool((cache.data[:seqs, :, :, 0] == 1).all()) and not bool(cache.data[seqs].any())
    k, v = (torch.full((T, H, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.cache_read(cache, batch, out=(k, v))
    out = torch.full((T, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    m.paged_attention(x, cache, batch, out=out)
    for y in (k, v, out):
        assert bool((y[:seqs] == 1).all()) and bool((y[seqs] == 3).all())


@pytest.mark.parametrize("lens,new,H,G,D", [([2000, 900, 5, 1500], 1, 8, 4, 128), ([216] * 20 + [90] * 27, 1, 8, 4, 128),
                                            ([3000, 700], 3, 2, 8, 64), ([1500, 1100], 40, 1, 4, 128)])
def test_partials_are_this_calls(lens, new, H, G, D):
    """The workspace holds NaN before each call: a chunk that was joined before
    it was written would show.  Results repeat bit for bit."""
    m = sz()
    table, kv, starts, T, pages = ref.layout(lens, [new] * len(lens), 16, seed=2)
    data, scales = filled(E4M3, pages, H, 16, D, 5)
    cache = on_gpu(E4M3, data, scales)
    batch = batch_of(table, kv, starts, T, max_new=new, max_kv=max(lens))
    q = torch.randn(T, H * G, D, generator=gen(6)).to(torch.bfloat16).cuda()
    ws = m.attention_workspace(cache, batch, H * G)
    first = None
    for _ in range(30):
        ws[4096:].fill_(255)
        out = m.paged_attention(q, cache, batch, ws=ws, check=False)
        first = out if first is None else first
        assert torch.equal(out, first) and not bool(ws[:4096].any())
    assert bool(torch.isfinite(first).all())
