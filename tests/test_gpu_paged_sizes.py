"""The paged cache at the ends of its sizes: the largest pages and the most
heads, tens of thousands of sequences, tensors of more than 2^31 values, and
strides that a single token or head leaves open."""
import pytest
import torch

import tests.pagedref as ref
from tests.test_gpu_paged import BF16, E4M3, E5M2, batch_of, bits, filled, gen, on_gpu, run_attention, sz

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    (BF16, [1500, 1024, 1], [1, 1, 1], 2, 4, 128, 1024, 0),
    (E4M3, [2049, 700], [3, 5], 1, 3, 64, 1024, 300),
    (E5M2, [1100, 2048], [40, 60], 2, 2, 128, 512, 0),
    (BF16, [1030, 5], [200, 5], 1, 2, 64, 1024, 77),
], ids=lambda c: "%s-%s-%d" % (ref.NAMES[c[0]], c[1], c[6]))
def test_large_pages(case):
    print("pages", case, flush=True)
    out, lse, want, want_l, tol, tol_l = run_attention(*case)
    assert not ref.close(out, want, tol)
    assert not ref.close(lse, want_l, tol_l)


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (E4M3, 64)])
def test_most_heads(dtype, D):
    """1,024 KV heads: written, read back and attended to."""
    H, P, lens, new = 1024, 16, [20, 3], [20, 1]
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=1)
    data, scales = filled(dtype, pages, H, P, D, 1)
    cache, batch = on_gpu(dtype, data, scales), batch_of(table, kv, starts, T, max_new=20, max_kv=20)
    x = torch.randn(T, 2, H, D, generator=gen(2)).to(torch.bfloat16)
    sz().cache_write(cache, batch, x[:, 0].cuda(), x[:, 1].cuda())
    k, v = sz().cache_read(cache, batch)
    got = torch.stack([k, v], 1).cpu()
    want = x if dtype == BF16 else ref.dequantise(*ref.quantise(x.double(), dtype)).to(torch.bfloat16)
    assert torch.equal(got, want)
    q = torch.randn(T, H, D, generator=gen(3)).to(torch.bfloat16)
    out = sz().paged_attention(q.cuda(), cache, batch)
    heads = [0, 1, 511, 512, 1023]
    data, scales = cache.data.cpu(), None if scales is None else cache.scales.cpu()
    some = data.view(torch.uint8 if dtype else torch.bfloat16)[:, :, heads].view(data.dtype)
    want, _, tol, _ = ref.attention(q[:, heads], some, None if scales is None else scales[:, :, heads], table, kv, starts,
                                    P, D ** -0.5, 0)
    assert not ref.close(out[:, heads], want, tol)


@pytest.mark.parametrize("dtype,G", [(BF16, 2), (E4M3, 32)])
def test_many_sequences_and_tensors_past_two_to_the_31(dtype, G):
    """100 sequences against 70,000 that repeat them: the same bits, and q and
    out of 2.3 billion values where G is 32."""
    H, D, P, n, times = 8, 128, 16, 100, 700
    lens = [1 + (7 * i) % 40 for i in range(n)]
    table, kv, starts, T, pages = ref.layout(lens, [1] * n, P, seed=4)
    data, scales = filled(dtype, pages, H, P, D, 4)
    cache = on_gpu(dtype, data, scales)
    q = torch.randn(n, H * G, D, generator=gen(3)).to(torch.bfloat16).cuda()
    small = batch_of(table, kv, starts, T, max_new=1, max_kv=40)
    a, al = sz().paged_attention(q, cache, small, lse=True)
    many = sz().PageBatch(table.cuda().repeat(times, 1), kv.cuda().repeat(times),
                          torch.arange(n * times + 1, dtype=torch.int32, device="cuda"), n * times, max_new=1, max_kv=40)
    wide = q.repeat(times, 1, 1)
    assert G < 32 or wide.numel() > 1 << 31
    b, bl = sz().paged_attention(wide, cache, many, lse=True)
    assert bool((b.view(times, n, H * G, D) == a).all()) and bool((bl.view(times, n, H * G) == al).all())
    sz().cache_check(cache, sz().PageBatch(many.page_table, many.kv_lens, torch.zeros_like(many.starts), 0))
    with pytest.raises(sz().SplitZipError):                    # 700 sequences write each page
        sz().cache_check(cache, many)


def test_a_long_axis_past_two_to_the_31_values():
    """1,100,000 tokens of 16 heads of 128, written and read back bit for bit."""
    m = sz()
    H, D, P, n = 16, 128, 256, 1100000
    pages = -(-n // P)
    cache = m.paged_cache(pages, P, H, D)
    table = torch.randperm(pages, device="cuda").to(torch.int32).view(1, -1)
    batch = m.PageBatch(table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                        torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
    x = torch.randint(-32000, 32000, (n, H, D), dtype=torch.int16, device="cuda").view(torch.bfloat16)
    assert x.numel() > 1 << 31
    y = x.flip(0)
    m.cache_write(cache, batch, x, y)
    k, v = m.cache_read(cache, batch)
    assert torch.equal(k.view(torch.int16), x.view(torch.int16)) and torch.equal(v.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_strides_that_do_not_count(dtype):
    """One token or one head: the stride of that axis may be anything."""
    m = sz()
    H, D, P = 2, 64, 16
    data, scales = filled(dtype, 3, H, P, D, 1)
    table = torch.tensor([[1, 0]], dtype=torch.int32)
    batch = batch_of(table, torch.tensor([20], dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32), 1)
    x = torch.randn(H, D, generator=gen(2)).to(torch.bfloat16).cuda()
    q = torch.randn(2 * H, D, generator=gen(3)).to(torch.bfloat16).cuda()
    results = []
    for token in (2 * H * D, 1, 12345):
        cache = on_gpu(dtype, data, scales)
        view = lambda t: t.as_strided((1, t.shape[0], D), (token, D, 1))
        m.cache_write(cache, batch, view(x), view(x))
        out = m.paged_attention(view(q), cache, batch)
        results.append((bits(cache.data), out.cpu(), *(t.cpu() for t in m.cache_read(cache, batch))))
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, results[0]))
    one = on_gpu(dtype, data[:, :, :1].contiguous(), None if scales is None else scales[:, :, :1].contiguous())
    batch = batch_of(table, torch.tensor([20], dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32), 3)
    x = torch.randn(3, D, generator=gen(2)).to(torch.bfloat16).cuda()
    results = []
    for head in (D, 3):
        view = x.as_strided((3, 1, D), (D, head, 1))
        m.cache_write(one, batch, view, view)
        results.append((bits(one.data), m.paged_attention(view, one, batch).cpu()))
    assert all(torch.equal(a, b) for a, b in zip(*results))
