"""The Python objects of the paged cache on the CPU: what the C structures were
made from does not change under them."""
import pytest
import torch


def objects():
    import fp8_kv_cache_sz_amd as sz
    cache = sz.paged_cache(4, 16, 2, 64, sz.E4M3, device="cpu")
    batch = sz.PageBatch(torch.zeros(2, 3, dtype=torch.int32), torch.tensor([3, 4], dtype=torch.int32),
                         torch.tensor([0, 1, 2], dtype=torch.int32), 2, max_new=1, max_kv=40)
    return cache, batch


def test_fields_of_the_c_structures_are_not_reassigned():
    """A new tensor or bound would be ignored, and the old one's memory freed
    under the kernels that still use it."""
    cache, batch = objects()
    for name in ("data", "scales", "status", "dtype", "pages", "kv_heads", "page_tokens", "head_dim", "device"):
        was = getattr(cache, name)
        with pytest.raises(AttributeError, match="make another PagedCache"):
            setattr(cache, name, was.clone() if isinstance(was, torch.Tensor) else object())
        with pytest.raises(AttributeError):
            delattr(cache, name)
        assert getattr(cache, name) is was
    for name in ("page_table", "kv_lens", "starts", "tokens", "max_new", "max_kv", "seqs", "width", "device"):
        was = getattr(batch, name)
        with pytest.raises(AttributeError, match="make another PageBatch"):
            setattr(batch, name, was.clone() if isinstance(was, torch.Tensor) else object())
        with pytest.raises(AttributeError):
            delattr(batch, name)
        assert getattr(batch, name) is was


def test_other_attributes_and_values_in_place_are_free():
    cache, batch = objects()
    cache.layer = 3
    cache.layer = 4
    batch.note = "x"
    del batch.note
    cache.data.view(torch.uint8).fill_(1)
    batch.kv_lens.add_(1)
    lens = batch.kv_lens
    batch.kv_lens += 2                                          # in place, then the same tensor assigned
    assert batch.kv_lens is lens and lens.tolist() == [6, 7] and cache.layer == 4


def calls(sz, cache, batch, x, out=None, lse=False):
    return [lambda: sz.cache_write(cache, batch, x, x, check=False),
            lambda: sz.cache_read(cache, batch, out=(x, x.clone()), check=False),
            lambda: sz.paged_attention(x, cache, batch, out=out, lse=lse, ws=torch.zeros(8), check=False)]


def test_tensors_that_autograd_follows_are_refused():
    """The calls have no derivative in either direction: what would lose a
    gradient or a tangent is refused, also as an output."""
    import fp8_kv_cache_sz_amd as sz
    from torch.autograd import forward_ad
    cache, batch = objects()
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    lse = torch.zeros(2, 2)
    on_cpu = dict(match="run on the GPU")                       # the last refusal: all others are passed
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        for call in calls(sz, cache, batch, dual):
            with pytest.raises(ValueError, match="has a tangent"):
                call()
        for call in calls(sz, cache, batch, x):                 # others inside the level are plain
            with pytest.raises(ValueError, **on_cpu):
                call()
        with pytest.raises(ValueError, match="out has a tangent"):
            calls(sz, cache, batch, x, out=dual)[2]()
        with pytest.raises(ValueError, match="lse has a tangent"):
            calls(sz, cache, batch, x, lse=forward_ad.make_dual(lse, lse))[2]()
        with pytest.raises(ValueError, match="data has a tangent"):
            sz.PagedCache(sz.BF16, forward_ad.make_dual(torch.zeros(4, 2, 2, 16, 64, dtype=torch.bfloat16),
                                                        torch.zeros(4, 2, 2, 16, 64, dtype=torch.bfloat16)))
    for out, rows in ((x.clone().requires_grad_(), lse), (x.clone(), lse.clone().requires_grad_())):
        call = calls(sz, cache, batch, x, out=out, lse=rows)[2]
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, **on_cpu):
            call()
    leaf = torch.zeros(4, 2, 2, 16, 64, dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(ValueError, match="data requires a gradient"):
        sz.PagedCache(sz.BF16, leaf)
    with torch.no_grad():
        sz.PagedCache(sz.BF16, leaf)


def test_outputs_that_meet_are_refused():
    """cache_read's two outputs: every pair of placements of two small tensors
    in one memory, against their values one by one."""
    from fp8_kv_cache_sz_amd.paged import _rows_meet
    dim = 64
    for tokens, heads in ((1, 1), (1, 3), (3, 1), (3, 2), (4, 3)):
        for token, head in ((heads * dim, dim), (dim, tokens * dim), (2 * heads * dim, dim), (heads * 2 * dim, 2 * dim),
                            (dim, 2 * tokens * dim), (heads * dim + 8, dim)):
            own = {t * token + h * head + d for t in range(tokens) for h in range(heads) for d in range(dim)}
            for apart in range(-1600, 1601, 8):
                other = {x + apart for x in own}
                want = bool(own & other)
                assert _rows_meet((0, token, head), (2 * apart, token, head), tokens, heads, dim) == want, \
                    (tokens, heads, token, head, apart)
    import fp8_kv_cache_sz_amd as sz
    cache, batch = objects()
    store = torch.zeros(2000, dtype=torch.bfloat16)
    view = lambda at, token, head: store.as_strided((2, 2, 64), (token, head, 1), at)
    for a, b in ((view(0, 128, 64), view(64, 128, 64)), (view(0, 128, 64), view(128, 64, 128)),
                 (view(0, 256, 64), view(136, 256, 64))):
        for out in ((a, b), (b, a)):
            with pytest.raises(ValueError, match="share memory"):
                sz.cache_read(cache, batch, out=out, check=False)
    for a, b in ((view(0, 128, 64), view(256, 128, 64)), (view(0, 256, 64), view(128, 256, 64)),
                 (view(0, 256, 128), view(64, 256, 128)), (view(0, 128, 64), view(256, 64, 128))):
        for out in ((a, b), (b, a)):
            with pytest.raises(ValueError, match="run on the GPU"):
                sz.cache_read(cache, batch, out=out, check=False)
