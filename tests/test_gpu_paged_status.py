"""What the device finds wrong in a batch is reported by each call, and stays
reported until it is read."""
import pytest
import torch

from tests.test_gpu_paged import BF16, E4M3, sz

pytestmark = pytest.mark.gpu

H, D, P = 1, 64, 16


def int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def batch(pages, lens, starts, tokens):
    return sz().PageBatch(int32(pages).view(len(lens), -1), int32(lens), int32(starts), tokens)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("side", [False, True])
def test_a_check_does_not_clear_what_was_reported(dtype, side):
    m = sz()
    cache = m.paged_cache(4, P, H, D, dtype)
    x = torch.ones(2, H, D, dtype=torch.bfloat16, device="cuda")
    good, bad = batch([0, 1], [1, 1], [0, 1, 2], 2), batch([0, 99], [1, 1], [0, 1, 2], 2)
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    m.cache_write(cache, bad, x, x, check=False)
    torch.cuda.synchronize()
    m.cache_write(cache, good, x, x, stream=stream)            # its check is about this batch alone
    m.cache_check(cache, good, stream=stream)
    with pytest.raises(m.SplitZipError):
        m.cache_write(cache, bad, x, x, stream=stream)
    with pytest.raises(m.SplitZipError):
        m.cache_check(cache, bad, stream=stream)
    with pytest.raises(m.SplitZipError):                       # the first write's, still there
        cache.raise_status()
    cache.raise_status()                                       # once
    m.paged_attention(x, cache, good)
    with pytest.raises(m.SplitZipError):                       # a check alone reports into no other call
        m.cache_check(cache, bad)
    m.paged_attention(x, cache, good)


STARTS = {"behind the axis": [9, 12], "all behind it": [200, 300], "past its end": [0, 2, 5], "before it": [-2, 0, 2],
          "all before it": [-9, -3], "descending onto an empty one": [0, 2, 2, 1, 2]}


@pytest.mark.parametrize("name", sorted(STARTS))
@pytest.mark.parametrize("heads", [1, 32], ids=["few", "many"])
def test_starts_outside_the_axis_are_reported(name, heads):
    """Also where no token's own sequence is wrong, and no sequence has a token."""
    m = sz()
    starts = STARTS[name]
    n = len(starts) - 1
    cache = m.paged_cache(8, P, H, D)
    before = cache.data.clone()
    x = torch.ones(2, H, D, dtype=torch.bfloat16, device="cuda")
    b = batch(list(range(n)), [3] * n, starts, 2)
    m.cache_write(cache, b, x, x, check=False)
    with pytest.raises(m.SplitZipError):
        cache.raise_status()
    with pytest.raises(m.SplitZipError):
        m.cache_read(cache, b)
    with pytest.raises(m.SplitZipError):
        m.paged_attention(x.expand(2, heads, D).contiguous(), cache, b)
    after = cache.data.clone()
    with pytest.raises(m.SplitZipError):
        m.cache_write(cache, b, x, x)
    assert torch.equal(cache.data, after)                      # a checked write writes nothing
    if "all" in name or name == "behind the axis":
        assert torch.equal(after, before)


def test_good_starts_are_not_reported():
    """Gaps before the first sequence and behind the last, empty sequences."""
    m = sz()
    cache = m.paged_cache(300, P, H, D)
    x = torch.ones(9, H, D, dtype=torch.bfloat16, device="cuda")
    for starts in ([0, 9], [4, 9], [9, 9], [0, 0], [3, 3, 5, 5, 5, 7], [2] * 100 + [5] * 100 + [6], [9] * 200):
        n = len(starts) - 1
        b = batch(list(range(n)), [9] * n, starts, 9)
        for heads in (1, 32):
            m.cache_write(cache, b, x, x, check=False)
            m.cache_read(cache, b)
            m.paged_attention(x.expand(9, heads, D).contiguous(), cache, b)
            cache.raise_status()
