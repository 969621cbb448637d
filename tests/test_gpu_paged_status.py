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
