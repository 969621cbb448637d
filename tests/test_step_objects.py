"""CPU checks of what the Python layer of a serving step makes its calls from."""
import pytest
import torch

import fp8_kv_cache_sz_amd as sz
from fp8_kv_cache_sz_amd import step


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.mark.parametrize("width", [0, 1, 7])
@pytest.mark.parametrize("max_kv", [None, 0, 500])
def test_trees_are_bounded_by_no_table(width, max_kv, monkeypatch):
    """draft_tree does not look at pages: without a bound of the batch's own,
    lengths are bounded by what a call takes, whatever the table's width."""
    got = []
    monkeypatch.setattr(step, "_launch", lambda name, call, index, device, args, stream, owned=(): got.append(args[0]._obj))
    batch = sz.PageBatch(torch.zeros(2, width, dtype=torch.int32), ints([300, 2]), ints([0, 1, 3]), 3, max_kv=max_kv)
    sz.draft_tree(batch, ints([-1, -1, 0]), check=False)
    assert got[0].max_kv == (1 << 30 if max_kv is None else max_kv) and got[0].table_width == width


def test_amplitudes_end_where_32_bits_end():
    """What Rotary takes the calls take: the largest that rounds to a finite
    32-bit number, and no larger one."""
    f = sz.rotary_frequencies(64)
    top = 2.0 ** 128 - 2.0 ** 104                            # the largest 32-bit number; from half a step on it rounds to infinity
    for good in (top, -top, top + 2.0 ** 102, 0.0, 1e-300):
        assert sz.Rotary(f, amplitude=good, device="cpu").amplitude == good
    for bad in (top + 2.0 ** 103, -top - 2.0 ** 103, 2.0 ** 128 * (1 - 2.0 ** -53)):
        with pytest.raises(ValueError):
            sz.Rotary(f, amplitude=bad, device="cpu")
