"""What a serving step's calls leave behind where their batch is empty or their
state contradicts itself: free pages, pages held, the status word."""
import ctypes

import pytest
import torch

from tests.test_gpu_paged import batch_of, sz
from tests.test_gpu_step import CAPACITY, FORMAT, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 70, 5000, 140000, 300000])
@pytest.mark.parametrize("in_place", [True, False])
def test_tokens_without_sequences_have_no_slots(tokens, in_place):
    """A batch of no sequences, whose arrays are null: every slot is -1, and the
    ring stays as it is."""
    print("no sequences", tokens, in_place, flush=True)
    m = sz()
    nat = m._native
    queue, ends = ints([4, 0, 3, 1, 2]).cuda(), ints([3, 4]).cuda()
    slots = torch.full((tokens,), 7, dtype=torch.int64, device="cuda")
    after = ends if in_place else ints([9, 9]).cuda()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool = nat.sz_pool(16, 5, queue.data_ptr(), ends.data_ptr())
    batch = nat.sz_batch(None, None, None, 0, 0, tokens, tokens, 0)
    n = nat.lib.sz_pages_assign_workspace_size(ctypes.byref(batch))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        rc = nat.lib.sz_pages_assign(ctypes.byref(pool), ctypes.byref(batch), None, None, after.data_ptr(), slots.data_ptr(),
                                     ws.data_ptr(), n, word.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        assert bool((slots == -1).all()) and after.tolist() == [3, 4] and ends.tolist() == [3, 4]
        assert queue.tolist() == [4, 0, 3, 1, 2] and int(word.item()) == 0
