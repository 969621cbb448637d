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


W, P = 4, 16


def assigned(seqs, free, ends=None, lens=None, held=None, word=0, tokens=0, beside=False):
    """A call for sequences of one page that each want another, with `free`
    pages in the ring; the status word, held and the ring's ends after it."""
    m = sz()
    table = torch.arange(seqs * W, dtype=torch.int32).view(seqs, W)
    pages = seqs * W + 40
    queue = ints(list(range(seqs * W, seqs * W + 40)) + [-3] * (pages - 40))
    pool = m.PagePool(P, queue.cuda(), ints(ends or [0, free]).cuda())
    pool.status.fill_(word)
    lens = ints([P + 1] * seqs) if lens is None else lens
    starts = torch.zeros(seqs + 1, dtype=torch.int32)
    starts[1:] = tokens                                      # all of the first sequence
    batch = batch_of(table, lens, starts, tokens, max_kv=W * P)
    held = (ints([1] * seqs) if held is None else held).cuda()
    kw = dict(held_out=torch.full_like(held, -1), ends_out=torch.full_like(pool.ends, -1)) if beside else {}
    m.pages_assign(pool, batch, held, slots=True if tokens else None, check=False, **kw)
    return int(pool.status.item()), kw.get("held_out", held).tolist(), kw.get("ends_out", pool.ends).tolist()


@pytest.mark.parametrize("beside", [False, True])
@pytest.mark.parametrize("seqs,tokens", [(3, 0), (3, 15), (60, 0), (60, 15), (1300, 0), (1300, 100000), (2500, 0), (2500, 100000)])
def test_a_shortage_hides_nothing_that_is_wrong(seqs, tokens, beside):
    """What contradicts itself is reported also where pages are short, in this
    call or in an earlier one, and a shortage alone is one."""
    run = lambda *a, **kw: assigned(seqs, *a, tokens=tokens, beside=beside, **kw)
    got, held, ends = run(2)
    assert got == CAPACITY and held == [2, 2] + [1] * (seqs - 2) and ends == [2, 0]
    for bad in ([-1, 5], [seqs * W + 40, 5], [0, seqs * W + 41], [0, -1]):
        got, held, ends = run(0, ends=bad)
        assert got == FORMAT and held == [1] * seqs, bad
    lens, heavy = ints([P + 1] * seqs), ints([1] * seqs)
    for where in (0, 1, seqs - 1):
        lens[where] = W * P + 1
        got, held, ends = run(1, lens=lens)
        served = 1 if where == 0 else 0
        assert got == FORMAT and held == [2 if i == served else 1 for i in range(seqs)] and ends == [1, 0]
        lens[where] = P + 1
        heavy[where] = -1
        assert run(1, held=heavy)[0] == FORMAT
        heavy[where] = 1
    assert run(2, word=FORMAT)[0] == FORMAT                  # what an earlier call on the word reported
    assert run(2, word=CAPACITY)[0] == CAPACITY and run(0, word=CAPACITY, ends=[-1, 5])[0] == FORMAT
    if seqs < 40:
        assert run(seqs)[0] == 0 and run(seqs, word=FORMAT)[0] == FORMAT
