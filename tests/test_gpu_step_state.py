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


def assign_within(page, queue, ends, table, lens, held):
    """(queue, ends, table, held, too many) after a call whose free pages
    suffice; pages that come back behind the last of the ring's free places are
    dropped."""
    queue, table, out = queue.tolist(), [r[:] for r in table.tolist()], held.tolist()
    (head, count), pages = ends.tolist(), len(queue)
    old, room = queue[:], pages - count
    taken, back = 0, []
    for i, n in enumerate(lens.tolist()):
        need = -(-n // page)
        for w in range(out[i], need):
            table[i][w] = old[(head + taken) % pages]
            taken += 1
        back += table[i][need:out[i]]
        out[i] = need
    assert taken <= count
    for k, x in enumerate(back[:room]):
        queue[(head + count + k) % pages] = x
    return queue, [(head + taken) % pages, count - taken + min(len(back), room)], table, out, len(back) > room


# pages, free ones, sequences, pages that the first one takes, pages that each other one holds, and how many of them give theirs back
OVERFULL = [(20, 10, 6, 6, 3, 5), (20, 20, 3, 20, 4, 2), (20, 0, 9, 0, 4, 8), (3, 2, 3, 1, 3, 2), (4000, 3000, 200, 900, 20, 150),
            (5000, 4000, 1500, 300, 4, 1400), (6000, 5000, 2600, 400, 3, 2590), (1000, 990, 2600, 300, 3, 2600)]


@pytest.mark.parametrize("case", OVERFULL, ids=str)
@pytest.mark.parametrize("beside", [False, True])
def test_pages_of_two_holders_do_not_reach_the_free_ones(case, beside):
    """Rows that hold what others hold, or what is free, give back more pages
    than the ring has places for, while another sequence takes some: those that
    are taken are the ring's free ones all the same, and it is reported."""
    print("overfull", case, beside, flush=True)
    m = sz()
    pages, free, seqs, take, each, givers = case
    head = pages - 2
    queue = torch.full((pages,), -3, dtype=torch.int32)
    queue[(head + torch.arange(free)) % pages] = torch.arange(free, dtype=torch.int32)
    width = max(take, each) + 1
    table = (torch.arange(seqs * width, dtype=torch.int32) % pages).view(seqs, width)
    held = ints([0] + [each] * (seqs - 1))
    lens = ints([take * P] + [0] * min(givers, seqs - 1) + [each * P] * max(0, seqs - 1 - givers))
    T = take * P
    starts = ints([0] + [T] * seqs)
    want = assign_within(P, queue, ints([head, free]), table, lens, held)
    assert want[4]
    for rep in range(3):
        pool = m.PagePool(P, queue.cuda(), ints([head, free]).cuda())
        batch = batch_of(table, lens, starts, T, max_kv=width * P)
        h = held.cuda()
        kw = dict(held_out=torch.full_like(h, -1), ends_out=torch.full_like(pool.ends, -1)) if beside else {}
        slots = m.pages_assign(pool, batch, h, slots=True, check=False, **kw)
        assert int(pool.status.item()) == FORMAT
        assert pool.queue.tolist() == want[0] and kw.get("ends_out", pool.ends).tolist() == want[1]
        assert batch.page_table.tolist() == want[2] and kw.get("held_out", h).tolist() == want[3]
        assert slots.tolist() == [want[2][0][p // P] * P + p % P for p in range(T)]


def test_a_full_ring_is_not_too_many():
    """Every page is free or held, some are taken and as many given back: nothing is reported."""
    m = sz()
    seqs = 100                                               # half of them hold 2 pages and want 4, the others give 4 back
    order = torch.randperm(400, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    table = torch.full((seqs, 4), -1, dtype=torch.int32)
    table[:50, :2], table[50:] = order[:100].view(50, 2), order[100:300].view(50, 4)
    queue = torch.full((400,), -3, dtype=torch.int32)
    queue[:100] = order[300:]
    lens, held = ints([4 * P] * 50 + [0] * 50), ints([2] * 50 + [4] * 50)
    want = assign_within(P, queue, ints([0, 100]), table, lens, held)
    assert not want[4] and want[1] == [100, 200]
    pool = m.PagePool(P, queue.cuda(), ints([0, 100]).cuda())
    batch = batch_of(table, lens, torch.zeros(seqs + 1, dtype=torch.int32), 0, max_kv=4 * P)
    h = held.cuda()
    m.pages_assign(pool, batch, h)
    assert pool.queue.tolist() == want[0] and pool.ends.tolist() == want[1] and batch.page_table.tolist() == want[2]
    assert h.tolist() == want[3]


@pytest.mark.parametrize("new", [1, 5, 70])
def test_trees_of_a_batch_without_a_table(new):
    """Masks and positions need no page: a table of no columns will do."""
    m = sz()
    starts, lens = ints([0, new, 2 * new]), ints([500, new])
    parents = ints([i - 1 for i in range(new)] * 2).cuda()
    masks, positions = m.draft_tree(batch_of(torch.zeros(2, 0, dtype=torch.int32), lens, starts, 2 * new, max_new=new), parents)
    assert positions.tolist() == list(range(500 - new, 500)) + list(range(new))
    want = [[(1 << min(64, max(0, i + 1 - 64 * w))) - 1 for w in range(-(-new // 64))] for i in range(new)]
    assert [[x % 2 ** 64 for x in row] for row in masks.tolist()] == want * 2
