"""The calls of a serving step around the paged cache against the plain
reference (stepref.py): pages and slots, trees' masks and positions, rotary
writes, trees' attention, kept rows."""
import math

import pytest
import torch

import tests.pagedref as ref
import tests.stepref as step
from tests.test_gpu_paged import BF16, DTYPES, E4M3, E5M2, batch_of, bits, filled, gen, on_gpu, sz

pytestmark = pytest.mark.gpu

CAPACITY, FORMAT = -3, -5


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


# ---- pages -------------------------------------------------------------------

def a_pool(seqs, P, seed, most, spare, grow=0.5):
    """Sequences that hold pages and now need others, and a ring that wraps."""
    g = gen(seed)
    draw = lambda hi, n: torch.randint(0, hi + 1, (n,), generator=g).tolist()
    held = draw(most, seqs)
    need = [int(x) if float(torch.rand(1, generator=g)) < grow else h for x, h in zip(draw(most, seqs), held)]
    lens = [max(0, n * P - d) if n else 0 for n, d in zip(need, draw(P - 1, seqs))]
    take = sum(max(0, -(-n // P) - h) for n, h in zip(lens, held))
    count = max(0, take + spare)
    pages = sum(held) + count + 3
    order = torch.randperm(pages, generator=g).tolist()
    head = int(torch.randint(0, pages, (1,), generator=g))
    queue = [-9] * pages
    for k in range(count):
        queue[(head + k) % pages] = order[k]
    table, at = [], count
    for h in held:
        table.append(order[at:at + h] + [-5] * (most + 1 - h))
        at += h
    new = [min(n, int(x)) for n, x in zip(lens, draw(2 * P, seqs))]
    return ints(queue), ints([head, count]), ints(table).view(seqs, most + 1), ints(lens), ints(held), new


ASSIGN = [(1, 16, 3, 5), (5, 16, 4, 0), (64, 32, 6, 2), (63, 16, 2, -3), (100, 64, 3, -200), (1000, 16, 2, 1),
          (1024, 16, 3, -50), (1025, 16, 2, 4), (2500, 32, 4, -1000), (3, 16, 400, 7), (40, 16, 300, -2000)]


@pytest.mark.parametrize("seqs,P,most,spare", ASSIGN)
@pytest.mark.parametrize("place", ["in place", "beside"])
def test_pages_assign(seqs, P, most, spare, place):
    print("assign", seqs, P, most, spare, place, flush=True)
    m = sz()
    queue, ends, table, lens, held, new = a_pool(seqs, P, seqs + most, most, spare)
    gap = 3
    starts = [gap]
    for n in new:
        starts.append(starts[-1] + n)
    T = starts[-1] + gap
    max_kv = (most + 1) * P
    pool = m.PagePool(P, queue.cuda(), ends.cuda())
    batch = batch_of(table, lens, ints(starts), T, max_new=max(new + [1]), max_kv=max_kv)
    h, e = held.cuda(), pool.ends
    slots = torch.full((T,), 77, dtype=torch.int64, device="cuda")
    want_q, want_e, want_t, want_h, short, wrong = step.assign(P, queue, ends, table, lens, held, most + 1, max_kv)
    assert not wrong and short == (spare < 0)
    kw = {}
    if place == "beside":
        kw = dict(held_out=torch.full_like(h, -1), ends_out=torch.full_like(e, -1))
    repeat = 2 if place == "beside" else 1                   # the same call again: the same result
    for _ in range(repeat):
        m.pages_assign(pool, batch, h, slots=slots, check=False, **kw)
        assert batch.page_table.tolist() == want_t
        assert pool.queue.tolist() == want_q
        assert (kw["held_out"] if kw else h).tolist() == want_h
        assert (kw["ends_out"] if kw else pool.ends).tolist() == want_e
        assert slots.tolist() == step.slots(P, len(queue), want_t, lens.tolist(), starts, T)
    if kw:
        assert torch.equal(h.cpu(), held) and torch.equal(pool.ends.cpu(), ends)
    assert int(pool.status.item()) == (CAPACITY if short else 0)
    if short:
        with pytest.raises(m.SplitZipError):
            pool.raise_status()
    pool.raise_status()


def test_many_slots_in_place():
    """More tokens than one launch gives slots to where the state is updated
    in place, and than a lane takes one of."""
    m = sz()
    P = 16
    for lens in ([90000, 1, 0, 60000, 7], [300000]):
        held = [0] * len(lens)
        width = -(-max(lens) // P)
        pages = sum(-(-n // P) for n in lens) + 9
        queue, ends = torch.randperm(pages, generator=gen(2)).to(torch.int32), ints([pages - 5, pages])
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + n)
        want = step.assign(P, queue, ends, table, ints(lens), ints(held), width, width * P)
        slots = step.slots(P, pages, want[2], lens, starts, starts[-1])
        for beside in (False, True):
            pool = m.PagePool(P, queue.cuda(), ends.cuda())
            batch = batch_of(table, ints(lens), ints(starts), starts[-1])
            h = ints(held).cuda()
            kw = dict(held_out=h.clone(), ends_out=pool.ends.clone()) if beside else {}
            got = m.pages_assign(pool, batch, h, slots=True, **kw)
            assert got.tolist() == slots
            assert batch.page_table.tolist() == want[2] and pool.queue.tolist() == want[0]
            assert (kw.get("held_out", h)).tolist() == want[3] and kw.get("ends_out", pool.ends).tolist() == want[1]


def test_pages_go_round():
    """Sequences that grow and end over a pool that is used many times over: no
    page is ever held twice, none is lost."""
    m = sz()
    P, seqs, most, pages = 16, 37, 9, 120
    g = gen(1)
    pool = m.page_pool(pages, P)
    table = torch.full((seqs, most), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    held = torch.zeros_like(lens)
    batch = m.PageBatch(table, lens, torch.zeros(seqs + 1, dtype=torch.int32, device="cuda"), 0)
    now = [0] * seqs
    for rep in range(60):
        for i in range(seqs):
            x = float(torch.rand(1, generator=g))
            now[i] = 0 if x < 0.1 else min(most * P, now[i] + int(40 * x))
        while sum(-(-n // P) for n in now) > pages:
            now[now.index(max(now))] = 0
        lens.copy_(ints(now))
        before = held.tolist()
        m.pages_assign(pool, batch, held, check=False)
        free = int(pool.ends[1])
        # what was given in this call is not handed out in it: a call may come up short once
        if int(pool.status.item()) == CAPACITY:
            pool.status.zero_()
            m.pages_assign(pool, batch, held)
            free = int(pool.ends[1])
        rows = [table[i, :h].tolist() for i, h in enumerate(held.tolist())]
        used = [p for r in rows for p in r]
        head = int(pool.ends[0])
        ring = pool.queue.tolist()
        free_pages = [ring[(head + k) % pages] for k in range(free)]
        assert sorted(used + free_pages) == list(range(pages)), (rep, before)
        assert held.tolist() == [-(-n // P) for n in now]


@pytest.mark.parametrize("seqs", [6, 1300])
def test_bad_lengths_and_pools_are_reported(seqs):
    m = sz()
    P, W = 16, 4
    table = torch.arange(seqs * W, dtype=torch.int32).view(seqs, W)
    pages = seqs * W + 40
    queue = torch.full((pages,), -3, dtype=torch.int32)
    queue[:40] = torch.arange(seqs * W, pages)
    lens, held = [20] * seqs, [1] * seqs
    lens[1], lens[2], held[3], held[4] = -1, W * P + 1, -2, W + 1
    lens[6:] = [16] * (seqs - 6)
    ends = [0, 40]
    want = step.assign(P, queue, ints(ends), table, ints(lens), ints(held), W, W * P)
    pool = m.PagePool(P, queue.cuda(), ints(ends).cuda())
    batch = batch_of(table, ints(lens), ints([0] * (seqs + 1)), 0, max_kv=W * P)
    h = ints(held).cuda()
    m.pages_assign(pool, batch, h, check=False)
    assert pool.queue.tolist() == want[0] and pool.ends.tolist() == want[1]
    assert batch.page_table.tolist() == want[2] and h.tolist() == want[3]
    assert int(pool.status.item()) == FORMAT
    pool.status.zero_()
    for bad in ([-1, 5], [pages, 5], [0, pages + 1], [0, -1]):
        pool = m.PagePool(P, queue.cuda(), ints(bad).cuda())
        batch = batch_of(table, ints([20] * seqs), ints([0] * (seqs + 1)), 0, max_kv=W * P)
        h = ints([1] * seqs).cuda()
        m.pages_assign(pool, batch, h, check=False)
        assert int(pool.status.item()) in (FORMAT, CAPACITY)
        assert h.tolist() == [1] * seqs and pool.ends.tolist() == [0, 0]
        assert bool((batch.page_table[:, 1] == -1).all())
    # pages that two sequences hold come back twice: more free pages than there are
    pool = m.PagePool(P, torch.zeros(3, dtype=torch.int32, device="cuda"), ints([1, 2]).cuda())
    batch = batch_of(torch.zeros(2, W, dtype=torch.int32), ints([0, 0]), ints([0, 0, 0]), 0, max_kv=W * P)
    h = ints([1, 3]).cuda()
    m.pages_assign(pool, batch, h, check=False)
    assert int(pool.status.item()) == FORMAT and pool.ends.tolist() == [1, 3] and h.tolist() == [0, 0]


# ---- trees -------------------------------------------------------------------

def forest(kind, n, g):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1 if i == 0 else 0 for i in range(n)]
    if kind == "roots":
        return [-1] * n
    if kind == "far":                                        # every token continues one of the first
        return [-1 if i < 2 else i % 2 for i in range(n)]
    return [int(torch.randint(-1, i, (1,), generator=g)) if i else -1 for i in range(n)]


SIZES = [[1], [2, 0, 64, 63], [65, 3], [128, 127, 1], [129, 256, 255], [257, 0, 512], [513, 1000], [1024, 1023, 5, 64]]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("kind", ["chain", "star", "roots", "far", "random"])
def test_draft_tree(sizes, kind):
    print("tree", sizes, kind, flush=True)
    m = sz()
    g = gen(len(kind) + sizes[0])
    starts, parents = [2], [5, 5]                            # tokens of no sequence, whose parents are none
    for n in sizes:
        parents += forest(kind, n, g)
        starts.append(starts[-1] + n)
    T = starts[-1] + 3
    parents += [9, -7, 9]
    lens = [n + 7 * i for i, n in enumerate(sizes)]
    lens[0] = max(0, sizes[0] - 3)                           # more new tokens than the cache has
    batch = batch_of(torch.zeros(len(sizes), 1, dtype=torch.int32), ints(lens), ints(starts), T, max_new=max(sizes),
                     max_kv=5000)
    words = -(-max(sizes) // 64)
    for extra in (0, 1):
        if words + extra > 16:
            continue
        masks = torch.full((T, words + extra), 77, dtype=torch.int64, device="cuda")
        positions = torch.full((T,), 78, dtype=torch.int32, device="cuda")
        m.draft_tree(batch, ints(parents).cuda(), out=(masks, positions))
        want, wrong = step.tree(parents, lens, starts, words + extra)
        assert not wrong
        rows, pos = masks.tolist(), positions.tolist()
        for t in range(T):
            assert rows[t] == (want[t][0] if t in want else [77] * (words + extra)), t
            assert pos[t] == (want[t][1] if t in want else 78), t
    a, b = m.draft_tree(batch, ints(parents).cuda(), check=False)
    assert torch.equal(a[2:T - 3], masks[2:T - 3, :words]) and torch.equal(b[2:T - 3], positions[2:T - 3])


def test_bad_parents_and_batches_are_reported():
    m = sz()
    parents = [-1, 0, 2, -2, 100, 4]                         # 2, 3 and 4 continue what is none
    starts, lens = [0, 6], [40]
    table = torch.zeros(1, 1, dtype=torch.int32)
    batch = batch_of(table, ints(lens), ints(starts), 6, max_new=6, max_kv=64)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    masks, positions = m.draft_tree(batch, ints(parents).cuda(), status=word, check=False)
    want, wrong = step.tree(parents, lens, starts, 1)
    assert wrong and int(word.item()) == FORMAT
    assert masks.tolist() == [want[t][0] for t in range(6)] and positions.tolist() == [want[t][1] for t in range(6)]
    with pytest.raises(m.SplitZipError):
        m.draft_tree(batch, ints(parents).cuda())
    m.draft_tree(batch, ints(parents).cuda(), check=False)   # nobody to report to
    for lens, starts in (([65], [0, 6]), ([-1], [0, 6]), ([40], [0, 7]), ([40], [3, 2])):
        batch = batch_of(table, ints(lens), ints(starts), 6, max_new=6, max_kv=64)
        out = (torch.full((6, 1), 7, dtype=torch.int64, device="cuda"), torch.full((6,), 7, dtype=torch.int32, device="cuda"))
        with pytest.raises(m.SplitZipError):
            m.draft_tree(batch, ints([-1] * 6).cuda(), out=out)
        assert set(out[0].flatten().tolist() + out[1].tolist()) == {7}


# ---- rotary ------------------------------------------------------------------

ROTARY = [  # D, R, interleaved, H, G, page
    (128, 128, False, 8, 4, 16), (128, 128, True, 2, 1, 64), (128, 64, False, 3, 7, 16), (128, 32, True, 1, 8, 32),
    (64, 64, False, 5, 2, 16), (64, 64, True, 9, 1, 16), (64, 16, False, 2, 5, 32), (128, 8, False, 2, 2, 16),
    (64, 8, True, 1, 1, 16), (128, 120, False, 1, 17, 16), (64, 56, True, 11, 1, 16), (128, 16, True, 8, 9, 128)]


def rotary_case(D, R, interleaved, amplitude=1.0, **kw):
    f = sz().rotary_frequencies(R, **kw)
    return f, sz().Rotary(f, interleaved=interleaved, amplitude=amplitude)


def expected_rows(x, dtype):
    """BF16 or FP8 rows (and scales) of 64-bit values that were rounded to 32."""
    return (x, None) if dtype == BF16 else ref.quantise(x.float().double(), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", ROTARY, ids=str)
@pytest.mark.parametrize("shape", ["one", "mixed", "drafts"])
def test_rotary_write(dtype, case, shape):
    D, R, interleaved, H, G, P = case
    print("rotary", ref.NAMES[dtype], case, shape, flush=True)
    m = sz()
    lens, new = {"one": ([1], [1]), "mixed": ([5, 0, 300, 64, 33], [5, 0, 1, 64, 20]),
                 "drafts": ([41, 23, 100], [7, 23, 13])}[shape]
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=3, gap=2)
    data, scales = filled(dtype, pages, H, P, D, 11)
    cache, batch = on_gpu(dtype, data, scales), batch_of(table, kv, starts, T)
    amplitude = 1.25 if shape == "drafts" else 1.0
    f, rotary = rotary_case(D, R, interleaved, amplitude, stretch=8.0, original=100)
    g = gen(R + H)
    x = torch.randn(T, H * G + 2 * H, D, generator=g) * torch.exp2(torch.randint(-20, 20, (T, H * G + 2 * H, 1), generator=g).float())
    x[0::7, H * G] = 0.0
    x = x.to(torch.bfloat16)
    positions = None
    at = [0] * T
    for i, n in enumerate(lens):
        for t in range(int(starts[i]), int(starts[i + 1])):
            at[t] = n - int(starts[i + 1]) + t
    if shape == "drafts":                                    # anywhere: near, far, behind zero
        at = [int(v) for v in torch.randint(-1000, 2 ** 31 - 1, (T,), generator=g)]
        at[3:6] = [2 ** 31 - 1, -2 ** 31, 0]
        positions = ints(at).cuda()
    wide = x.cuda()
    out = torch.full((T, H * G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got = m.rotary_write(cache, batch, rotary, wide[:, :H * G], wide[:, H * G:H * G + H], wide[:, H * G + H:],
                         positions=positions, out=out)
    assert got is out
    cos, sin = step.angles(at, f.tolist())
    want_q, size_q = step.turned(x[:, :H * G], cos, sin, interleaved, amplitude)
    want_k, size_k = step.turned(x[:, H * G:H * G + H], cos, sin, interleaved, amplitude)
    tol_q = step.turned_bound(want_q, size_q)
    rows_k, scales_k = expected_rows(want_k, dtype)
    rows_v, scales_v = expected_rows(x[:, H * G + H:].double(), dtype)
    want, want_s = data.clone(), None if scales is None else scales.clone()
    tol = torch.zeros(data.shape, dtype=torch.float64)
    raw = (lambda t: t) if dtype == BF16 else (lambda t: t.view(torch.uint8))
    mine = torch.zeros(T, dtype=torch.bool)
    for i, n in enumerate(lens):
        for t in range(int(starts[i]), int(starts[i + 1])):
            p = n - int(starts[i + 1]) + t
            mine[t] = True
            pg, row = int(table[i, p // P]), p % P
            raw(want)[pg, 1, :, row] = raw(rows_v[t]) if dtype != BF16 else x[t, H * G + H:]
            if dtype == BF16:
                want[pg, 0, :, row] = rows_k[t].to(torch.bfloat16)
                tol[pg, 0, :, row] = step.turned_bound(want_k[t], size_k[t]) + 2.0 ** -8 * want_k[t].abs()
            else:
                raw(want)[pg, 0, :, row] = raw(rows_k[t])
                want_s[pg, 0, :, row], want_s[pg, 1, :, row] = scales_k[t], scales_v[t]
    assert ref.close(out[mine], want_q[mine], tol_q[mine]) == ""
    assert bool((out[~mine.cuda()] == 7.0).all())
    if dtype == BF16:
        assert ref.close(cache.data, want.double(), tol) == ""
    else:
        assert torch.equal(bits(cache.data), bits(want)) and torch.equal(cache.scales.cpu(), want_s)
    # in place, and without queries
    other = on_gpu(dtype, data, scales)
    again = wide.clone()
    q = again[:, :H * G]
    assert m.rotary_write(other, batch, rotary, q, again[:, H * G:H * G + H], again[:, H * G + H:], positions=positions, out=q) is q
    assert torch.equal(q[mine.cuda()], out[mine.cuda()]) and torch.equal(bits(q[~mine.cuda()]), bits(wide[~mine.cuda(), :H * G]))
    assert torch.equal(again[:, H * G:], wide[:, H * G:]) and torch.equal(bits(other.data), bits(cache.data))
    third = on_gpu(dtype, data, scales)
    assert m.rotary_write(third, batch, rotary, None, wide[:, H * G:H * G + H], wide[:, H * G + H:], positions=positions) is None
    assert torch.equal(bits(third.data), bits(cache.data))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R", [32, 128])
def test_rotary_at_position_zero_is_a_write(dtype, R):
    """No angle: the bytes of cache_write, over BF16's whole range, and NaN and
    infinities among the values that are not turned, and among V."""
    m = sz()
    H, D, P = 4, 128, 16
    lens, new = [70, 9], [70, 2]
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=3)
    data, scales = filled(dtype, pages, H, P, D, 11)
    one, two = on_gpu(dtype, data, scales), on_gpu(dtype, data, scales)
    batch = batch_of(table, kv, starts, T)
    g = gen(9)
    x = torch.randn(T, 2, H, D, generator=g) * torch.exp2(torch.randint(-120, 120, (T, 2, H, 1), generator=g).float())
    x[1::5, 1, 0, 3] = -0.0
    x[2::5, 1, H - 1, 1], x[3::5, 1, H - 1, 2], x[3::5, 1, H - 1, 3] = math.nan, math.inf, -math.inf
    if R < D:
        x[2::5, 0, 0, R], x[3::5, 0, 1, R + 5], x[4::5, 0, 1, D - 1] = math.nan, math.inf, -math.inf
    x = x.to(torch.bfloat16).cuda()
    rotary = rotary_case(D, R, False)[1]
    m.cache_write(one, batch, x[:, 0], x[:, 1])
    m.rotary_write(two, batch, rotary, None, x[:, 0], x[:, 1], positions=torch.zeros(T, dtype=torch.int32, device="cuda"))
    a, b = one.data.cpu().float(), two.data.cpu().float()
    same = (bits(one.data) == bits(two.data))
    if dtype != BF16:
        same |= torch.isnan(a) & torch.isnan(b)
        assert torch.equal(one.scales, two.scales) and bool(same.all())
    else:
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
        assert torch.equal(bits(one.data[:, 1]), bits(two.data[:, 1]))       # V as it is


def test_rotary_frequencies():
    m = sz()
    f = m.rotary_frequencies(128, base=500000.0)
    for i in (0, 1, 33, 63):
        assert abs(float(f[i]) - 500000.0 ** (-i / 64)) < 1e-15
    assert torch.equal(m.rotary_frequencies(128, base=500000.0, stretch=4.0), f / 4)
    s = m.rotary_frequencies(128, base=500000.0, stretch=8.0, original=8192, low=1.0, high=4.0)
    for i in range(64):
        turns = 8192 * float(f[i]) / (2 * math.pi)
        want = float(f[i]) if turns >= 4 else float(f[i]) / 8 if turns <= 1 else \
            float(f[i]) * ((turns - 1) / 3 + (1 - (turns - 1) / 3) / 8)
        assert abs(float(s[i]) - want) < 1e-12 * want


# ---- trees' attention ----------------------------------------------------------

def random_masks(lens, new, T, starts, words, g, kind):
    masks = torch.zeros(T, words, dtype=torch.int64)
    for i, n in enumerate(new):
        s0 = int(starts[i])
        if kind == "tree":
            rows, _ = step.tree([0] * s0 + forest("random", n, g), [0] * i + [lens[i]], [s0] * (i + 1) + [s0 + n], words)
            for t in range(s0, s0 + n):
                masks[t] = torch.tensor(rows[t][0], dtype=torch.int64)
        else:                                                # any bits at all, also those of no token
            masks[s0:s0 + n] = torch.randint(-2 ** 63, 2 ** 63 - 1, (n, words), generator=g)
            masks[s0:s0 + n:3] = 0                           # a row that names nobody
    return masks


ATTEND = [  # dtype, H, G, D, page, lens, new, window
    (BF16, 2, 4, 128, 16, [1], [1], 0), (E4M3, 1, 1, 64, 16, [3], [3], 0), (BF16, 2, 4, 128, 16, [37, 500], [4, 3], 0),
    (E5M2, 2, 4, 128, 32, [37, 500, 8], [8, 5, 8], 0), (E4M3, 3, 2, 64, 16, [700, 90], [16, 11], 0),
    (BF16, 1, 8, 64, 16, [150, 30], [4, 4], 20), (E5M2, 1, 1, 128, 16, [40, 33], [32, 30], 0),
    (BF16, 2, 4, 128, 16, [500, 30, 0, 7], [13, 26, 0, 7], 0), (E4M3, 2, 4, 128, 64, [300, 129], [70, 65], 0),
    (E5M2, 1, 7, 64, 16, [190, 64], [64, 63], 0), (BF16, 1, 5, 64, 32, [400, 130], [130, 129], 33),
    (E4M3, 2, 8, 128, 16, [65, 200], [60, 61], 5), (BF16, 1, 2, 128, 16, [10, 100], [30, 70], 0),
    (E5M2, 1, 4, 128, 16, [2, 6], [8, 8], 0), (BF16, 4, 1, 64, 16, [1200, 900, 5], [3, 1, 5], 0),
    (E4M3, 1, 4, 128, 16, [2500], [40], 0), (BF16, 2, 2, 128, 128, [300], [200], 17),
]


def widened(table, page, keys):
    """The table with columns for so many keys: the launch is shaped for them."""
    more = -(-keys // page) - table.shape[1]
    return torch.cat([table, torch.full((len(table), max(0, more)), -7, dtype=torch.int32)], 1)


def check_tree(case, kind, tight, extra=0, keys=0):
    dtype, H, G, D, P, lens, new, window = case
    print("attend", ref.NAMES[dtype], case[1:], kind, tight, flush=True)
    m = sz()
    g = gen(sum(new) + D)
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=4, gap=1)
    data, scales = filled(dtype, pages, H, P, D, 21)
    words = max(1, -(-(max(new) if tight else T) // 64)) + extra
    masks = random_masks(lens, new, T, starts, words, g, kind)
    q = torch.randn(T, H * G, D, generator=g).to(torch.bfloat16)
    bounds = dict(max_new=max(new), max_kv=max(max(lens), keys)) if tight else {}
    cache, batch = on_gpu(dtype, data, scales), batch_of(widened(table, P, keys), kv, starts, T, **bounds)
    out = torch.full((T, H * G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H * G), 7.0, device="cuda")
    scale = 0.7 / math.sqrt(D)
    m.tree_attention(q.cuda(), cache, batch, masks.cuda(), scale=scale, window=window, out=out, lse=lse)
    want, want_l, tol, tol_l = step.tree_attention(q, data, scales, table, kv, starts, P, scale, window, masks)
    mine = ~torch.isnan(tol_l[:, 0])
    assert ref.close(out[mine], want[mine], tol[mine]) == ""
    assert ref.close(lse[mine], want_l[mine], tol_l[mine]) == ""
    rest = ~mine.cuda()
    assert bool((out[rest] == 7.0).all()) and bool((lse[rest] == 7.0).all())


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "%s-%s" % (ref.NAMES[c[0]], "-".join(map(str, c[1:]))))
@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("keys", [0, 2500], ids=["small", "large"])
def test_tree_attention(case, kind, keys):
    """Small batches take their rows in blocks of 16, large ones (by the host's
    bounds) in tiles of 128."""
    check_tree(case, kind, True, keys=keys)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (E4M3, 128), (E5M2, 64)])
@pytest.mark.parametrize("seqs", [3, 40, 64, 70, 200])
def test_tree_attention_of_many_sequences(dtype, D, seqs):
    """More workgroups than the card holds at once, whose order follows the
    sequences' lengths, equal and empty ones among them."""
    H, G, P = 8, 4, 16
    lens = [(37 * i) % 50 + 1 for i in range(seqs)]
    lens[1] = lens[2] = 50
    new = [min(33, n) for n in lens]
    lens[0], new[0] = 0, 0
    m = sz()
    g = gen(seqs)
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=4)
    data, scales = filled(dtype, pages, H, P, D, 21)
    masks = random_masks(lens, new, T, starts, 1, g, "tree")
    q = torch.randn(T, H * G, D, generator=g).to(torch.bfloat16)
    # every sequence may have 33 tokens: the axis is padded behind the last
    batch = batch_of(widened(table, P, 2500), kv, starts, max(T, 33 * seqs), max_new=33, max_kv=2500)
    pad = lambda t: torch.cat([t, t.new_zeros(max(0, 33 * seqs - T), *t.shape[1:])])
    out, lse = m.tree_attention(pad(q).cuda(), on_gpu(dtype, data, scales), batch, pad(masks).cuda(), lse=True)
    keep = torch.arange(0, T, max(7, T // 250))              # some rows against 64 bits
    want, want_l, tol, tol_l = step.tree_attention(q, data, scales, table, kv, starts, P, D ** -0.5, 0, masks, only=set(keep.tolist()))
    assert ref.close(out[keep], want[keep], tol[keep]) == ""
    assert ref.close(lse[keep], want_l[keep], tol_l[keep]) == ""


@pytest.mark.parametrize("dtype,D,H,new,keys", [(E5M2, 128, 8, 8, 2500), (BF16, 128, 8, 4, 2500), (BF16, 64, 8, 8, 2500),
                                                (E4M3, 64, 8, 2, 2500), (E4M3, 128, 4, 8, 120), (BF16, 64, 8, 9, 60)])
@pytest.mark.parametrize("seqs", [33, 64, 65, 130, 256, 257])
def test_few_rows_of_many_sequences(dtype, D, H, new, keys, seqs):
    """As above for rows that one workgroup takes, and for several blocks of 16."""
    G, P = 4, 16
    lens = [(37 * i) % 57 + 1 for i in range(seqs)]
    lens[1] = lens[2] = 57
    take = [min(new, n) for n in lens]
    lens[0], take[0] = 0, 0
    m = sz()
    g = gen(seqs)
    table, kv, starts, T, pages = ref.layout(lens, take, P, seed=4)
    data, scales = filled(dtype, pages, H, P, D, 21)
    masks = random_masks(lens, take, T, starts, 1, g, "tree")
    q = torch.randn(T, H * G, D, generator=g).to(torch.bfloat16)
    batch = batch_of(widened(table, P, keys), kv, starts, T, max_new=new, max_kv=keys)
    out, lse = m.tree_attention(q.cuda(), on_gpu(dtype, data, scales), batch, masks.cuda(), lse=True)
    keep = torch.arange(0, T, max(3, T // 150))
    want, want_l, tol, tol_l = step.tree_attention(q, data, scales, table, kv, starts, P, D ** -0.5, 0, masks, only=set(keep.tolist()))
    assert ref.close(out[keep], want[keep], tol[keep]) == ""
    assert ref.close(lse[keep], want_l[keep], tol_l[keep]) == ""


@pytest.mark.parametrize("case", ATTEND[2:9:2], ids=lambda c: "%s-%s" % (ref.NAMES[c[0]], "-".join(map(str, c[1:]))))
def test_tree_attention_loose_bounds_and_spare_words(case):
    check_tree(case, "any", False, extra=2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [3, 8, 40, 90])
@pytest.mark.parametrize("keys", [0, 2500], ids=["small", "large"])
def test_chains_are_causal_attention(dtype, new, keys):
    """A tree without branches sees what paged_attention sees."""
    m = sz()
    H, G, D, P = 2, 4, 128, 16
    lens = [new + 300, new, new + 63]
    table, kv, starts, T, pages = ref.layout(lens, [new] * 3, P, seed=4)
    data, scales = filled(dtype, pages, H, P, D, 5)
    cache, batch = on_gpu(dtype, data, scales), batch_of(widened(table, P, keys), kv, starts, T, max_new=new)
    masks, positions = m.draft_tree(batch, ints([i - 1 for i in range(new)] * 3).cuda())
    assert positions.tolist() == [n - new + i for n in lens for i in range(new)]
    q = torch.randn(T, H * G, D, generator=gen(3)).to(torch.bfloat16).cuda()
    for window in (0, 1, 37):
        a, al = m.paged_attention(q, cache, batch, window=window, lse=True)
        b, bl = m.tree_attention(q, cache, batch, masks, window=window, lse=True)
        if window == 1:                                      # the new ones that a mask names are all seen
            continue
        if window and new > window:
            continue
        # either is within its bound of the 64-bit result: twice that between them (2^-7 of the values' size, 2^-20 of lse)
        assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -6 * float(cache_values(cache).abs().max())
        assert float((al - bl).abs().max()) <= 1e-4


def cache_values(cache):
    x = cache.data.float()
    return x if cache.scales is None else x * torch.exp2(cache.scales.float() - 127).unsqueeze(-1)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("case", [(BF16, 2, 4, 128, 4), (E5M2, 2, 4, 64, 8), (E5M2, 2, 4, 128, 70), (BF16, 1, 4, 64, 45)],
                         ids=str)
@pytest.mark.parametrize("keys", [0, 2500], ids=["small", "large"])
def test_tree_attention_hidden_values_stay_hidden(case, value, keys):
    """NaN and infinities in K and V of branches that a token does not see, of
    tokens that nobody sees, before the window and behind the end."""
    dtype, H, G, D, new = case
    m = sz()
    P, window = 16, 90
    lens = [200 + new, 50 + new]
    table, kv, starts, T, pages = ref.layout(lens, [new] * 2, P, seed=4)
    data, scales = filled(dtype, pages, H, P, D, 5)
    g = gen(new)
    masks = torch.zeros(T, -(-new // 64), dtype=torch.int64)
    for i in range(2):
        s0 = int(starts[i])
        for j in range(new):                                 # even tokens see even ones, odd tokens themselves; 1 is bad
            for x in (range(0, j + 1, 2) if j % 2 == 0 else [j]):
                masks[s0 + j, x // 64] |= (1 << x % 64) - (2 ** 64 if x % 64 == 63 else 0)
    q = torch.randn(T, H * G, D, generator=g).to(torch.bfloat16)
    run = lambda d: m.tree_attention(q.cuda(), on_gpu(dtype, d, scales), batch_of(widened(table, P, keys), kv, starts, T, max_new=new),
                                     masks.cuda(), window=window, lse=True)
    clean = run(data)
    bad = data.clone()
    def spoil(i, p):
        pg = int(table[i, p // P])
        rows = bad[pg, :, :, p % P].float()
        rows[..., 1::3] = value
        bad.view(torch.uint8 if dtype != BF16 else torch.bfloat16)[pg, :, :, p % P] = \
            rows.to(bad.dtype).view(torch.uint8 if dtype != BF16 else torch.bfloat16)
    for i in range(2):
        past = lens[i] - new
        spoil(i, past + 1)                                   # an odd token: only it sees it
        if new % 16:
            for p in range(lens[i], -(-lens[i] // P) * P):   # behind the end
                spoil(i, p)
        for p in range(0, max(0, past + 1 - window)):        # no window reaches it
            spoil(i, p)
    got = run(bad)
    seen = torch.zeros(T, dtype=torch.bool)
    for i in range(2):
        seen[int(starts[i]) + 1] = True
    ok = ~seen.cuda()
    assert not bool(torch.isnan(got[0][ok]).any()) and not bool(torch.isnan(got[1][ok]).any())
    # hidden values may change the path a block takes, not what it adds up to: within both results' bounds
    want, want_l, tol, tol_l = step.tree_attention(q, data, scales, table, kv, starts, P, D ** -0.5, window, masks)
    assert ref.close(got[0][ok], want[~seen], tol[~seen]) == ""
    assert ref.close(got[1][ok], want_l[~seen], tol_l[~seen]) == ""
    assert ref.close(clean[0], want, tol) == ""
    assert bool((~torch.isfinite(got[0][~ok])).any())        # the one that sees it does


# ---- kept rows ---------------------------------------------------------------

KEEP = [  # dtype, H, D, page, lens, new, kept
    (BF16, 2, 128, 16, [10, 40, 5], [10, 26, 0], [[0, 2, 3, 4, 9], [1, 5, 25], []]),
    (E5M2, 3, 64, 16, [100, 17], [40, 16], [list(range(1, 40)), [15]]),
    (E4M3, 8, 128, 64, [300, 64, 65], [200, 60, 3], [list(range(0, 200, 2)), list(range(60)), [2]]),
    (BF16, 1, 64, 32, [500], [300], [list(range(130, 300))]),
    (E4M3, 5, 64, 16, [20, 3], [30, 8], [[3, 12, 14, 29], [6, 7]]),          # more new tokens than the cache has
]


@pytest.mark.parametrize("case", KEEP, ids=lambda c: "%s-%s" % (ref.NAMES[c[0]], "-".join(map(str, c[1:6]))))
@pytest.mark.parametrize("layers", [1, 3, 66])
def test_cache_keep(case, layers):
    dtype, H, D, P, lens, new, kept = case
    print("keep", ref.NAMES[dtype], case[1:6], layers, flush=True)
    m = sz()
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=6, gap=1)
    batch = batch_of(table, kv, starts, T, max_new=max(new), max_kv=max(lens))
    width = max(len(k) for k in kept) + 1
    rows = torch.full((len(lens), width), -4, dtype=torch.int32)
    for i, k in enumerate(kept):
        rows[i, :len(k)] = ints(k)
    held = [filled(dtype, pages, H, P, D, 30 + i) for i in range(min(layers, 3))]
    held = [held[i % len(held)] for i in range(layers)]
    caches = [on_gpu(dtype, d, s) for d, s in held]
    m.cache_keep(m.CacheLayers(caches) if layers > 1 else caches[0], batch, rows.cuda(), ints([len(k) for k in kept]).cuda())
    for (data, scales), cache in zip(held, caches):
        raw = data if dtype == BF16 else data.view(torch.uint8)
        want, want_s = raw.clone(), None if scales is None else scales.clone()
        for i, k in enumerate(kept):
            past = lens[i] - new[i]
            for to, frm in enumerate(k):
                src, dst = past + frm, past + to
                if dst < 0:
                    continue
                want[int(table[i, dst // P]), :, :, dst % P] = raw[int(table[i, src // P]), :, :, src % P]
                if scales is not None:
                    want_s[int(table[i, dst // P]), :, :, dst % P] = scales[int(table[i, src // P]), :, :, src % P]
        assert torch.equal(bits(cache.data), bits(want))
        if scales is not None:
            assert torch.equal(cache.scales.cpu(), want_s)
    assert int(caches[0].status.item()) == 0


@pytest.mark.parametrize("kept,count", [([1, 1], 2), ([2, 1], 2), ([-1, 1], 2), ([3, 8], 2), ([0, 1], 3), ([0, 1], -1),
                                        ([0, 1], 9)], ids=str)
def test_bad_kept_tokens_are_reported(kept, count):
    """A sequence whose kept tokens contradict themselves stays as it is, its neighbour is moved."""
    m = sz()
    H, D, P = 2, 64, 16
    lens, new = [30, 30], [8, 8]
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=6)
    data, scales = filled(E4M3, pages, H, P, D, 3)
    cache, batch = on_gpu(E4M3, data, scales), batch_of(table, kv, starts, T, max_new=8, max_kv=30)
    m.cache_keep(cache, batch, ints([kept, [3, 7]]).cuda(), ints([count, 2]).cuda(), check=False)
    assert int(cache.status.item()) == FORMAT
    want = data.view(torch.uint8).clone()
    for to, frm in enumerate([3, 7]):
        src, dst = 22 + frm, 22 + to
        want[int(table[1, dst // P]), :, :, dst % P] = data.view(torch.uint8)[int(table[1, src // P]), :, :, src % P]
    assert torch.equal(bits(cache.data), bits(want))
    # a page that is none of the cache's: its rows stay, and are reported
    cache.status.zero_()
    bad = table.clone()
    bad[0, 1] = pages
    batch = batch_of(bad, kv, starts, T, max_new=8, max_kv=30)
    cache = on_gpu(E4M3, data, scales)
    m.cache_keep(cache, batch, ints([[2, 5], [0, 1]]).cuda(), ints([2, 2]).cuda(), check=False)
    assert int(cache.status.item()) == FORMAT and torch.equal(bits(cache.data), bits(data))
