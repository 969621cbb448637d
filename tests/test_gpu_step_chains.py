"""Trees' attention beside causal attention: chains against the 64-bit reference
of each, with every window, and results that do not depend on when and beside
whom they are computed."""
import math

import pytest
import torch

import tests.pagedref as ref
import tests.stepref as step
from tests.test_gpu_paged import BF16, DTYPES, E4M3, E5M2, batch_of, filled, gen, on_gpu, sz
from tests.test_gpu_step import ints, random_masks, widened

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [3, 8, 40, 90])
@pytest.mark.parametrize("window", [0, 1, 37, 60, 400])
@pytest.mark.parametrize("keys", [0, 2500], ids=["small", "large"])
def test_chains_and_causal_tokens(dtype, new, window, keys):
    """A chain's token i names i + 1 new ones.  Without a window, or with one of
    i + 1 at least, it sees what a causal token sees; with a shorter one all
    that it names and nothing cached, where a causal token sees its last
    `window`.  Either call within its own bound, row by row."""
    print("chains", ref.NAMES[dtype], new, window, keys, flush=True)
    m = sz()
    H, G, D, P = 1, 4, 128, 16
    lens = [new + 300, new, new + 63]
    table, kv, starts, T, pages = ref.layout(lens, [new] * 3, P, seed=4)
    data, scales = filled(dtype, pages, H, P, D, 5)
    cache, batch = on_gpu(dtype, data, scales), batch_of(widened(table, P, keys), kv, starts, T, max_new=new)
    masks, _ = m.draft_tree(batch, ints([i - 1 for i in range(new)] * 3).cuda())
    q = torch.randn(T, H * G, D, generator=gen(3)).to(torch.bfloat16)
    scale = D ** -0.5
    causal = ref.attention(q, data, scales, table, kv, starts, P, scale, window)
    tree = step.tree_attention(q, data, scales, table, kv, starts, P, scale, window, masks.cpu())
    alike = torch.tensor([window == 0 or i < window for i in range(new)] * 3)
    assert torch.equal(causal[0][alike], tree[0][alike]) and torch.equal(causal[1][alike], tree[1][alike])
    assert bool((causal[1][~alike] != tree[1][~alike]).all())
    for call, more, want in ((m.paged_attention, (), causal), (m.tree_attention, (masks,), tree)):
        out, lse = call(q.cuda(), cache, batch, *more, window=window, lse=True)
        assert ref.close(out, want[0], want[2]) == "" and ref.close(lse, want[1], want[3]) == "", call.__name__


# dtype, H, G, D, sequences' lengths, new tokens, window, the table's keys: blocks of rows, one and two products of
# them, in order of lengths, chunks joined in the launch and in one of their own, tiles with and without chunks
SHAPES = [(BF16, 8, 4, 128, [900, 30, 300], 13, 0, 0), (E5M2, 8, 4, 128, [900, 30, 300, 1], 8, 0, 2500),
          (E4M3, 2, 4, 64, [900, 5000, 300], 2, 100, 0), (E4M3, 2, 4, 64, [900, 5000, 300], 2, 0, 0),
          (BF16, 1, 4, 128, [9000, 40, 300], 4, 0, 0), (E5M2, 8, 4, 128, [(37 * i) % 150 + 9 for i in range(70)], 8, 0, 2500),
          (E4M3, 2, 8, 128, [4000, 70, 600], 61, 0, 0), (BF16, 8, 4, 64, [(97 * i) % 300 + 40 for i in range(40)], 33, 50, 2500),
          (E5M2, 1, 2, 128, [700, 300], 200, 0, 0)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%s-%s" % (ref.NAMES[s[0]], "-".join(map(str, s[1:4] + (len(s[4]),) + s[5:]))))
def test_results_do_not_depend_on_neighbours(shape):
    """The same bits again, in another order, and beside sequences that hold
    other keys, NaN among them, and are shorter."""
    dtype, H, G, D, lens, new, window, keys = shape
    print("neighbours", ref.NAMES[dtype], shape[1:4], len(lens), new, window, flush=True)
    m = sz()
    P, seqs = 16, len(lens)
    take = [min(new, n) for n in lens]
    table, kv, starts, T, pages = ref.layout(lens, take, P, seed=4)
    data, scales = filled(dtype, pages, H, P, D, 21)
    g = gen(seqs)
    masks = random_masks(lens, take, T, starts, -(-new // 64), g, "tree")
    q = torch.randn(T, H * G, D, generator=g).to(torch.bfloat16)
    table = widened(table, P, keys)
    ws = None

    def run(order, lengths, data):
        nonlocal ws
        rows = torch.cat([torch.arange(int(starts[i]), int(starts[i + 1])) for i in order])
        begin = ints([0] + torch.tensor([take[i] for i in order]).cumsum(0).tolist())
        batch = batch_of(table[order].contiguous(), ints([lengths[i] for i in order]), begin, T, max_new=new, max_kv=max(max(lens), keys))
        cache = on_gpu(dtype, data, scales)
        ws = m.attention_workspace(cache, batch, H * G) if ws is None else ws
        out, lse = m.tree_attention(q[rows].cuda(), cache, batch, masks[rows].cuda(), window=window, lse=True, ws=ws)
        back = torch.empty(T, dtype=torch.int64)
        back[rows] = torch.arange(T)
        return out.cpu()[back], lse.cpu()[back]

    first = run(list(range(seqs)), lens, data)
    assert bool(torch.isfinite(first[0]).all()) and bool(torch.isfinite(first[1]).all())
    for order in (list(range(seqs)), list(range(seqs))[::-1], torch.randperm(seqs, generator=g).tolist()):
        again = run(order, lens, data)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    # every other sequence's keys are NaN, and it is as short as its new tokens let it be
    other = data.clone()
    raw = other if dtype == BF16 else other.view(torch.uint8)
    for i in range(1, seqs, 2):
        raw[table[i, :-(-lens[i] // P)].long()] = math.nan if dtype == BF16 else 0x7F
    short = [take[i] if i % 2 else n for i, n in enumerate(lens)]
    mine = torch.cat([torch.arange(int(starts[i]), int(starts[i + 1])) for i in range(0, seqs, 2)])
    for order in (list(range(seqs)), list(range(seqs))[::-1]):
        again = run(order, short, other)
        assert torch.equal(first[0][mine], again[0][mine]) and torch.equal(first[1][mine], again[1][mine])
