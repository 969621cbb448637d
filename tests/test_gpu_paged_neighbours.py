"""A sequence's attention among others: under the same host fields its bits do
not depend on what the other sequences are, or on its place in the batch."""
import pytest
import torch

import tests.pagedref as ref
from tests.test_gpu_paged import BF16, E4M3, E5M2, filled, gen, on_gpu, sz

pytestmark = pytest.mark.gpu

CASES = {
    # dtype, the sequence (length, new), others (lengths, new) in turn, H, G, D, window, max_new, max_kv, tokens
    "one token, chunks joined in the launch": (E4M3, (1500, 1), [([40, 1600], [1, 1]), ([2000, 3], [1, 0]), ([5, 5], [0, 1])],
                                               2, 4, 128, 0, 1, 2000, 4),
    "one token, chunks joined after it": (BF16, (3000, 1), [([3000] * 30, [1] * 30), ([7 * i for i in range(30)], [i % 2 for i in range(30)])],
                                          4, 7, 128, 0, 1, 4000, 40),
    "whole contexts": (E5M2, (300, 1), [([300] * 130, [1] * 130), ([1 + i for i in range(130)], [i % 2 for i in range(130)])],
                       8, 2, 64, 0, 1, 400, 131),
    "two blocks of rows": (E5M2, (900, 5), [([700, 20], [5, 5]), ([1, 1000], [1, 2])], 2, 5, 128, 64, 5, 1000, 20),
    "tiles in chunks": (BF16, (1500, 40), [([300, 20], [17, 20]), ([1, 1400], [1, 33])], 2, 4, 128, 0, 40, 1600, 80),
    "tiles": (E4M3, (333, 60), [([300, 20], [17, 20]), ([60, 333], [60, 50])], 2, 4, 64, 100, 60, 400, 180),
    "both kernels": (BF16, (700, 2), [([300, 20], [100, 20]), ([1, 900], [1, 33])], 2, 4, 128, 0, 100, 900, 130),
    "eight waves": (E4M3, (1100, 1030), [([1200], [900]), ([300], [1])], 8, 8, 64, 0, 1030, 1200, 2060),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_bits_do_not_depend_on_the_other_sequences(name):
    dtype, (n, new), others, H, G, D, window, max_new, max_kv, tokens = CASES[name]
    print("neighbours", name, flush=True)
    P, W = 16, -(-max_kv // 16)
    B = len(others[0][0]) + 1
    own_pages = -(-n // P)
    pages = own_pages + B * W // 4 + W
    g = gen(4)
    data, scales = filled(dtype, pages, H, P, D, 4)
    mine = (torch.randn(new, H * G, D, generator=g) * 1.5).to(torch.bfloat16)
    results = []
    for turn, (lens, news) in enumerate(others):
        for at in (0, B // 2, B - 1):                          # the sequence's place among the others
            table = torch.randint(own_pages, pages, (B, W), generator=g, dtype=torch.int32)
            table[at, :own_pages] = torch.arange(own_pages, dtype=torch.int32)
            all_lens, all_new = list(lens), list(news)
            all_lens.insert(at, n)
            all_new.insert(at, new)
            starts = [turn]
            for x in all_new:
                starts.append(starts[-1] + x)
            assert starts[-1] <= tokens
            q = (torch.randn(tokens, H * G, D, generator=g) * 3).to(torch.bfloat16)
            q[starts[at]:starts[at] + new] = mine
            other = data.clone()
            if turn:                                           # the others' pages hold something else
                other = filled(dtype, pages, H, P, D, 5 + turn)[0]
                other.view(torch.uint8)[:own_pages] = data.view(torch.uint8)[:own_pages]
            batch = sz().PageBatch(table.cuda(), torch.tensor(all_lens, dtype=torch.int32).cuda(),
                                   torch.tensor(starts, dtype=torch.int32).cuda(), tokens, max_new=max_new, max_kv=max_kv)
            out, lse = sz().paged_attention(q.cuda(), on_gpu(dtype, other, scales), batch, window=window, lse=True)
            results.append((out[starts[at]:starts[at] + new].cpu(), lse[starts[at]:starts[at] + new].cpu()))
    assert bool(torch.isfinite(results[0][0]).all())
    for out, lse in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(lse, results[0][1])
