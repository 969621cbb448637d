"""Weights at the ends of their range: keys whose probability is 0 add nothing,
however large their values are, and the smallest ones still carry an infinity.
One sequence of one head is cut into chunks of a block for each wave; 64
sequences of 16 heads are not cut, so that waves take block after block."""
import math

import pytest
import torch

import tests.pagedref as ref
from tests.test_gpu_paged import BF16, E4M3, E5M2, batch_of, on_gpu, sz

pytestmark = pytest.mark.gpu

P, n = 16, 700


def run(dtype, D, new, G, H, seqs, late, value, ordinary):
    """Every 32nd key has score `late` (in powers of two) and `value`, the
    others score 0 and `ordinary` values; q is one unit vector, scores are
    exact.  All sequences read the same pages."""
    table, kv, starts, T, pages = ref.layout([n], [new], P, seed=2)
    data = torch.zeros(pages, 2, H, P, D, dtype=torch.float64)
    table, kv, starts, T = table.repeat(seqs, 1), kv.repeat(seqs), torch.arange(seqs + 1, dtype=torch.int32) * new, T * seqs
    for p in range(n):
        pg, r = int(table[0, p // P]), p % P
        data[pg, 0, :, r, 0] = late if p % 32 == 9 else 0.0
        data[pg, 1, :, r] = value if p % 32 == 9 else ordinary
    scales = None
    if dtype == BF16:
        data = data.to(torch.bfloat16)
    else:
        data, scales = ref.quantise(data, dtype)              # powers of two, infinities: exact
    q = torch.zeros(T, H * G, D, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    out = sz().paged_attention(q.cuda(), on_gpu(dtype, data, scales),
                               batch_of(table, kv, starts, T, max_new=new, max_kv=n), scale=math.log(2.0))
    return out.float().cpu()


SHAPES = [(BF16, 128, 1, 4), (BF16, 64, 1, 1), (E5M2, 128, 1, 8), (E4M3, 64, 1, 2), (BF16, 64, 5, 4), (E4M3, 128, 3, 8),
          (BF16, 128, 40, 2), (E5M2, 128, 40, 2)]


@pytest.mark.parametrize("H,seqs", [(1, 1), (16, 64)])
@pytest.mark.parametrize("dtype,D,new,G", SHAPES)
def test_values_of_no_weight_do_not_count(dtype, D, new, G, H, seqs):
    # 2^-4096 is 0 in any arithmetic here, and 22 times 0 times 2^126 nothing
    for value in (2.0 ** 126, -2.0 ** 126):
        assert bool((run(dtype, D, new, G, H, seqs, -4096.0, value, 0.0) == 0.0).all()), value


@pytest.mark.parametrize("H,seqs", [(1, 1), (16, 64)])
@pytest.mark.parametrize("dtype,D,new,G", [s for s in SHAPES if s[0] != E4M3])
@pytest.mark.parametrize("late", [-16.0, -112.0])
def test_values_of_little_weight_stay_infinite(dtype, D, new, G, H, seqs, late):
    for value in (math.inf, -math.inf):
        assert bool((run(dtype, D, new, G, H, seqs, late, value, 1.0) == value).all()), value
