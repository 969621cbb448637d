"""Single tokens and drafts keep probabilities in two BF16 terms: on the GPU
within the bound of that (tests/pagedfine.py), and on the CPU, where the same
arithmetic is played through, a bound that one term alone would not meet."""
import pytest
import torch

import tests.pagedfine as fine
import tests.pagedref as ref

BF16, E5M2, E4M3 = ref.BF16, ref.E5M2, ref.E4M3


def played(x, K, V, scale, terms):
    """Attention with 32-bit probabilities that enter the product as one or two
    BF16 terms; everything else in 64 bits."""
    s = x @ K.T.contiguous() * scale
    p = torch.exp(s - s.amax(-1, keepdim=True)).float()
    high = (p.view(torch.int32) & -65536).view(torch.float32)
    rest = (p - high).to(torch.bfloat16)
    o = high.double() @ V + (rest.double() @ V if terms == 2 else 0)
    return (o / p.double().sum(-1, keepdim=True)).to(torch.bfloat16).double()


@pytest.mark.parametrize("n", [20, 300, 3000])
@pytest.mark.parametrize("positive", [False, True])
def test_the_bound_tells_one_term_from_two(n, positive):
    g = torch.Generator().manual_seed(n)
    x, K, V = (torch.randn(m, 128, generator=g).to(torch.bfloat16).double() for m in (16, n, n))
    V = V.abs() if positive else V
    want, tol = fine.bounds(x, K, V, 128 ** -0.5)
    assert not ref.close(played(x, K, V, 128 ** -0.5, 2), want, tol)
    # 3,000 values of both signs: p|V| is 30 times the result and the worst case
    # of its 32-bit sum, 4 n 2^-24 of it, more than what one term loses
    if positive or n < 3000:
        assert ref.close(played(x, K, V, 128 ** -0.5, 1), want, tol)


CASES = [
    # dtype, lens, new, H, G, D, P, window
    (BF16, [1], [1], 1, 1, 128, 16, 0),
    (BF16, [1, 31, 33, 64, 129, 1000], [1] * 6, 2, 4, 128, 16, 0),
    (E4M3, [1, 31, 33, 64, 129, 1000], [1] * 6, 2, 4, 64, 16, 0),
    (E5M2, [900, 40, 5], [3, 4, 5], 2, 3, 64, 16, 0),
    (E4M3, [2500, 3, 700], [1, 1, 1], 3, 16, 128, 16, 0),
    (BF16, [900, 40, 5], [3, 4, 5], 2, 3, 128, 128, 17),
    (E5M2, [600, 3], [2, 5], 2, 2, 128, 32, 65),
    (BF16, [800] * 40, [1] * 40, 8, 2, 128, 16, 0),               # contexts that are not cut
    (E4M3, [777] * 40, [2] * 40, 8, 4, 64, 16, 0),
    (E5M2, [777] * 40, [1] * 40, 8, 1, 128, 16, 300),
    # 17 to 32 rows in two blocks
    (E5M2, [300, 90, 17], [5, 1, 8], 2, 4, 128, 32, 0),
    (BF16, [700, 40], [8, 7], 2, 4, 64, 16, 0),
    (E4M3, [500] * 40, [4] * 40, 8, 8, 128, 16, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("later", [False, True], ids=["level", "rising"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s-%s-%dx%d" % (ref.NAMES[c[0]], c[1][:3], c[2][0], c[4]))
def test_few_rows_are_as_exact_as_their_result(case, later):
    """`later`: keys grow along the sequence, so that the reference rises."""
    from tests.test_gpu_paged import batch_of, filled, gen, on_gpu, sz
    dtype, lens, new, H, G, D, P, window = case
    print("fine", case, later, flush=True)
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=2, gap=1)
    if lens[0] == lens[-1] and len(lens) > 10:                    # many alike: on a few's pages
        table = table[:3].repeat(len(lens), 1)[:len(lens)].contiguous()
        used, at = torch.unique(table, return_inverse=True)
        table, pages = at.to(torch.int32), len(used)
    data, scales = filled(dtype, pages, H, P, D, 6)
    if later:
        for i in range(min(len(lens), 3)):
            for w in range(-(-lens[i] // P)):
                pg = int(table[i, w])
                if dtype == BF16:
                    data[pg, 0] *= 1 + 4 * w * P / max(lens)
                else:
                    scales[pg, 0] += int(2.5 * w * P / max(lens))
    q = (torch.randn(T, H * G, D, generator=gen(3)) * 1.5).to(torch.bfloat16)
    out = torch.full((T, H * G, D), 3.0, dtype=torch.bfloat16, device="cuda")
    sz().paged_attention(q.cuda(), on_gpu(dtype, data, scales), batch_of(table, kv, starts, T, max_new=max(new), max_kv=max(lens)),
                         window=window, out=out)
    want, tol = fine.attention(q, data, scales, table, kv, starts, P, D ** -0.5, window)
    none = want.isnan().all(-1).all(-1)
    want[none], tol[none] = 3.0, 0.0
    assert not ref.close(out, want, tol)
