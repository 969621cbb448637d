"""Attention of prompts that fill the card several times over, two workgroups to
a SIMD: waves of one workgroup then run far apart, and every place where one
may overwrite what another still reads has its chance.  Each call repeats bit
for bit, and sampled rows are compared with 64-bit attention."""
import pytest
import torch

import tests.pagedref as ref
from tests.test_gpu_paged import BF16, E4M3, E5M2, batch_of, filled, gen, on_gpu, sz

pytestmark = pytest.mark.gpu

CASES = [
    # dtype, lens, new, H, G, D, P, window
    (BF16, [2048, 1700, 1400, 1111], [2048, 1700, 1400, 1111], 8, 4, 128, 32, 0),
    (BF16, [900] * 24, [300] * 24, 4, 2, 64, 16, 0),
    (E4M3, [2048, 1900], [2048, 1900], 8, 4, 128, 64, 0),            # eight waves
    (E5M2, [1500, 1300, 900], [1500, 1300, 900], 8, 4, 64, 16, 400),      # eight waves
    (E5M2, [700] * 40, [40] * 40, 8, 4, 128, 16, 0),                 # four
    (E4M3, [500] * 40, [33] * 40, 8, 4, 64, 32, 0),                  # four
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s-%dx%d-%d" % (ref.NAMES[c[0]], len(c[1]), c[1][0], c[5]))
def test_prompts_repeat_and_are_right(case):
    dtype, lens, new, H, G, D, P, window = case
    print("full card", case, flush=True)
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=7)
    data, scales = filled(dtype, pages, H, P, D, 31)
    cache = on_gpu(dtype, data, scales)
    q = (torch.randn(T, H * G, D, generator=gen(5)) * 1.5).to(torch.bfloat16)
    on = q.cuda()
    batch = batch_of(table, kv, starts, T, max_new=max(new), max_kv=max(lens))
    ws = sz().attention_workspace(cache, batch, H * G)
    call = lambda: sz().paged_attention(on, cache, batch, window=window, lse=True, ws=ws, check=False)
    first, first_l = call()
    for rep in range(20):
        out, lse = call()
        assert torch.equal(out, first) and torch.equal(lse, first_l), rep
    cache.raise_status()
    # One token in 41, all heads.  Bounds as in ref.attention:
    # e for a probability, 2^-8 for its rounding and for the result's.
    got, got_l, u, scale = first.cpu(), first_l.cpu(), 2.0 ** -24, D ** -0.5
    for i, n in enumerate(lens):
        if i % 6:
            continue
        rows = ref.gather(data, scales, table, i, n, P)
        for t in range(int(starts[i]), int(starts[i + 1]), 41):
            p = n - int(starts[i + 1]) + t
            at = slice(max(0, p - window + 1) if window else 0, p + 1)
            k, v = rows[at, 0].transpose(0, 1), rows[at, 1].transpose(0, 1)               # [H, keys, D]
            x = q[t].double().view(H, G, D)
            s = torch.matmul(x, k.transpose(1, 2).contiguous()) * scale
            size = torch.matmul(x.abs(), k.abs().transpose(1, 2).contiguous()) * scale
            w = torch.softmax(s, -1)
            want, a = torch.matmul(w, v.contiguous()), torch.matmul(w, v.abs().contiguous())
            e = (D + 2) * 2 * u * size.amax(-1) + 2 * u * s.abs().amax(-1) + 2.0 ** -22 + 2 * s.shape[-1] * u
            tol = (2.0 ** -8 * (a + want.abs()) + 2 * e.unsqueeze(-1) * a) * (1 + 2.0 ** -7) + 1e-38
            assert not ref.close(got[t].view(H, G, D), want, tol), (i, t)
            want_l = torch.logsumexp(s, -1)
            assert not ref.close(got_l[t].view(H, G), want_l, e + 4 * u * want_l.abs() + 2.0 ** -22), (i, t)
