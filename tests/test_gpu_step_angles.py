"""Rotary writes of values whose partner is 0: what comes out is a product, and
is held to its own size however small the angle."""
import pytest
import torch

import tests.pagedref as ref
import tests.stepref as step
from tests.test_gpu_paged import BF16, DTYPES, batch_of, filled, gen, on_gpu, sz

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,R,interleaved", [(128, 128, False), (128, 128, True), (64, 64, False), (64, 24, False), (128, 40, True)])
@pytest.mark.parametrize("base", [1e4, 1e7, 1e12])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_small_angles_keep_their_size(dtype, D, R, interleaved, base, sign):
    """A pair (x, 0) becomes (x c, x s) and (0, y) becomes (-y s, y c).  The
    angle's 32-bit rounding, two conversions and a fused multiply, is 3 2^-24 of
    it, the sine's series, the amplitude and the product 6 2^-24 more: 2^-20 of
    the result, whatever its size, in front of its one rounding to BF16."""
    print("angles", ref.NAMES[dtype], D, R, interleaved, base, sign, flush=True)
    m = sz()
    H, G, P = 2, 2, 16
    lens, new = [9, 70, 5000], [9, 30, 3]
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=3)
    data, scales = filled(dtype, pages, H, P, D, 11)
    cache, batch = on_gpu(dtype, data, scales), batch_of(table, kv, starts, T)
    f = sign * m.rotary_frequencies(R, base=base)
    x = torch.randn(T, H * (G + 2), D, generator=gen(R)).to(torch.bfloat16)
    pair = torch.arange(R // 2)
    first, second = (2 * pair, 2 * pair + 1) if interleaved else (pair, pair + R // 2)
    x[:, :, first[::2]] = 0                                  # the pairs' first and second values in turn
    x[:, :, second[1::2]] = 0
    positions = torch.cat([torch.arange(n - k, n) for n, k in zip(lens, new)])
    cos, sin = step.angles(positions.tolist(), f.tolist())
    g = x.cuda()
    q = m.rotary_write(cache, batch, m.Rotary(f, interleaved=interleaved), g[:, :H * G], g[:, H * G:H * G + H], g[:, H * G + H:])
    turned, _ = step.turned(x, cos, sin, interleaved, 1.0)
    got = [(q.double().cpu(), turned[:, :H * G])]
    if dtype == BF16:
        keys, _ = m.cache_read(cache, batch)
        got.append((keys.double().cpu(), turned[:, H * G:H * G + H]))
    for have, want in got:
        off = (have - want).abs() - want.abs() * (2.0 ** -8 + 2.0 ** -20)
        assert float(off.max()) <= 0, (float(off.max()), float((((have - want) / want).nan_to_num(0)).abs().max()))
