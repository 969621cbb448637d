"""The paged cache's calls against the plain 64-bit reference (pagedref.py):
write and read bit for bit, attention within the bounds that its roundings
give, over element types, head layouts, page sizes, lengths, strides, windows
and hidden rows."""
import math

import pytest
import torch

import tests.pagedref as ref

pytestmark = pytest.mark.gpu

BF16, E5M2, E4M3 = ref.BF16, ref.E5M2, ref.E4M3
DTYPES = [BF16, E5M2, E4M3]


def sz():
    import fp8_kv_cache_sz_amd
    return fp8_kv_cache_sz_amd


def gen(seed):
    return torch.Generator().manual_seed(seed)


def filled(dtype, pages, H, P, D, seed):
    """A CPU cache of random finite values: (data, scales)."""
    g = gen(seed)
    x = torch.randn(pages, 2, H, P, D, generator=g, dtype=torch.float64)
    x = x * torch.exp(torch.randn(2, H, 1, D, generator=g, dtype=torch.float64))
    if dtype == BF16:
        return x.to(torch.bfloat16), None
    data, scales = ref.quantise(x.to(torch.bfloat16).double(), dtype)
    return data, scales


def on_gpu(dtype, data, scales):
    return sz().PagedCache(dtype, data.cuda(), None if scales is None else scales.cuda())


def batch_of(table, lens, starts, tokens, **kw):
    return sz().PageBatch(table.cuda(), lens.cuda(), starts.cuda(), tokens, **kw)


def bits(t):
    return t.cpu().contiguous().view(torch.uint8)


# lens (tokens in the cache), new
SHAPES = {
    "one": ([1], [1]),
    "page_edge": ([16, 17, 15, 32], [1, 2, 15, 17]),
    "mixed": ([5, 0, 300, 64, 33], [5, 0, 1, 64, 20]),
    "many": ([(7 * i) % 41 + 1 for i in range(150)], [1 + (i % 2 if (7 * i) % 41 else 0) for i in range(150)]),
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,D,P", [(8, 128, 16), (1, 128, 64), (3, 64, 32), (5, 64, 16)])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_write_and_read(dtype, H, D, P, shape):
    lens, new = SHAPES[shape]
    print("write/read", ref.NAMES[dtype], H, D, P, shape, flush=True)
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=3, gap=2)
    data, scales = filled(dtype, pages, H, P, D, 11)
    cache = on_gpu(dtype, data, scales)
    batch = batch_of(table, kv, starts, T)
    # rows over BF16's whole range, zero rows, signed zeros, NaN and infinities
    g = gen(5)
    x = torch.randn(T, 2, H, D, generator=g) * torch.exp2(torch.randint(-120, 120, (T, 2, H, 1), generator=g).float())
    x[0::7, 0, 0] = 0.0
    x[1::5, 1, 0, 3] = -0.0
    x[2::5, 0, H - 1, 1] = math.nan
    x[3::5, 1, H - 1, 2] = math.inf
    x[3::5, 1, H - 1, 3] = -math.inf
    x[4::5, 0, 0, :] = 2.0 ** -133                     # BF16 subnormals
    x = x.to(torch.bfloat16)
    wide = torch.zeros(T, 2, H + 1, D, dtype=torch.bfloat16)
    wide[:, :, :H] = x
    wide = wide.cuda()
    sz().cache_write(cache, batch, wide[:, 0, :H], wide[:, 1, :H])      # strided rows

    want, want_s = data.clone(), None if scales is None else scales.clone()
    q, s = (x, None) if dtype == BF16 else ref.quantise(x.double(), dtype)
    for i, n in enumerate(lens):
        for t in range(int(starts[i]), int(starts[i + 1])):
            p = n - int(starts[i + 1]) + t
            pg = int(table[i, p // P])
            want.view(torch.uint8 if dtype != BF16 else torch.bfloat16)[pg, :, :, p % P] = \
                q[t] if dtype == BF16 else q[t].view(torch.uint8)
            if s is not None:
                want_s[pg, :, :, p % P] = s[t]
    same = (bits(cache.data) == bits(want))
    if dtype != BF16:                                  # a NaN has more than one bit pattern
        same |= torch.isnan(cache.data.cpu().float()) & torch.isnan(want.float())
    assert bool(same.all())
    if s is not None:
        assert torch.equal(cache.scales.cpu(), want_s)

    mark = torch.full((T, H, D), 7.0, dtype=torch.bfloat16)
    out = (mark.cuda(), mark.cuda())
    k, v = sz().cache_read(cache, batch, out=out)
    expect = mark.repeat(2, 1, 1, 1)
    for i, n in enumerate(lens):
        a, b = int(starts[i]), int(starts[i + 1])
        if b > a:
            rows = ref.gather(want, want_s, table, i, n, P)[n - (b - a):]
            expect[0, a:b], expect[1, a:b] = rows[:, 0].to(torch.bfloat16), rows[:, 1].to(torch.bfloat16)
    got = torch.stack([k, v]).cpu()
    assert bool(((bits(got) == bits(expect)).view(2, T, H, D, 2).all(-1) | (got.isnan() & expect.isnan())).all())


@pytest.mark.parametrize("dtype", [E5M2, E4M3])
def test_write_rounds_every_bf16_value(dtype):
    """Every finite BF16 pattern, each in a row with a maximum that puts it at
    another place of the FP8 range: ties, subnormals and both scale limits."""
    D, H, P = 128, 4, 16
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    every = every[torch.isfinite(every.float())]
    every = every[: len(every) // 127 * 127].view(-1, 127)
    g = gen(9)
    for lift in (0, 3, 9):
        top = every.abs().amax(-1, keepdim=True).float() * 2.0 ** lift
        top = top.clamp_max(3.3e38) * (1 + torch.rand(top.shape, generator=g) * 0.9)
        x = torch.cat([every, top.clamp_max(3.38e38).to(torch.bfloat16)], 1)
        T = x.shape[0] // (2 * H)
        x = x[: T * 2 * H].view(T, 2, H, D)
        table, kv, starts, _, pages = ref.layout([T], [T], P, seed=lift)
        cache = sz().paged_cache(pages, P, H, D, dtype)
        sz().cache_write(cache, batch_of(table, kv, starts, T), x[:, 0].contiguous().cuda(), x[:, 1].contiguous().cuda())
        q, s = ref.quantise(x.double(), dtype)
        pos = torch.arange(T)
        pg = table[0].long()[pos // P]
        assert torch.equal(cache.scales.cpu()[pg, :, :, pos % P], s)
        assert torch.equal(cache.data.cpu().view(torch.uint8)[pg, :, :, pos % P], q.view(torch.uint8))


ATTENTION = [
    # dtype, lens, new, H, G, D, P, window
    (BF16, [1], [1], 1, 1, 128, 16, 0),
    (BF16, [1, 31, 32, 33, 64, 65, 127, 128, 129], [1] * 9, 2, 4, 128, 16, 0),
    (E5M2, [1, 31, 32, 33, 64, 65, 127, 128, 129], [1] * 9, 2, 4, 128, 32, 0),
    (E4M3, [1, 31, 32, 33, 64, 65, 127, 128, 129], [1] * 9, 2, 4, 64, 16, 0),
    (BF16, [2000], [1], 4, 7, 128, 64, 0),
    (E4M3, [1999, 3, 700], [1, 1, 1], 3, 16, 128, 16, 0),
    (E5M2, [900, 40, 5], [3, 4, 5], 2, 3, 64, 16, 0),
    (BF16, [900, 40, 5], [3, 4, 5], 2, 3, 128, 128, 17),
    (E4M3, [600], [1], 8, 4, 128, 16, 1),
    (BF16, [600, 70], [2, 1], 2, 8, 64, 32, 65),
    # more than 16 rows: tiles
    (BF16, [17], [17], 1, 1, 128, 16, 0),
    (BF16, [200, 5, 130, 64], [200, 5, 130, 64], 2, 4, 128, 32, 0),
    (E5M2, [300, 77], [150, 77], 2, 4, 128, 16, 0),
    (E4M3, [300, 77], [33, 65], 3, 5, 64, 64, 0),
    (BF16, [1500], [20], 2, 4, 128, 32, 0),
    (E4M3, [1500], [129], 1, 7, 128, 16, 100),
    (BF16, [400, 129], [300, 129], 2, 2, 64, 16, 33),
    (E5M2, [260], [260], 1, 1, 64, 256, 1),
    # both kinds of sequence in one call, and sequences without new tokens or without any
    (BF16, [900, 300, 0, 64, 1], [1, 100, 0, 0, 1], 2, 4, 128, 16, 0),
    (E4M3, [20, 1000, 500], [20, 1, 2], 2, 8, 128, 32, 50),
    # more new tokens than the cache has: the first ones stand nowhere and see nothing
    (BF16, [3, 2], [5, 4], 1, 3, 128, 16, 0),
    (E5M2, [30, 0], [40, 7], 2, 4, 64, 16, 0),
    (BF16, [100], [120], 1, 4, 128, 16, 20),
    # a group larger than 16 rows, and one row per KV head
    (BF16, [100, 40], [1, 1], 1, 32, 128, 16, 0),
    (E4M3, [100, 40], [1, 1], 6, 1, 128, 16, 0),
]


def run_attention(dtype, lens, new, H, G, D, P, window, spoil=None, seed=1, gap=1, tight=True, scale=None):
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=seed, gap=gap)
    data, scales = filled(dtype, pages, H, P, D, seed + 20)
    g = gen(seed + 40)
    q = (torch.randn(T, H * G, D, generator=g) * 1.5).to(torch.bfloat16)
    if spoil is not None:
        spoil(data, scales, table, q)
    cache = on_gpu(dtype, data, scales)
    kw = dict(max_new=max(new), max_kv=max(lens)) if tight else {}
    batch = batch_of(table, kv, starts, T, **kw)
    scale = D ** -0.5 if scale is None else scale
    wide = torch.zeros(T, H * G + 1, D + 8, dtype=torch.bfloat16)
    wide[:, :H * G, :D] = q
    out = torch.full((T, H * G, D), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H * G), 3.0, dtype=torch.float32, device="cuda")
    sz().paged_attention(wide.cuda()[:, :H * G, :D], cache, batch, scale=scale, window=window, out=out, lse=lse)
    want, want_l, tol, tol_l = ref.attention(q, data, scales, table, kv, starts, P, scale, window)
    none = torch.ones(T, dtype=torch.bool)
    none[int(starts[0]):int(starts[-1])] = False
    want[none], want_l[none] = 3.0, 3.0               # tokens of no sequence keep what they held
    tol[none], tol_l[none] = 0.0, 0.0
    return out, lse, want, want_l, tol, tol_l


@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: "%s-%s-%s" % (ref.NAMES[c[0]], c[1], c[2]) if len(c[1]) < 6 else None)
@pytest.mark.parametrize("tight", [True, False], ids=["tight", "loose"])
def test_attention(case, tight):
    print("attention", case, tight, flush=True)
    out, lse, want, want_l, tol, tol_l = run_attention(*case, tight=tight)
    assert not ref.close(out, want, tol)
    assert not ref.close(lse, want_l, tol_l)
