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
    "empties": ([3] + [0] * 130 + [5] + [0] * 70 + [2, 9], [3] + [0] * 130 + [4] + [0] * 70 + [2, 1]),
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
    # 17 to 32 rows: two blocks of rows, or tiles
    (BF16, [300, 90, 40], [5, 4, 6], 2, 5, 64, 16, 0),
    (E5M2, [300, 90, 17], [17, 1, 17], 2, 1, 128, 32, 0),
    (E4M3, [900, 33, 200], [4, 2, 3], 1, 8, 128, 16, 40),
    (E4M3, [1300, 31], [8, 1], 2, 4, 64, 64, 0),
    (E5M2, [130, 20], [1, 1], 1, 32, 64, 16, 0),
    (BF16, [10, 700], [20, 25], 1, 1, 64, 16, 7),
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


# Keys in 4 to 36 chunks that a launch of their own joins: a group of lanes to
# a row and several, more rows to a workgroup than heads, heads left over, rows
# of both kernels.
JOINED = [
    (BF16, [1500], [20], 3, 5, 64, 32, 0),
    (E4M3, [420], [33], 1, 7, 128, 16, 0),
    (E4M3, [420], [33], 1, 7, 128, 16, 150),
    (E5M2, [1000, 200, 40, 9], [6, 1, 40, 1], 1, 9, 128, 16, 0),
    (BF16, [700, 100], [40, 17], 2, 3, 128, 64, 0),
    (BF16, [9000, 8000, 17], [2, 1, 2], 2, 7, 64, 64, 0),
    (E5M2, [9000, 100, 4500], [1, 1, 1], 2, 11, 128, 256, 0),
]


@pytest.mark.parametrize("case", JOINED, ids=lambda c: "%s-%s-%s" % (ref.NAMES[c[0]], c[1], c[2]))
def test_attention_joined(case):
    print("joined", case, flush=True)
    out, lse, want, want_l, tol, tol_l = run_attention(*case)
    assert not ref.close(out, want, tol)
    assert not ref.close(lse, want_l, tol_l)


# Larger than a laid-out test needs, but the smallest that fills the tile
# kernel's eight-wave form (FP8, 256 rows a workgroup over all of the card).
def test_attention_many_rows_fp8():
    H, G, D, P = 8, 8, 64, 64
    lens, new = [1100, 1029], [1025, 1029]
    dtype = E4M3
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=2)
    data, scales = filled(dtype, pages, H, P, D, 22)
    q = (torch.randn(T, H * G, D, generator=gen(42)) * 1.5).to(torch.bfloat16)
    cache = on_gpu(dtype, data, scales)
    out, lse = sz().paged_attention(q.cuda(), cache, batch_of(table, kv, starts, T, max_new=1029, max_kv=1100),
                                    window=700, lse=True)
    # every 37th token and all heads of two KV heads against the reference
    for i, n in enumerate(lens):
        rows = ref.gather(data, scales, table, i, n, P)
        for t in range(int(starts[i]), int(starts[i + 1]), 37):
            p = n - int(starts[i + 1]) + t
            at = slice(max(0, p - 699), p + 1)
            for h in range(0, H * G, 11):
                k, v = rows[at, 0, h // G], rows[at, 1, h // G]
                s = (k @ q[t, h].double()) * D ** -0.5
                w = torch.softmax(s, 0)
                want = w @ v
                tol = 2.0 ** -8 * (w @ v.abs() + want.abs()) * 1.02 + 1e-6 * (w @ v.abs())
                assert not ref.close(out[t, h], want, tol), (i, t, h)
                # 2^-24 (2 (D + 2) |s| terms + 2 n), as ref.attention's
                assert abs(float(lse[t, h]) - float(torch.logsumexp(s, 0))) < 2e-5


def spoil_hidden(value):
    """Places `value` in K and V of positions that some or all rows do not
    see: behind each sequence's end in its last page, and in the newest
    token's own row (which earlier tokens of the call do not see)."""
    def spoil(data, scales, table, q):
        d = data.view(torch.uint8) if data.element_size() == 1 else data
        bad = torch.full((1,), value).to(data.dtype)
        bad = bad.view(torch.uint8) if data.element_size() == 1 else bad
        for i, (n, P) in enumerate(spoil.sequences):
            last = int(table[i, (n - 1) // P])
            r = (n - 1) % P
            d[last, :, :, r + 1:] = bad
            d[last, :, :, r] = bad
    return spoil


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("case", [
    (BF16, [200, 40], [5, 3], 2, 3, 128, 16, 0),
    (E5M2, [200, 40], [5, 3], 2, 3, 64, 32, 0),
    (E5M2, [200, 40], [9, 6], 2, 3, 128, 32, 0),
    (BF16, [200, 70], [90, 70], 2, 2, 128, 16, 0),
    (E5M2, [200, 70], [90, 70], 1, 2, 128, 64, 0),
    (BF16, [200, 70], [90, 70], 1, 2, 64, 16, 37),
], ids=lambda c: ref.NAMES[c[0]] + str(c[1]) + str(c[2]))
def test_attention_hidden_values_stay_hidden(case, value):
    """The newest token's K and V, and the page behind it, hold NaN or
    infinities: rows that do not see them are exact, rows that do get what
    the formula gives."""
    spoil = spoil_hidden(value)
    spoil.sequences = [(n, case[6]) for n in case[1]]
    print("hidden", case, value, flush=True)
    out, lse, want, want_l, tol, tol_l = run_attention(*case, spoil=spoil)
    # NaN where the formula is NaN; rows of the newest token have an infinite
    # score somewhere: 0 inf and inf - inf are NaN in any precision
    newest = torch.isnan(want).any(-1) | torch.isinf(want).any(-1) | ~torch.isfinite(want_l)
    clean = ~newest
    assert not ref.close(out[clean.cuda()], want[clean], tol[clean])
    assert not ref.close(lse[clean.cuda()], want_l[clean], tol_l[clean])
    assert bool((~torch.isfinite(out.cpu().float()))[newest].any(-1).all())


@pytest.mark.parametrize("rows", ["few", "many"])
@pytest.mark.parametrize("kinds", [(math.inf,), (-math.inf,), (math.inf, -math.inf), (math.nan,)],
                         ids=["inf", "-inf", "both", "nan"])
def test_attention_infinite_values_seen_by_some(rows, kinds):
    """Infinities and NaN in V alone (finite scores): the tokens that see
    them get exactly what sums of them are, the others stay finite."""
    H, G, D, P, n = 1, 2, 128, 16, 100
    new = 6 if rows == "few" else 80
    table, kv, starts, T, pages = ref.layout([n], [new], P, seed=4)
    data, _ = filled(BF16, pages, H, P, D, 3)
    q = torch.randn(T, H * G, D, generator=gen(8)).to(torch.bfloat16)
    plain = data.clone()
    places = [n - 5, n - 3]                                    # d = 7 of position n - 5, d = 7 and 9 of n - 3
    for k, p in enumerate(places):
        pg, r = int(table[0, p // P]), p % P
        data[pg, 1, 0, r, 7] = kinds[k % len(kinds)]
        if k:
            data[pg, 1, 0, r, 9] = kinds[0]
    run = lambda d: sz().paged_attention(q.cuda(), on_gpu(BF16, d, None), batch_of(table, kv, starts, T,
                                         max_new=new, max_kv=n)).cpu()
    got, clean = run(data), run(plain)
    for t in range(T):
        p = n - new + t
        seen = [kinds[k % len(kinds)] for k, at in enumerate(places) if at <= p]
        expect = clean[t].clone()
        if seen:
            expect[:, 7] = sum(seen)                           # inf - inf and NaN are NaN
        if len(seen) == 2:
            expect[:, 9] = kinds[0]
        rest = [d for d in range(D) if d not in (7, 9)]
        assert torch.equal(got[t][:, rest], clean[t][:, rest]), t
        for d in (7, 9):
            a, b = got[t][:, d].float(), expect[:, d].float()
            assert bool(((a == b) | (a.isnan() & b.isnan())).all()), (t, d, a, b)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("new", [1, 14, 40])
@pytest.mark.parametrize("later", [0.0, 40.0], ids=["level", "outweighed"])
def test_attention_infinite_values_seen_by_all(dtype, new, later):
    """Infinities and NaN in V far before the new tokens: the sums of them,
    also where a later key outweighs theirs by e^400."""
    H, G, D, P, n = 1, 2, 128, 16, 700
    table, kv, starts, T, pages = ref.layout([n], [new], P, seed=4)
    data, scales = filled(dtype, pages, H, P, D, 3)
    q = (torch.randn(1, 1, D, generator=gen(8)) + 0.01 * torch.randn(T, H * G, D, generator=gen(9))).to(torch.bfloat16)

    def put(which, p, values):
        pg, r = int(table[0, p // P]), p % P
        for d, x in values:
            data[pg, which, 0, r, d] = x
        return pg, r
    put(1, 100, [(7, math.inf), (9, -math.inf), (11, math.inf), (13, math.nan)])
    put(1, 301, [(7, math.inf), (11, -math.inf), (15, -math.inf)])
    pg, r = put(0, 600, list(enumerate((q[0, 0].double() * later).tolist())) if later else [])
    if later and scales is not None:
        scales[pg, 0, 0, r] = 127
    out, lse = sz().paged_attention(q.cuda(), on_gpu(dtype, data, scales),
                                    batch_of(table, kv, starts, T, max_new=new, max_kv=n), lse=True)
    want, want_l, tol, tol_l = ref.attention(q, data, scales, table, kv, starts, P, D ** -0.5, 0)
    assert bool(torch.isfinite(want_l).all()) and bool(want[..., 7].isinf().all())
    assert not ref.close(lse, want_l, tol_l)
    special = [7, 9, 11, 13, 15]
    assert not ref.close(out[..., special], want[..., special], tol[..., special])
    rest = [d for d in range(D) if d not in special]
    assert not ref.close(out[..., rest], want[..., rest], tol[..., rest])


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (E4M3, 128)])
@pytest.mark.parametrize("near", [0, 16])
def test_attention_far_and_near_rows(dtype, D, near):
    """32 rows, one half with scores of +-2^25 and the other with ordinary
    ones: each half as it would be by itself."""
    H, G, P, n, T = 1, 4, 16, 500, 8
    table, kv, starts, T, pages = ref.layout([n], [T], P, seed=6)
    data, scales = filled(dtype, pages, H, P, D, 13)
    q = torch.randn(T, G, D, generator=gen(3))
    rows = torch.arange(T * G).view(T, G)
    at = (rows >= near) & (rows < near + 16)                   # the ordinary ones
    q = torch.where(at.unsqueeze(-1), q, q * 2.0 ** 25).to(torch.bfloat16)
    out, lse = sz().paged_attention(q.cuda(), on_gpu(dtype, data, scales),
                                    batch_of(table, kv, starts, T, max_new=T, max_kv=n), lse=True)
    want, want_l, tol, tol_l = ref.attention(q, data, scales, table, kv, starts, P, D ** -0.5, 0)
    assert not ref.close(out[at.cuda()], want[at], tol[at])
    assert not ref.close(lse[at.cuda()], want_l[at], tol_l[at])
    # the leading score is far ahead of the next: its V row, rounded once
    assert not ref.close(out[~at.cuda()], want[~at], want[~at].abs() * 2.0 ** -8)
    assert not ref.close(lse[~at.cuda()], want_l[~at], want_l[~at].abs() * 2.0 ** -20)


def test_attention_scores_out_of_range():
    """Scores of +-2^40 and beyond: the largest alone counts, nothing overflows."""
    H, D, P, n = 1, 64, 16, 90
    table, kv, starts, T, pages = ref.layout([n, n], [1, 60], P, seed=6)
    data, _ = filled(BF16, pages, H, P, D, 13)
    data[:, 0] *= 2.0 ** 20
    q = (torch.randn(T, 2, D, generator=gen(3)) * 2.0 ** 20).to(torch.bfloat16)
    out, lse = sz().paged_attention(q.cuda(), on_gpu(BF16, data, None), batch_of(table, kv, starts, T), lse=True)
    want, want_l, _, _ = ref.attention(q, data, None, table, kv, starts, P, D ** -0.5, 0)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    # the leading score is far ahead of the next: the result is its V row, rounded once
    assert not ref.close(out, want, want.abs() * 2.0 ** -8)
    assert not ref.close(lse, want_l, want_l.abs() * 2.0 ** -20)
    # all scores minus infinity: 0/0, as the formula says
    data[:, 0] = -math.inf
    q = torch.ones(T, 2, D, dtype=torch.bfloat16)
    out = sz().paged_attention(q.cuda(), on_gpu(BF16, data, None), batch_of(table, kv, starts, T))
    assert bool(torch.isnan(out).all())


def test_results_do_not_depend_on_neighbours_or_repetition():
    """The same sequence alone, among others and again gives the same bits
    under the same bounds (no atomics in the sums)."""
    H, G, D, P = 2, 4, 128, 16
    table, kv, starts, T, pages = ref.layout([1000, 500, 1000], [1, 1, 1], P, seed=1)
    data, scales = filled(E4M3, pages, H, P, D, 5)
    cache = on_gpu(E4M3, data, scales)
    q = torch.randn(T, H * G, D, generator=gen(1)).to(torch.bfloat16).cuda()
    batch = batch_of(table, kv, starts, T, max_new=1, max_kv=1000)
    ws = sz().attention_workspace(cache, batch, H * G)
    first = sz().paged_attention(q, cache, batch, ws=ws)
    for _ in range(20):
        assert torch.equal(first, sz().paged_attention(q, cache, batch, ws=ws))
    assert int(ws[:4096].view(torch.int32).abs().sum()) == 0      # counters are left at zero


def bad_batches(table, kv, starts, T):
    """Batches that contradict themselves, their bounds or the cache."""
    t = table.clone()
    t[0, 0] = 10 ** 6
    yield "page past the cache", (t, kv, starts)
    t = table.clone()
    t[1, 0] = -1
    yield "negative page", (t, kv, starts)
    k = kv.clone()
    k[1] = 10 ** 8
    yield "length past the table", (table, k, starts)
    k = kv.clone()
    k[0] = -5
    yield "negative length", (table, k, starts)
    s = starts.clone()
    s[1] = 10 ** 7
    yield "start past the tokens", (table, kv, s)
    s = starts.clone()
    s[1], s[2] = s[2].clone(), s[1].clone()
    yield "starts descend", (table, kv, s)
    s = starts.clone()
    s[0] = -3
    yield "negative start", (table, kv, s)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("new", [(1, 1, 1), (40, 3, 25)], ids=["tokens", "prompts"])
def test_bad_batches_are_reported_and_touch_nothing_else(dtype, new):
    """Each contradiction is reported by every call, and by the check before a
    write, which then writes nothing; sequences that are right keep their
    results."""
    H, G, D, P = 2, 4, 128, 16
    lens = [50, 33, 70]
    table, kv, starts, T, pages = ref.layout(lens, list(new), P, seed=9)
    data, scales = filled(dtype, pages, H, P, D, 7)
    q = torch.randn(T, H * G, D, generator=gen(2)).to(torch.bfloat16).cuda()
    x = torch.randn(T, H, D, generator=gen(3)).to(torch.bfloat16).cuda()
    cache = on_gpu(dtype, data, scales)
    good = sz().paged_attention(q, cache, batch_of(table, kv, starts, T, max_new=max(new), max_kv=80)).cpu()
    for name, (t, k, s) in bad_batches(table, kv, starts, T):
        print("bad batch:", name, flush=True)
        batch = batch_of(t, k, s, T, max_new=max(new), max_kv=80)
        before = bits(cache.data), None if scales is None else bits(cache.scales)
        with pytest.raises(sz().SplitZipError):
            sz().cache_write(cache, batch, x, x)
        assert torch.equal(bits(cache.data), before[0])
        assert scales is None or torch.equal(bits(cache.scales), before[1])
        # a read looks at the pages of its own tokens only (the first page of
        # a sequence is theirs if they start in it)
        seq = {"page past the cache": 0, "negative page": 1}.get(name)
        if seq is not None and lens[seq] - new[seq] >= P:
            sz().cache_read(cache, batch)
        else:
            with pytest.raises(sz().SplitZipError):
                sz().cache_read(cache, batch)
        with pytest.raises(sz().SplitZipError):
            sz().paged_attention(q, cache, batch)
        assert int(cache.status.item()) == 0                  # reported once, then clear
        # unchecked: the third sequence is untouched by the others' faults
        if name not in ("starts descend", "start past the tokens"):
            out = torch.zeros_like(q)
            sz().paged_attention(q, cache, batch, out=out, check=False)
            a, b = int(starts[2]), int(starts[3])
            assert torch.equal(out[a:b].cpu(), good[a:b]), name
            cache.status.zero_()
    # more new tokens than max_new, and a length over max_kv
    for kw in (dict(max_new=max(new) - 1, max_kv=80), dict(max_new=max(new), max_kv=69)):
        with pytest.raises(sz().SplitZipError):
            sz().paged_attention(q, cache, batch_of(table, kv, starts, T, **kw))
    # two sequences that write one page
    t = table.clone()
    t[1, (lens[1] - 1) // P] = t[0, (lens[0] - 1) // P]
    with pytest.raises(sz().SplitZipError):
        sz().cache_write(cache, batch_of(t, kv, starts, T), x, x)
    sz().cache_read(cache, batch_of(t, kv, starts, T))         # reading it twice is fine


def test_a_serving_run_with_the_codec():
    """Prompt and steps as they are used: write into E5M2 pages, attend, send
    the pages through the codec into another cache, go on there; the other
    cache gives the same bits."""
    m = sz()
    H, G, D, P, pages = 4, 2, 128, 16, 40
    g = gen(12)
    table = torch.randperm(pages, generator=g).to(torch.int32)[:36].view(3, 12)
    lens, new = [0, 0, 0], [70, 33, 128]
    cache = m.paged_cache(pages, P, H, D, m.E5M2)
    other = m.paged_cache(pages, P, H, D, m.E5M2)
    plain = torch.zeros(3, 192, 2, H, D, dtype=torch.bfloat16)
    for step in range(4):
        lens = [a + b for a, b in zip(lens, new)]
        starts = torch.tensor([0] + [sum(new[:i + 1]) for i in range(3)], dtype=torch.int32)
        T = int(starts[-1])
        batch = batch_of(table, torch.tensor(lens, dtype=torch.int32), starts, T, max_new=max(new), max_kv=192)
        qkv = torch.randn(T, (G + 2) * H, D, generator=g).to(torch.bfloat16)
        x = qkv.cuda()
        q, k, v = x[:, :G * H], x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:]
        m.cache_write(cache, batch, k, v)
        a = m.paged_attention(q, cache, batch)
        if step == 1:                                           # the cache moves: values losslessly, scales as they are
            book = m.calibrate(cache.data)
            buf, size, _ = m.encode(cache.data, book)
            assert size < cache.data.numel()
            m.decode(buf[:size], m.E5M2, cache.data.numel(), out=other.data.view(torch.uint8).view(-1))
            other.scales.copy_(cache.scales)
            assert torch.equal(bits(other.data), bits(cache.data))
        if step >= 1:
            m.cache_write(other, batch, k, v)                   # as the first cache got them
            assert torch.equal(bits(other.data), bits(cache.data)) and torch.equal(other.scales, cache.scales)
            assert torch.equal(a, m.paged_attention(q, other, batch))
        # 64-bit reference over everything written so far
        data, scales = cache.data.cpu(), cache.scales.cpu()
        want, _, tol, _ = ref.attention(qkv[:, :G * H], data, scales, table, torch.tensor(lens), starts, P, D ** -0.5, 0)
        assert not ref.close(a, want, tol)
        # read back: within half an E5M2 step of what was written
        kk, vv = m.cache_read(cache, batch)
        top = k.float().abs().amax(-1, keepdim=True)
        assert bool(((kk.float() - k.float()).abs() <= k.float().abs() / 8 + top * 2.0 ** -31).all())
        new = [1, 1, 1] if step else [5, 1, 2]
