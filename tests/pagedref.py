"""Plain 64-bit reference of the paged cache's calls, on the CPU, with the
bounds that rounding puts on a 32-bit kernel with BF16 probabilities."""
import math

import torch

BF16, E5M2, E4M3 = 0, 1, 2
ELEMENT = {BF16: torch.bfloat16, E5M2: torch.float8_e5m2, E4M3: torch.float8_e4m3fn}
TOP = {E5M2: 57344.0, E4M3: 448.0}
NAMES = {BF16: "bf16", E5M2: "e5m2", E4M3: "e4m3"}


def layout(lens, new, page, seed=0, spare=2, gap=0):
    """Page table (every page used once, shuffled), kv_lens, starts and the
    token count for sequences of `lens` tokens, the last `new` of them new.
    `gap` tokens before the first and behind the last belong to no sequence."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    width = max(need + [1])
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), width), -7, dtype=torch.int32)       # unused entries are not page numbers
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    starts = [gap]
    for n in new:
        starts.append(starts[-1] + n)
    return (table, torch.tensor(lens, dtype=torch.int32), torch.tensor(starts, dtype=torch.int32), starts[-1] + gap,
            pages)


def quantise(x, dtype):
    """[..., D] 64-bit values -> (FP8 tensor, scale bytes), by the header's
    rule in Python integers and comparisons."""
    finite = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    a = finite.amax(-1)
    k = torch.full(a.shape, -126, dtype=torch.int64)
    for step in range(-126, 128):
        k = torch.where(a > TOP[dtype] * 2.0 ** step, torch.full_like(k, step + 1), k)
    y = x * torch.tensor([2.0 ** -i for i in range(-126, 129)], dtype=torch.float64)[k + 126].unsqueeze(-1)
    return round_fp8(y, dtype), (k + 127).to(torch.uint8)


def round_fp8(y, dtype):
    """64-bit values to FP8, nearest even, from the sorted list of the type's values."""
    every = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    val = every.view(ELEMENT[dtype]).double()
    pos = torch.isfinite(val) & (every < 128)
    grid, code = val[pos], every[pos]                                   # ascending, code parity = last bit
    mag = y.abs()
    hi = torch.searchsorted(grid, mag.nan_to_num(0.0, 0.0, 0.0).contiguous()).clamp_max(len(grid) - 1)
    lo = (hi - 1).clamp_min(0)
    dl, dh = mag - grid[lo], grid[hi] - mag
    up = (dh < dl) | ((dh == dl) & (code[hi] % 2 == 0))
    q = torch.where(up, code[hi], code[lo])
    q = torch.where(mag == 0, torch.zeros_like(q), q)
    inf_code = 0x7C if dtype == E5M2 else 0x7F
    q = torch.where(torch.isinf(y), torch.full_like(q, inf_code), q)
    q = torch.where(torch.isnan(y), torch.full_like(q, 0x7F), q)
    return (q | (torch.signbit(y).to(torch.uint8) << 7)).view(ELEMENT[dtype])


def dequantise(data, scales):
    """64-bit values of a cache tensor, or of rows of one."""
    x = data.double()
    if scales is None:
        return x
    power = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64)
    return x * power[scales.long()].unsqueeze(-1)


def gather(data, scales, table, i, n, page):
    """[n, 2, H, D] 64-bit rows of positions 0..n-1 of sequence i."""
    pos = torch.arange(n)
    pg = table[i].long()[pos // page]
    rows = data.view(torch.uint8) if data.element_size() == 1 else data
    rows = rows[pg, :, :, pos % page]
    if data.element_size() == 1:
        rows = rows.view(data.dtype)
    return dequantise(rows, None if scales is None else scales[pg, :, :, pos % page])


def attention(q, data, scales, table, lens, starts, page, scale, window):
    """(out, lse, tol_out, tol_lse) in 64 bits for the rows of the sequences;
    NaN in the tolerances of tokens that belong to none.

    With u = 2^-24 a score of D products, each exact in 32 bits, is off by at
    most (D + 2) 2u sum |scale q_d K_d| (2u: the accumulation may truncate);
    the exponent's one rounded product adds 2u |s|, the power itself 2^-22, a
    sum over n keys 2 n u: e in all, relative, for each probability and for
    their sum.  Each probability is then rounded to BF16 (2^-8 of it), and so
    is the result."""
    T, Hq, D = q.shape
    H = data.shape[2]
    G = Hq // H
    u = 2.0 ** -24
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    tol_o, tol_l = out.clone(), lse.clone()
    for i, n in enumerate(lens.tolist()):
        s0, s1 = int(starts[i]), int(starts[i + 1])
        if s1 == s0:
            continue
        kv = gather(data, scales, table, i, n, page)
        pos = torch.arange(n - (s1 - s0), n)
        j = torch.arange(n)
        seen = j[None] <= pos[:, None]
        if window:
            seen &= j[None] > pos[:, None] - window
        for h in range(Hq):
            K, V = kv[:, 0, h // G], kv[:, 1, h // G]
            x = q[s0:s1, h].double()
            for r in range(s1 - s0):                                    # row by row: hidden keys take no part at all
                at = seen[r].nonzero().flatten()
                if len(at) == 0:
                    out[s0 + r, h], lse[s0 + r, h] = 0.0, -math.inf
                    tol_o[s0 + r, h], tol_l[s0 + r, h] = 0.0, 0.0
                    continue
                k, v = K[at], V[at]
                s = (k @ x[r]) * scale
                size = (k.abs() @ x[r].abs()) * scale
                lse[s0 + r, h] = torch.logsumexp(s, 0)
                p = torch.softmax(s, 0)
                out[s0 + r, h] = p @ v
                e = float((D + 2) * 2 * u * size.max() + 2 * u * s.abs().max() + 2.0 ** -22 + 2 * len(at) * u)
                a = p @ v.abs()
                tol_o[s0 + r, h] = (2.0 ** -8 * (a + out[s0 + r, h].abs()) + 2 * e * a) * (1 + 2.0 ** -7) + 1e-38
                tol_l[s0 + r, h] = e + 4 * u * lse[s0 + r, h].abs() + 2.0 ** -22
    return out, lse, tol_o, tol_l


def close(got, want, tol):
    """All within tol, NaN and infinities in the same places; returns a message or ''."""
    got = got.double().cpu()
    if not torch.equal(torch.isnan(got), torch.isnan(want)):
        return "NaN in other places: %d, %d wanted" % (torch.isnan(got).sum(), torch.isnan(want).sum())
    inf = torch.isinf(want)
    if not torch.equal(got[inf], want[inf]):
        return "infinities differ"
    ok = torch.isfinite(want)
    far = (got[ok] - want[ok]).abs() - tol[ok].nan_to_num(math.inf)
    if far.numel() and not float(far.max()) <= 0:
        w = int(far.argmax())
        return "off by %g at %g, allowed %g" % ((got[ok] - want[ok]).abs()[w], want[ok][w], tol[ok][w])
    return ""
