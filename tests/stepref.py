"""Plain reference of the calls of a serving step, on the CPU: whole numbers in
Python loops, angles as fractions modulo 2 pi to 50 places, products and sums
in 64 bits, with the bounds that the calls' roundings give."""
import math
from fractions import Fraction

import torch

import tests.pagedref as ref

TWO_PI = 2 * Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)


# ---- pages -------------------------------------------------------------------

def assign(page, queue, ends, table, lens, held, width, max_kv):
    """(queue, ends, table, held, capacity_short, wrong) after the call."""
    queue, table, held = queue.tolist(), [r[:] for r in table.tolist()], held.tolist()
    pages = len(queue)
    head, count = ends.tolist()
    wrong = not (0 <= head < pages and 0 <= count <= pages)
    if wrong:
        head, count = 0, 0
    taken = given = wanted = 0
    short = False
    out = held[:]
    for i, n in enumerate(lens.tolist()):
        if not (0 <= n <= max_kv and 0 <= held[i] <= width):
            wrong = True
            continue
        need = -(-n // page)
        if need > held[i]:
            wanted += need - held[i]
            if wanted <= count:
                for w in range(held[i], need):
                    table[i][w] = queue[(head + taken) % pages]
                    taken += 1
                out[i] = need
            else:
                short = True
                for w in range(held[i], need):
                    table[i][w] = -1
        else:
            for w in range(need, held[i]):
                queue[(head + count + given) % pages] = table[i][w]
                given += 1
            out[i] = need
    after = count - taken + given
    return queue, [(head + taken) % pages, min(after, pages)], table, out, short, wrong or after > pages


def slots(page, pages, table, lens, starts, tokens):
    """The slot of every token, from the table after the call."""
    out = [-1] * tokens
    for i, n in enumerate(lens):
        for t in range(starts[i], starts[i + 1]):
            p = n - (starts[i + 1] - starts[i]) + (t - starts[i])
            if p >= 0 and 0 <= table[i][p // page] < pages:
                out[t] = table[i][p // page] * page + p % page
    return out


# ---- trees -------------------------------------------------------------------

def tree(parents, lens, starts, words):
    """{token: (mask words as signed 64-bit, position)} and whether a parent was none."""
    out, wrong = {}, False
    for i, n in enumerate(lens):
        new = starts[i + 1] - starts[i]
        masks = []
        for j in range(new):
            p = parents[starts[i] + j]
            if not -1 <= p < j:
                wrong, p = True, -1
            masks.append(1 << j | (masks[p] if p >= 0 else 0))
            row = [(masks[j] >> 64 * w) & (2 ** 64 - 1) for w in range(words)]
            out[starts[i] + j] = ([x - 2 ** 64 if x >= 2 ** 63 else x for x in row], n - new + bin(masks[j]).count("1") - 1)
    return out, wrong


def named(masks, tok, first, n):
    """The new tokens that a row of masks names."""
    return [j for w, x in enumerate(masks[tok].tolist()) for j in range(64 * w, 64 * w + 64)
            if x >> (j - 64 * w) & 1 and first <= j < n]


def tree_attention(q, data, scales, table, lens, starts, page, scale, window, masks, only=None):
    """(out, lse, tol_out, tol_lse) as pagedref.attention, the visible keys by
    the masks; the bounds are derived there.  `only`: the tokens to look at."""
    T, Hq, D = q.shape
    H = data.shape[2]
    u = 2.0 ** -24
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    tol_o, tol_l = out.clone(), lse.clone()
    for i, n in enumerate(lens.tolist()):
        s0, s1 = int(starts[i]), int(starts[i + 1])
        past = n - (s1 - s0)
        if s1 == s0:
            continue
        kv = ref.gather(data, scales, table, i, n, page)
        for r in range(s1 - s0):
            at = []
            if only is not None and s0 + r not in only:
                continue
            if past + r >= 0:
                new = named(masks, s0 + r, max(0, -past), s1 - s0)
                lo = max(0, past + max(1, len(new)) - window) if window else 0
                at = list(range(lo, max(past, 0))) + [past + j for j in new]
            for h in range(Hq):
                if not at:
                    out[s0 + r, h], lse[s0 + r, h], tol_o[s0 + r, h], tol_l[s0 + r, h] = 0.0, -math.inf, 0.0, 0.0
                    continue
                k, v = kv[at, 0, h * H // Hq], kv[at, 1, h * H // Hq]
                x = q[s0 + r, h].double()
                s = (k @ x) * scale
                size = (k.abs() @ x.abs()) * scale
                lse[s0 + r, h] = torch.logsumexp(s, 0)
                p = torch.softmax(s, 0)
                out[s0 + r, h] = p @ v
                e = float((D + 2) * 2 * u * size.max() + 2 * u * s.abs().max() + 2.0 ** -22 + 2 * len(at) * u)
                a = p @ v.abs()
                tol_o[s0 + r, h] = (2.0 ** -8 * (a + out[s0 + r, h].abs()) + 2 * e * a) * (1 + 2.0 ** -7) + 1e-38
                tol_l[s0 + r, h] = e + 4 * u * lse[s0 + r, h].abs() + 2.0 ** -22
    return out, lse, tol_o, tol_l


# ---- rotary ------------------------------------------------------------------

def angles(positions, frequencies):
    """cos, sin [tokens, R / 2] in 64 bits: p f modulo 2 pi as a fraction."""
    c = torch.empty(len(positions), len(frequencies), dtype=torch.float64)
    s = c.clone()
    known = {}
    for t, p in enumerate(positions):
        if p not in known:
            known[p] = [float(Fraction(f) * p % TWO_PI) for f in frequencies]
        c[t] = torch.tensor([math.cos(a) for a in known[p]], dtype=torch.float64)
        s[t] = torch.tensor([math.sin(a) for a in known[p]], dtype=torch.float64)
    return c, s


def turned(x, cos, sin, interleaved, amplitude):
    """x [tokens, heads, D] in 64 bits, and |x| + |partner| of each value (0
    where nothing is turned)."""
    x = x.double()
    R = 2 * cos.shape[1]
    i = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    j = i + 1 if interleaved else i + R // 2
    out, size = x.clone(), torch.zeros_like(x)
    c, s = cos[:, None], sin[:, None]
    out[..., i] = amplitude * (x[..., i] * c - x[..., j] * s)
    out[..., j] = amplitude * (x[..., j] * c + x[..., i] * s)
    size[..., i] = size[..., j] = abs(amplitude) * (x[..., i].abs() + x[..., j].abs())
    return out, size


def turned_bound(want, size):
    """How far a BF16 result that was computed in 32 bits may be off.  The
    fraction of a turn is cut at 2^-32 turns (1.5e-9) and its product with 2 pi
    rounded twice (pi/4 2^-23: 9.4e-8); the series, seven rounded steps of
    falling size, and the amplitude add 4 2^-24 (2.4e-7) to the sine and cosine: 3.4e-7 of |x| + |y|.
    Two products and their sum add 2 2^-24 (1.2e-7): below 2^-21 together.  Then
    one rounding to BF16."""
    before = size * 2.0 ** -21
    return before + 2.0 ** -8 * (want.abs() + before) + 2.0 ** -134
