"""What attention of at most 16 rows of a sequence (new tokens times query heads
of a KV head) keeps: the result's own rounding, and little beside it.

A probability p enters its product as two BF16 terms, its upper 16 bits and
the rest of less than 2^-7 p, which is rounded to BF16 (2^-8 of it): 2^-15 p.
Its 32-bit value is off by e p (pagedref.attention's e: the score's sum, the
exponent's product, the power; the sum of the powers is off by e too), its
products with V are exact in 32 bits, and the two sums of n of them are off by
2 n 2u each, u = 2^-24.  Sums are rescaled where the running reference rises,
where waves meet and where chunks are joined: 2^-22 for each such power and 2u
for its product, over at most 64 of them.  The sum then takes one rounding to
BF16: half a step, 2^-8 of the power of two below the result."""
import torch

import tests.pagedref as ref

U = 2.0 ** -24


def bounds(x, K, V, scale):
    """64-bit rows x [R, D] over visible keys K, V [n, D]: (out, tolerance)."""
    n, D = K.shape
    s = x @ K.T.contiguous() * scale
    size = x.abs() @ K.abs().T.contiguous() * scale
    w = torch.softmax(s, -1)
    out, a = w @ V, w @ V.abs()
    e = (D + 2) * 2 * U * size.amax(-1) + 2 * U * s.abs().amax(-1) + 2.0 ** -22 + 2 * n * U
    inner = (2.0 ** -15 + 2 * e + 4 * n * U + 64 * (2.0 ** -22 + 2 * U)).unsqueeze(-1) * a * (1 + 2.0 ** -10)
    return out, inner + half_step(out.abs() + inner)


def half_step(x):
    """Half a BF16 step at magnitude x."""
    _, e = torch.frexp(x.clamp_min(2.0 ** -126))                # x = f 2^e, f in [1/2, 1)
    return torch.ldexp(torch.ones_like(x), e - 9)


def attention(q, data, scales, table, lens, starts, page, scale, window):
    """(out, tolerance) [T, q_heads, D] in 64 bits; NaN for tokens of no
    sequence, (0, 0) where no key is seen."""
    T, Hq, D = q.shape
    H = data.shape[2]
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.float64)
    tol = out.clone()
    for i, n in enumerate(lens.tolist()):
        s0, s1 = int(starts[i]), int(starts[i + 1])
        if s1 == s0:
            continue
        kv = ref.gather(data, scales, table, i, n, page)
        for t in range(s0, s1):
            p = n - s1 + t
            if p < 0:
                out[t], tol[t] = 0.0, 0.0
                continue
            at = slice(max(0, p - window + 1) if window else 0, p + 1)
            for h in range(H):
                g = slice(h * (Hq // H), (h + 1) * (Hq // H))
                out[t, g], tol[t, g] = bounds(q[t, g].double(), kv[at, 0, h], kv[at, 1, h], scale)
    return out, tol
