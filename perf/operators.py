"""The paged KV cache's operators, as they are measured: writing new tokens'
keys and values into pages (quantised to FP8 on the way in), reading tokens
back out of pages, and attention of new tokens over the pages.

A cache is one tensor [pages, 2, kv_heads, page_tokens, head_dim] (keys, then
values) of BF16, FP8 E5M2 or FP8 E4M3; FP8 rows (one token's one head) carry a
power-of-two scale 2**(byte - 127).  A batch lists, for each sequence, its
pages, its length with the new tokens, and where its new tokens start in the
packed token axis: new token i of a sequence with n new tokens and length L
stands at position L - n + i.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEVICE = "cuda"
FP8 = {"e5m2": torch.float8_e5m2, "e4m3": torch.float8_e4m3fn}
FP8_MAX_EXP = {"e5m2": 15, "e4m3": 8}        # the largest finite value is 1.75 * 2**this


def listed():
    def case(name, op, dtype, seqs, past, new, ragged, kv_heads, head_dim, page, group=1, window=0):
        return {"name": name, "op": op, "dtype": dtype, "seqs": seqs, "past": past, "new": new, "ragged": ragged,
                "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "group": group, "window": window}
    return [
        # one user's next token goes into the cache: latency alone
        case("write_token_e4m3", "write", "e4m3", 1, 1000, 1, False, 8, 128, 16),
        # one step of a server with 256 users, into the codec's own FP8 type
        case("write_step_e5m2", "write", "e5m2", 256, 500, 1, True, 8, 128, 64),
        # a batch of prompts of different lengths
        case("write_prompts_e4m3", "write", "e4m3", 7, 0, 8192, True, 8, 128, 32),
        # a short conversation leaves the cache
        case("read_short_bf16", "read", "bf16", 1, 0, 77, False, 8, 128, 16),
        # a 64K-token context leaves the cache (4 KV heads of 128, one layer of the long-context configuration)
        case("read_long_e5m2", "read", "e5m2", 1, 0, 65536, False, 4, 128, 64),
        # many sequences of different lengths
        case("read_ragged_e4m3", "read", "e4m3", 33, 0, 4001, True, 8, 128, 32),
        # one user's next token over a short conversation: latency
        case("attend_token_bf16", "attend", "bf16", 1, 1000, 1, False, 8, 128, 16, group=4),
        # one step of 64 users with up to 8K tokens each (8 KV heads of 128, as the 8K-token configuration)
        case("attend_step_e4m3", "attend", "e4m3", 64, 8191, 1, True, 8, 128, 32, group=4),
        # one user's next token over a 64K-token context, seven query heads to a KV head
        case("attend_long_bf16", "attend", "bf16", 1, 65535, 1, False, 4, 128, 64, group=7),
        # five draft tokens of each of 16 users, checked at once, over a sliding window of 1,000 tokens, small heads
        case("attend_drafts_e5m2", "attend", "e5m2", 16, 5000, 5, True, 2, 64, 16, group=8, window=1000),
        # a chunk of a long prompt over what the cache already holds
        case("attend_chunk_e5m2", "attend", "e5m2", 1, 16384, 2048, False, 8, 128, 64, group=4),
        # a batch of whole prompts of different lengths
        case("attend_prompts_bf16", "attend", "bf16", 6, 0, 4096, True, 8, 128, 32, group=4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng: random.Random):
    """A case of the same ranges: one token to long contexts, one sequence to
    hundreds, every element type, head layout, page size; the plain form's
    padded scores stay under 2**31 values."""
    op = rng.choice(["write", "read", "attend", "attend"])
    c = {"op": op, "dtype": rng.choice(["bf16", "e5m2", "e4m3"]), "ragged": rng.random() < 0.7,
         "head_dim": rng.choice([64, 128, 128]), "page": rng.choice([16, 32, 64, 128]), "group": 1, "window": 0}
    c["kv_heads"] = rng.choice([1, 2, 3, 4, 8])
    if op != "attend":
        c["seqs"] = _log_int(rng, 1, 256)
        c["new"] = _log_int(rng, 1, max(1, 65536 // c["seqs"]))
        c["past"] = _log_int(rng, 1, max(1, 65536 // c["seqs"])) if rng.random() < 0.5 else 0
        return c
    c["group"] = rng.choice([1, 2, 4, 5, 7, 8])
    c["seqs"] = _log_int(rng, 1, 64)
    c["new"] = rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 9, max(9, 4096 // c["seqs"]))])
    # padded scores seqs * new * query heads * keys, and padded keys seqs * keys * kv_heads
    keys = min(65536, 2 ** 31 // (c["seqs"] * c["new"] * c["kv_heads"] * c["group"]),
               2 ** 22 // (c["seqs"] * c["kv_heads"]))
    c["past"] = _log_int(rng, 1, max(1, keys - c["new"]))
    if rng.random() < 0.25:
        c["window"] = _log_int(rng, 1, c["past"] + c["new"])
    return c


def _lengths(case):
    """Each sequence's (past, new) tokens, the same for every seed.  Ragged
    cases step down from the longest to about an eighth, in no simple stride."""
    n = case["seqs"]
    if not case["ragged"] or n == 1:
        return [(case["past"], case["new"])] * n
    rnd = random.Random(case["past"] * 31 + case["new"])
    share = [1.0 - 0.875 * i / (n - 1) for i in range(n)]
    rnd.shuffle(share)
    return [(int(case["past"] * s), max(1, int(case["new"] * s)) if case["past"] == 0 else case["new"]) for s in share]


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    lens = _lengths(case)
    H, D, P, dtype = case["kv_heads"], case["head_dim"], case["page"], case["dtype"]
    kv = [p + n for p, n in lens]
    width = -(-max(kv) // P)
    needed = [-(-x // P) for x in kv]
    pages = sum(needed) + 3                            # a pool is never all in use
    order = torch.randperm(pages, generator=g, device=DEVICE, dtype=torch.int64).to(torch.int32)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device=DEVICE)
    at = 0
    for b, w in enumerate(needed):
        table[b, :w] = order[at:at + w]
        at += w
    starts = [0]
    for _, n in lens:
        starts.append(starts[-1] + n)
    T = starts[-1]
    s = {"case": dict(case), "table": table, "max_new": max(n for _, n in lens), "max_kv": max(kv), "tokens": T,
         "kv_lens": torch.tensor(kv, dtype=torch.int32, device=DEVICE),
         "starts": torch.tensor(starts, dtype=torch.int32, device=DEVICE)}
    # cache contents: values with a scale for each channel, as keys and values of real models have
    chan = torch.exp(0.5 * torch.randn(2, H, 1, D, generator=g, device=DEVICE))
    shape = (pages, 2, H, P, D)
    if dtype == "bf16":
        s["data"] = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.bfloat16).mul_(chan.to(torch.bfloat16))
        s["scales"] = None
    else:
        # whole FP8 range of finite values that a row under its scale holds, scales around those of unit-sized rows
        lift = 2.0 ** (FP8_MAX_EXP[dtype] - 2)
        x = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.bfloat16)
        s["data"] = x.mul_(chan.to(torch.bfloat16) * lift / 4).clamp_(-1.75 * lift * 4, 1.75 * lift * 4).to(FP8[dtype])
        s["scales"] = torch.randint(127 - FP8_MAX_EXP[dtype] + 1, 127 - FP8_MAX_EXP[dtype] + 4, shape[:-1], generator=g,
                                    device=DEVICE, dtype=torch.uint8)
        del x
    if case["op"] == "write":
        # K and V as slices of one projection's output, as models make them
        kv_new = torch.randn(T, 2, H, D, generator=g, device=DEVICE) * chan.reshape(1, 2, H, D)
        kv_new = kv_new.to(torch.bfloat16)
        s["k"], s["v"] = kv_new[:, 0], kv_new[:, 1]
    elif case["op"] == "attend":
        q = torch.randn(T, H * case["group"], D, generator=g, device=DEVICE)
        s["q"] = (q / chan[0].reshape(1, H, 1, D).expand(T, H, case["group"], D).reshape(T, -1, D)).to(torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(D)
        s["window"] = case["window"]
    if own:
        import fp8_kv_cache_sz_amd as sz
        kind = {"bf16": sz.BF16, "e5m2": sz.E5M2, "e4m3": sz.E4M3}[dtype]
        s["cache"] = sz.PagedCache(kind, s["data"], s["scales"])
        s["batch"] = sz.PageBatch(table, s["kv_lens"], s["starts"], T, max_new=s["max_new"], max_kv=s["max_kv"])
        if case["op"] == "attend":
            s["ws"] = sz.attention_workspace(s["cache"], s["batch"], H * case["group"])
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        import fp8_kv_cache_sz_amd as sz
        if op == "write":
            sz.cache_write(state["cache"], state["batch"], state["k"], state["v"], check=False)
            return _cache_values(state)
        if op == "read":
            return sz.cache_read(state["cache"], state["batch"], check=False)
        return sz.paged_attention(state["q"], state["cache"], state["batch"], scale=state["scale"],
                                  window=state["window"], lse=True, ws=state["ws"], check=False)
    if op == "write":
        _plain_write(state)
        return _cache_values(state)
    if op == "read":
        return _plain_read(state)
    return _plain_attend(state)


def _cache_values(state):
    return [state["data"]] if state["scales"] is None else [state["data"], state["scales"]]


# ---- plain forms -----------------------------------------------------------

def _places(state):
    """Each new token's (page, row)."""
    starts, P = state["starts"].long(), state["case"]["page"]
    t = torch.arange(state["tokens"], device=DEVICE)
    b = torch.searchsorted(starts, t, right=True) - 1
    pos = state["kv_lens"].long()[b] - starts[b + 1] + t
    return state["table"].long()[b, pos // P], pos % P


def _pow2(k):
    """2.0**k for whole k in -126..127, from its bits."""
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _plain_write(state):
    case = state["case"]
    page, row = _places(state)
    x = torch.stack([state["k"], state["v"]], 1)                              # [T, 2, H, D]
    if case["dtype"] == "bf16":
        state["data"][page, :, :, row] = x
        return
    x = x.float()
    a = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs().amax(-1)
    bits = a.view(torch.int32)
    k = (bits >> 23) - 127 - FP8_MAX_EXP[case["dtype"]] + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    k = k.clamp_min(-126)
    q = (x * _pow2(-k).unsqueeze(-1)).to(FP8[case["dtype"]])
    state["data"].view(torch.uint8)[page, :, :, row] = q.view(torch.uint8)
    state["scales"][page, :, :, row] = (k + 127).to(torch.uint8)


def _values(state, page, row):
    """Rows [..., 2, H, D] of the cache at the places [...], in 32 bits."""
    if state["scales"] is None:
        return state["data"][page, :, :, row].float()
    q = state["data"].view(torch.uint8)[page, :, :, row].view(state["data"].dtype).float()
    return q * _pow2(state["scales"][page, :, :, row].int() - 127).unsqueeze(-1)


def _plain_read(state):
    x = _values(state, *_places(state)).to(torch.bfloat16)
    return x[:, 0].contiguous(), x[:, 1].contiguous()


def _plain_attend(state):
    """All sequences at once, padded to the longest."""
    case = state["case"]
    B, H, G, D, P = case["seqs"], case["kv_heads"], case["group"], case["head_dim"], case["page"]
    n, keys, T = state["max_new"], state["max_kv"], state["tokens"]
    starts, lens = state["starts"].long(), state["kv_lens"].long()
    j = torch.arange(keys, device=DEVICE)
    inside = j < lens[:, None]                                               # [B, keys]
    page = torch.where(inside, state["table"].long()[:, j // P], 0)
    kv = _values(state, page, (j % P).expand(B, keys))                       # [B, keys, 2, H, D]
    k = kv[:, :, 0].permute(0, 2, 3, 1).contiguous()                         # [B, H, D, keys]
    v = torch.where(inside[:, None, :, None], kv[:, :, 1].permute(0, 2, 1, 3), 0.0)      # [B, H, keys, D]
    del kv
    i = torch.arange(n, device=DEVICE)
    new = starts[1:] - starts[:-1]
    at = (starts[:-1, None] + i).clamp_max(T - 1)                            # [B, n] token of each padded row
    pos = lens[:, None] - new[:, None] + i
    q = state["q"][at].float().reshape(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    seen = (j <= pos[..., None]) & inside[:, None]                           # [B, n, keys]
    if state["window"]:
        seen &= j > pos[..., None] - state["window"]
    s = torch.matmul(q, k).mul_(state["scale"]).reshape(B, H, n, G, keys)
    del k
    s = s.masked_fill_(~seen[:, None, :, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, H, n * G, keys), v).reshape(B, H, n, G, D) / torch.where(l == 0, 1.0, l)
    lse = (m + l.log()).squeeze(-1)
    t = torch.arange(T, device=DEVICE)
    b = torch.searchsorted(starts, t, right=True) - 1
    i = t - starts[b]
    return o[b, :, i].reshape(T, H * G, D).to(torch.bfloat16), lse[b, :, i].reshape(T, H * G)


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    lens = _lengths(case)
    H, G, D = case["kv_heads"], case["group"], case["head_dim"]
    T = sum(n for _, n in lens)
    row = 2 * H * (2 * D if case["dtype"] == "bf16" else D + 1)               # one token's K and V in the cache
    pages = sum(-(-(p + n) // case["page"]) for p, n in lens)
    if case["op"] != "attend":
        return {"bytes": T * (row + 4 * H * D) + 4 * pages, "flops": 2 * T * H * D}
    w = case["window"]
    keys, pairs = 0, 0
    for past, n in lens:
        first = max(0, past + 1 - w) if w else 0
        keys += past + n - first
        if w:
            pairs += sum(min(w, past + i + 1) for i in range(n))
        else:
            pairs += n * past + n * (n + 1) // 2
    return {"bytes": keys * row + T * H * G * (4 * D + 4) + 4 * pages, "flops": 4 * D * H * G * pairs}


# ---- 64 bits -------------------------------------------------------------------

def _power(k):
    """2**k in 64 bits, exact also where a power function's last bit is not."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _rounded(x, kind):
    """x in 64 bits to the nearest FP8 value, ties to even, by the spacing of
    the values around it."""
    man, low = (2, -14) if kind == "e5m2" else (3, -6)
    _, e = torch.frexp(x)
    step = _power(torch.clamp(e - 1, min=low) - man)
    return torch.round(x / step) * step


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    H, G, D, P = case["kv_heads"], case["group"], case["head_dim"], case["page"]
    table, lens, starts = s["table"].tolist(), s["kv_lens"].tolist(), s["starts"].tolist()

    def rows(b, lo, hi):
        """[hi - lo, 2, H, D] in 64 bits: positions lo..hi of sequence b."""
        pages = torch.tensor(table[b], device=DEVICE)[lo // P:(hi - 1) // P + 1]
        x = s["data"].view(torch.uint8 if s["scales"] is not None else torch.bfloat16)[pages]
        x = x.view(s["data"].dtype).double()
        if s["scales"] is not None:
            x = x * _power(s["scales"][pages].long() - 127).unsqueeze(-1)
        x = x.permute(0, 3, 1, 2, 4).reshape(-1, 2, H, D)
        return x[lo % P:lo % P + hi - lo]

    if case["op"] == "write":
        data = s["data"].double()
        scales = None if s["scales"] is None else s["scales"].double()
        for b, n in enumerate(lens):
            first, new = starts[b], starts[b + 1] - starts[b]
            x = torch.stack([s["k"][first:first + new], s["v"][first:first + new]], 1).double()
            pos = torch.arange(n - new, n, device=DEVICE)
            page = torch.tensor(table[b], device=DEVICE)[pos // P]
            if scales is not None:
                a = x.abs().amax(-1, keepdim=True)
                top = 1.75 * 2.0 ** FP8_MAX_EXP[case["dtype"]]
                f, e = torch.frexp(a / top)                                   # a / top = f 2**e, f in [1/2, 1)
                k = torch.where(f == 0.5, e - 1, e).clamp_min(-126)
                x = _rounded(x / _power(k), case["dtype"])
                scales[page, :, :, pos % P] = (k + 127).double().squeeze(-1)
            data[page, :, :, pos % P] = x
        return [data] if scales is None else [data, scales]
    if case["op"] == "read":
        x = torch.cat([rows(b, n - (starts[b + 1] - starts[b]), n) for b, n in enumerate(lens)])
        return x[:, 0], x[:, 1]
    out = torch.empty(s["tokens"], H * G, D, dtype=torch.float64, device=DEVICE)
    lse = torch.empty(s["tokens"], H * G, dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(lens):
        x = rows(b, 0, n)
        first, new = starts[b], starts[b + 1] - starts[b]
        part = max(1, 2 ** 27 // (n * G))                                     # query tokens at a time
        for h in range(H):
            K, V = x[:, 0, h].contiguous(), x[:, 1, h].contiguous()
            for i0 in range(0, new, part):
                i1 = min(new, i0 + part)
                q = s["q"][first + i0:first + i1, h * G:(h + 1) * G].double()
                z = (q.reshape(-1, D) @ K.T.contiguous() * s["scale"]).reshape(i1 - i0, G, n)
                p = torch.arange(n - new + i0, n - new + i1, device=DEVICE)[:, None, None]
                j = torch.arange(n, device=DEVICE)
                hidden = (j > p) | (j <= p - s["window"]) if s["window"] else j > p
                z = z.masked_fill(hidden, float("-inf"))
                r = torch.logsumexp(z, -1)
                w = torch.exp(z - r.unsqueeze(-1))
                out[first + i0:first + i1, h * G:(h + 1) * G] = (w.reshape(-1, n) @ V).reshape(i1 - i0, G, D)
                lse[first + i0:first + i1, h * G:(h + 1) * G] = r
    return out, lse
