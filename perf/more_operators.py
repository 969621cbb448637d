"""A serving step that drafts trees of tokens over the paged KV cache, as its
operators are measured: pages assigned to sequences from their lengths, masks
and positions of the trees, rotary positions on the way into the cache,
attention of the trees' tokens, and the accepted tokens' rows moved to where
the next step expects them.

Caches and batches are those of perf/operators.py: [pages, 2, kv_heads,
page_tokens, head_dim] of BF16, E5M2 or E4M3 (FP8 rows under a scale
2**(byte - 127)); sequence i has kv_lens[i] tokens, of which the last
starts[i + 1] - starts[i] are new.
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
    def assign(name, seqs, past, new, page, short=False):
        return {"name": name, "op": "assign", "seqs": seqs, "past": past, "new": new, "page": page, "short": short}

    def tree(name, seqs, nodes, ragged):
        return {"name": name, "op": "tree", "seqs": seqs, "past": 500, "new": nodes, "ragged": ragged}

    def rows(name, op, dtype, seqs, past, new, ragged, kv_heads, head_dim, page, group, **more):
        return {"name": name, "op": op, "dtype": dtype, "seqs": seqs, "past": past, "new": new, "ragged": ragged,
                "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "group": group, **more}

    return [
        # one step of a server with 256 users: one token each, some of them done, few need a page
        assign("assign_step", 256, 8191, 1, 64),
        # a thousand prompts come in at once, small pages
        assign("assign_prompts", 1000, 0, 2048, 16),
        # one step of 16 users, 26 drafted tokens each
        tree("tree_step", 16, 26, False),
        # wide searches of many users at once: 500 drafted tokens, ragged
        tree("tree_wide", 128, 500, True),
        # one user's next token: latency alone
        rows("rotary_token_e4m3", "rotary", "e4m3", 1, 1000, 1, False, 8, 128, 16, 4, rotated=128, layout="half",
             scaled=False),
        # drafted trees of 64 users behind long contexts, half of each head rotated, in neighbouring pairs
        rows("rotary_trees_bf16", "rotary", "bf16", 64, 100000, 24, True, 4, 128, 64, 7, rotated=64,
             layout="interleaved", scaled=True),
        # a batch of prompts of different lengths
        rows("rotary_prompts_e5m2", "rotary", "e5m2", 7, 0, 8192, True, 8, 128, 32, 4, rotated=128, layout="half",
             scaled=True),
        # one user's tree over a short conversation: latency
        rows("attend_tree_bf16", "attend", "bf16", 1, 1000, 13, False, 8, 128, 16, 4, window=0),
        # eight drafted tokens of each of 64 users: 32 rows to a KV head
        rows("attend_small_trees_e5m2", "attend", "e5m2", 64, 4000, 8, True, 8, 128, 32, 4, window=0),
        # 61 drafted tokens of each of 32 users with up to 8K tokens: 244 rows to a KV head
        rows("attend_trees_e4m3", "attend", "e4m3", 32, 8192, 61, True, 8, 128, 32, 4, window=0),
        # five of 26 drafted tokens were accepted, all 32 layers' rows of 16 users
        rows("keep_step_bf16", "keep", "bf16", 16, 100, 26, True, 8, 128, 16, 1, layers=32, kept=5),
        # eight of 64, 28 layers of 4 heads, 64 users
        rows("keep_many_e5m2", "keep", "e5m2", 64, 100, 64, True, 4, 128, 16, 1, layers=28, kept=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng: random.Random):
    """A case of the same ranges; the plain attention's padded scores stay
    under 2**27 values, all layers' pages of a keep under 2**29 bytes."""
    op = rng.choice(["assign", "tree", "rotary", "rotary", "attend", "attend", "attend", "keep"])
    if op == "assign":
        seqs = _log_int(rng, 1, 2000)
        new = rng.choice([1, _log_int(rng, 1, 16), _log_int(rng, 1, max(1, min(65536, 2 ** 20 // seqs)))])
        return {"op": op, "seqs": seqs, "past": rng.choice([0, _log_int(rng, 1, max(1, min(65536, 2 ** 22 // seqs)))]),
                "new": new, "page": rng.choice([16, 32, 64, 128]), "short": rng.random() < 0.2}
    if op == "tree":
        new = _log_int(rng, 1, 1024)
        return {"op": op, "seqs": _log_int(rng, 1, max(1, 2 ** 16 // new)), "past": _log_int(rng, 1, 65536), "new": new,
                "ragged": rng.random() < 0.7}
    c = {"op": op, "dtype": rng.choice(["bf16", "e5m2", "e4m3"]), "ragged": rng.random() < 0.7,
         "head_dim": rng.choice([64, 128, 128]), "page": rng.choice([16, 32, 64, 128]),
         "kv_heads": rng.choice([1, 2, 3, 4, 8]), "group": rng.choice([1, 2, 4, 5, 7, 8])}
    if op == "rotary":
        c["seqs"] = _log_int(rng, 1, 256)
        c["new"] = _log_int(rng, 1, max(1, min(32768, 2 ** 20 // (c["kv_heads"] * (c["group"] + 1))) // c["seqs"]))
        # the past's pages are there, and are not looked at: their number is bounded
        c["past"] = _log_int(rng, 1, min(2 ** 17, 2 ** 22 // (c["seqs"] * c["kv_heads"]))) if rng.random() < 0.6 else 0
        c["rotated"] = rng.choice([c["head_dim"], c["head_dim"], 64, 32, 16])
        c["layout"] = rng.choice(["half", "interleaved"])
        c["scaled"] = rng.random() < 0.5
    elif op == "attend":
        c["seqs"] = _log_int(rng, 1, 64)
        c["new"] = rng.choice([_log_int(rng, 1, 16), _log_int(rng, 8, 64), _log_int(rng, 32, 200)])
        keys = min(65536, 2 ** 27 // (c["seqs"] * c["new"] * c["kv_heads"] * c["group"]),
                   2 ** 21 // (c["seqs"] * c["kv_heads"]))
        c["past"] = _log_int(rng, 1, max(1, keys - c["new"]))
        c["window"] = _log_int(rng, 1, c["past"] + c["new"]) if rng.random() < 0.25 else 0
    else:
        c["group"] = 1
        c["new"] = _log_int(rng, 2, 128)
        c["kept"] = rng.randint(1, max(1, min(10, c["new"] // 2)))
        c["layers"] = rng.choice([1, rng.randint(2, 28)])
        token = 2 * c["kv_heads"] * c["head_dim"] * (2 if c["dtype"] == "bf16" else 1)
        most = 2 ** 29 // (token * c["layers"])                              # tokens
        c["seqs"] = _log_int(rng, 1, max(1, min(256, most // (c["new"] + 2 * c["page"] + 64))))
        c["past"] = _log_int(rng, 1, max(1, min(4000, most // c["seqs"] - c["new"] - 2 * c["page"])))
    return c


def _shares(case):
    n = case["seqs"]
    if not case.get("ragged", True) or n == 1:
        return [1.0] * n
    rnd = random.Random(case["past"] * 31 + case["new"])
    share = [1.0 - 0.875 * i / (n - 1) for i in range(n)]
    rnd.shuffle(share)
    return share


def _lengths(case):
    """Each sequence's (past, new) tokens, the same for every seed.  Ragged
    cases step down from the longest to about an eighth, in no simple stride;
    new tokens are ragged where there is no past or where they are a tree's."""
    trees = case["op"] in ("tree", "keep")
    return [(int(case["past"] * s), max(min(case["new"], 2), int(case["new"] * s)) if case["past"] == 0 or trees
             else case["new"]) for s in _shares(case)]


def _drafted(case):
    return case["past"] > 0 and 1 < case["new"] <= 64


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEVICE)


def _parents(lens, g):
    """Trees as a search makes them: each token's parent is one of the eight
    before it, the first has none, and now and then another has none either."""
    T = sum(n for _, n in lens)
    i = torch.cat([torch.arange(n, device=DEVICE) for _, n in lens])
    back = torch.randint(1, 9, (T,), generator=g, device=DEVICE)
    root = torch.rand(T, generator=g, device=DEVICE) < 0.02
    return torch.where(root, -1, (i - back).clamp_min(-1)).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    op = case["op"]
    lens = _lengths(case)
    starts = [0]
    for _, n in lens:
        starts.append(starts[-1] + n)
    T, kv = starts[-1], [p + n for p, n in lens]
    s = {"case": dict(case), "tokens": T, "max_new": max(n for _, n in lens), "max_kv": max(kv), "starts": _ints(starts)}
    if op == "assign":
        _prepare_pool(s, lens, kv, g)
        return s
    s["kv_lens"] = _ints(kv)
    if op == "tree":
        s["parents"] = _parents(lens, g)
        if own:
            import fp8_kv_cache_sz_amd as sz
            s["batch"] = sz.PageBatch(torch.zeros(len(kv), 1, dtype=torch.int32, device=DEVICE), s["kv_lens"],
                                      s["starts"], T, max_new=s["max_new"], max_kv=s["max_kv"])
        return s
    H, D, P, dtype, G = case["kv_heads"], case["head_dim"], case["page"], case["dtype"], case["group"]
    # A rotation writes the new tokens' pages alone: the past's are all one page there
    needed = [-(-x // P) for x in kv]
    first = [p // P if op == "rotary" else 0 for p, _ in lens]
    pages = sum(needed) - sum(first) + 3               # a pool is never all in use
    order = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    table = torch.zeros(len(lens), max(needed), dtype=torch.int32, device=DEVICE)
    at = 0
    for b, (f, w) in enumerate(zip(first, needed)):
        table[b, :f] = order[-1]
        table[b, f:w] = order[at:at + w - f]
        at += w - f
    s["table"] = table
    # cache contents: values with a scale for each channel, as keys and values of real models have
    chan = torch.exp(0.5 * torch.randn(2, H, 1, D, generator=g, device=DEVICE))
    shape = (pages, 2, H, P, D)
    s["layers"] = []
    for _ in range(case.get("layers", 1)):
        if dtype == "bf16":
            data = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.bfloat16).mul_(chan.to(torch.bfloat16))
            s["layers"].append((data, None))
            continue
        lift = 2.0 ** (FP8_MAX_EXP[dtype] - 2)
        x = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.bfloat16)
        data = x.mul_(chan.to(torch.bfloat16) * lift / 4).clamp_(-1.75 * lift * 4, 1.75 * lift * 4).to(FP8[dtype])
        s["layers"].append((data, torch.randint(127 - FP8_MAX_EXP[dtype] + 1, 127 - FP8_MAX_EXP[dtype] + 4, shape[:-1],
                                                generator=g, device=DEVICE, dtype=torch.uint8)))
    s["data"], s["scales"] = s["layers"][0]
    if op == "rotary":
        # q, K and V as slices of one projection's output, as models make them
        x = torch.randn(T, H * G + 2 * H, D, generator=g, device=DEVICE)
        x[:, H * G:] *= chan.reshape(1, 2 * H, D)
        x = x.to(torch.bfloat16)
        s["q"], s["k"], s["v"] = x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:]
        s["frequencies"] = _frequencies(case)
        # drafted tokens stand behind the past by their depth in the tree, prompts' tokens at their places
        s["positions"] = _tree(s, _parents(lens, g), s["kv_lens"])[1] if _drafted(case) else None
        s["amplitude"] = 0.1 * math.log(8.0) + 1.0 if case["scaled"] else 1.0
    elif op == "attend":
        q = torch.randn(T, H * G, D, generator=g, device=DEVICE)
        s["q"] = (q / chan[0].reshape(1, H, 1, D).expand(T, H, G, D).reshape(T, -1, D)).to(torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(D)
        s["masks"] = _tree(s, _parents(lens, g), s["kv_lens"])[0]
    else:
        # the accepted path: its first tokens at their places already, the others from behind the last place kept
        s["counts"] = _ints([min(case["kept"], n) for _, n in lens])
        kept = torch.zeros(len(lens), case["kept"], dtype=torch.int32, device=DEVICE)
        for b, (_, n) in enumerate(lens):
            m = min(case["kept"], n)
            far = min(m - 1, n - m)
            kept[b, :m - far] = torch.arange(m - far, device=DEVICE)
            kept[b, m - far:m] = m + torch.sort(torch.randperm(n - m, generator=g, device=DEVICE)[:far])[0]
        s["kept"] = kept
    if own:
        import fp8_kv_cache_sz_amd as sz
        kind = {"bf16": sz.BF16, "e5m2": sz.E5M2, "e4m3": sz.E4M3}[dtype]
        s["caches"] = [sz.PagedCache(kind, data, scales) for data, scales in s["layers"]]
        s["batch"] = sz.PageBatch(table, s["kv_lens"], s["starts"], T, max_new=s["max_new"], max_kv=s["max_kv"])
        if op == "rotary":
            s["rotary"] = sz.Rotary(s["frequencies"], interleaved=case["layout"] == "interleaved",
                                    amplitude=s["amplitude"])
        elif op == "attend":
            s["ws"] = sz.attention_workspace(s["caches"][0], s["batch"], H * G)
        else:
            s["caches"] = sz.CacheLayers(s["caches"])
    return s


def _prepare_pool(s, lens, kv, g):
    """A ring of free pages, and sequences of which one in 32 is done (length
    0, its pages go back); with `short` the ring does not hold enough."""
    case = s["case"]
    P, seqs = case["page"], len(lens)
    done = [b % 32 == 31 and case["past"] > 0 for b in range(seqs)]
    held = [-(-p // P) for p, _ in lens]
    need = [0 if d else -(-x // P) for d, x in zip(done, kv)]
    take = sum(max(0, n - h) for n, h in zip(need, held))
    count = take * 2 // 3 if case["short"] else take + 5
    pages = sum(held) + count + 2
    order = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    head = int(torch.randint(0, pages, (1,), generator=g, device=DEVICE))
    queue = torch.full((pages,), -1, dtype=torch.int32, device=DEVICE)
    queue[(head + torch.arange(count, device=DEVICE)) % pages] = order[:count]
    width = max(max(need), max(held), 1)
    w = torch.arange(width, device=DEVICE)
    h = _ints(held)
    at = count + torch.cumsum(h, 0) - h
    table = torch.where(w < h[:, None], order[(at[:, None] + w).clamp_max(pages - 1)], -1)
    new = [0 if d else n for d, (_, n) in zip(done, lens)]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s.update(table=table, queue=queue, ends=_ints([head, count]), held=h, pages=pages, tokens=starts[-1],
             kv_lens=_ints([0 if d else x for d, x in zip(done, kv)]), starts=_ints(starts), max_new=max(new),
             held_out=torch.zeros_like(h), ends_out=_ints([0, 0]),
             slots=torch.zeros(starts[-1], dtype=torch.int64, device=DEVICE))
    if own:
        import fp8_kv_cache_sz_amd as sz
        s["pool"] = sz.PagePool(P, queue, s["ends"])
        s["batch"] = sz.PageBatch(table, s["kv_lens"], s["starts"], s["tokens"], max_new=s["max_new"], max_kv=width * P)
        s["ws"] = sz.assign_workspace(s["batch"])


def _frequencies(case):
    """base**(-2i / R) in 64 bits; scaled: wavelengths that a context of 8,192
    holds less than once are 8 times as long, those that it holds over four
    times as they were, and a blend between."""
    R = case["rotated"]
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    if case["scaled"]:
        keep = ((8192.0 * f / (2 * math.pi) - 1.0) / 3.0).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / 8.0)
    return f.to(DEVICE)


def run(state):
    op = state["case"]["op"]
    if own:
        import fp8_kv_cache_sz_amd as sz
        if op == "assign":
            sz.pages_assign(state["pool"], state["batch"], state["held"], held_out=state["held_out"],
                            ends_out=state["ends_out"], slots=state["slots"], ws=state["ws"], check=False)
            return _assigned(state)
        if op == "tree":
            return sz.draft_tree(state["batch"], state["parents"], check=False)
        if op == "rotary":
            q = sz.rotary_write(state["caches"][0], state["batch"], state["rotary"], state["q"], state["k"], state["v"],
                                positions=state["positions"], check=False)
            return [q] + _contents(state)
        if op == "attend":
            return sz.tree_attention(state["q"], state["caches"][0], state["batch"], state["masks"],
                                     scale=state["scale"], window=state["case"]["window"], lse=True, ws=state["ws"],
                                     check=False)
        sz.cache_keep(state["caches"], state["batch"], state["kept"], state["counts"], check=False)
        return _contents(state)
    if op == "assign":
        _plain_assign(state)
        return _assigned(state)
    if op == "tree":
        return _tree(state, state["parents"], state["kv_lens"])
    if op == "rotary":
        return [_plain_rotary(state)] + _contents(state)
    if op == "attend":
        return _plain_attend(state)
    _plain_keep(state)
    return _contents(state)


def _contents(state):
    return [t for layer in state["layers"] for t in layer if t is not None]


def _assigned(state):
    return [state["table"], state["queue"], state["held_out"], state["ends_out"], state["slots"]]


# ---- plain forms -----------------------------------------------------------

def _tokens(state):
    """Each new token's sequence, its index there, and that index's place."""
    starts = state["starts"].long()
    t = torch.arange(state["tokens"], device=DEVICE)
    b = torch.searchsorted(starts, t, right=True) - 1
    return b, t - starts[b], state["kv_lens"].long()[b] - starts[b + 1] + t


def _plain_assign(state):
    """Sequences take free pages from the ring's head in their order, as far
    as they go round; pages that a sequence no longer needs go to its end."""
    P, pages = state["case"]["page"], state["pages"]
    table, queue = state["table"], state["queue"]
    held, lens = state["held"].long(), state["kv_lens"].long()
    head, count = state["ends"].long()
    need = (lens + P - 1) // P
    take, give = (need - held).clamp_min(0), (held - need).clamp_min(0)
    upto = take.cumsum(0)
    served = upto <= count
    w = torch.arange(table.shape[1], device=DEVICE)
    fresh = (w >= held[:, None]) & (w < need[:, None])
    at = (head + (upto - take)[:, None] + w - held[:, None]) % pages
    new_table = torch.where(fresh, torch.where(served[:, None], queue[at], -1), table)
    back = (w >= need[:, None]) & (w < held[:, None])
    to = (head + count + (give.cumsum(0) - give)[:, None] + w - need[:, None]) % pages
    queue[to[back]] = table[back]
    table.copy_(new_table)
    state["held_out"].copy_(torch.where(served | (take == 0), need, held))
    taken = (take * served).sum()
    state["ends_out"].copy_(torch.stack([(head + taken) % pages, count - taken + give.sum()]))
    b, _, pos = _tokens(state)
    page = table[b, pos // P].long()
    state["slots"].copy_(torch.where(page >= 0, page * P + pos % P, -1))


def _ancestors(state, parents):
    """[B, n, n]: which tokens of its sequence are above a token, itself included."""
    n, T = state["max_new"], state["tokens"]
    starts = state["starts"].long()
    i = torch.arange(n, device=DEVICE)
    there = i < (starts[1:] - starts[:-1])[:, None]
    up = torch.where(there, parents.long()[(starts[:-1, None] + i).clamp_max(T - 1)], -1)
    seen = torch.eye(n, dtype=torch.bool, device=DEVICE).repeat(len(up), 1, 1)
    for _ in range(max(1, (n - 1).bit_length())):                            # twice as far up each time
        ok = up >= 0
        at = up.clamp_min(0)
        seen = seen | (seen.gather(1, at[..., None].expand(-1, -1, n)) & ok[..., None])
        up = torch.where(ok, up.gather(1, at), -1)
    return seen


def _tree(state, parents, kv_lens):
    """(masks [tokens, words], positions [tokens]) of the trees."""
    seen = _ancestors(state, parents)
    b, i, _ = _tokens({**state, "kv_lens": kv_lens})
    mine = seen[b, i]                                                        # [tokens, n]
    words = -(-mine.shape[1] // 64)
    bits = torch.nn.functional.pad(mine, (0, 64 * words - mine.shape[1])).reshape(len(mine), words, 64).long()
    masks = (bits << torch.arange(64, device=DEVICE)).sum(-1)
    new = (state["starts"][1:] - state["starts"][:-1]).long()
    positions = kv_lens.long()[b] - new[b] + mine.sum(-1) - 1
    return masks, positions.to(torch.int32)


def _pow2(k):
    """2.0**k for whole k in -126..127, from its bits."""
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _turned(x, cos, sin, case):
    """x [T, heads, D] with its first R values turned by [T, R / 2] angles."""
    R = case["rotated"]
    if case["layout"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
    else:
        a, b = x[..., :R:2], x[..., 1:R:2]
    u, v = a * cos - b * sin, b * cos + a * sin
    out = torch.cat([u, v], -1) if case["layout"] == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([out, x[..., R:]], -1)


def _plain_rotary(state):
    case = state["case"]
    b, _, pos = _tokens(state)
    at = pos if state["positions"] is None else state["positions"].long()
    angle = at.double()[:, None, None] * state["frequencies"]
    cos, sin = angle.cos() * state["amplitude"], angle.sin() * state["amplitude"]
    q = _turned(state["q"].float(), cos.float(), sin.float(), case).to(torch.bfloat16)
    # keys in 64 bits: their row's scale depends on which side of a border its largest value is
    k = _turned(state["k"].double(), cos, sin, case).float()
    page, row = state["table"].long()[b, pos // case["page"]], pos % case["page"]
    x = torch.stack([k, state["v"].float()], 1)                              # [T, 2, H, D]
    if case["dtype"] == "bf16":
        state["data"][page, :, :, row] = x.to(torch.bfloat16)
        return q
    bits = x.abs().amax(-1).view(torch.int32)
    e = (bits >> 23) - 127 - FP8_MAX_EXP[case["dtype"]] + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    e = e.clamp_min(-126)
    y = (x * _pow2(-e).unsqueeze(-1)).to(FP8[case["dtype"]])
    state["data"].view(torch.uint8)[page, :, :, row] = y.view(torch.uint8)
    state["scales"][page, :, :, row] = (e + 127).to(torch.uint8)
    return q


def _plain_attend(state):
    """All sequences at once, padded to the longest."""
    case = state["case"]
    B, H, G, D, P = case["seqs"], case["kv_heads"], case["group"], case["head_dim"], case["page"]
    n, keys, T = state["max_new"], state["max_kv"], state["tokens"]
    starts, lens = state["starts"].long(), state["kv_lens"].long()
    new = starts[1:] - starts[:-1]
    past = lens - new
    j = torch.arange(keys, device=DEVICE)
    inside = j < lens[:, None]                                               # [B, keys]
    page = torch.where(inside, state["table"].long()[:, j // P], 0)
    row = (j % P).expand(B, keys)
    if state["scales"] is None:
        kv = state["data"][page, :, :, row].float()                          # [B, keys, 2, H, D]
    else:
        kv = state["data"].view(torch.uint8)[page, :, :, row].view(state["data"].dtype).float()
        kv *= _pow2(state["scales"][page, :, :, row].int() - 127).unsqueeze(-1)
    k = kv[:, :, 0].permute(0, 2, 3, 1).contiguous()                         # [B, H, D, keys]
    v = torch.where(inside[:, None, :, None], kv[:, :, 1].permute(0, 2, 1, 3), 0.0)      # [B, H, keys, D]
    del kv
    i = torch.arange(n, device=DEVICE)
    at = (starts[:-1, None] + i).clamp_max(T - 1)                            # [B, n] token of each padded row
    masks = state["masks"][at]                                               # [B, n, words]
    bits = ((masks[..., None] >> torch.arange(64, device=DEVICE)) & 1).flatten(-2)       # [B, n, 64 words]
    bits = bits.bool() & (torch.arange(bits.shape[-1], device=DEVICE) < new[:, None, None])
    node = j - past[:, None]                                                 # [B, keys] index among the new tokens
    seen = bits.gather(2, node.clamp(0, bits.shape[-1] - 1)[:, None].expand(B, n, keys)) & (node >= 0)[:, None]
    before = (node < 0)[:, None].expand(B, n, keys)
    if case["window"]:
        named = bits.sum(-1).clamp_min(1)
        before = before & (j >= (past[:, None] + named - case["window"])[..., None])
    seen = (seen | before) & inside[:, None]
    q = state["q"][at].float().reshape(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    s = torch.matmul(q, k).mul_(state["scale"]).reshape(B, H, n, G, keys)
    del k
    s = s.masked_fill_(~seen[:, None, :, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, H, n * G, keys), v).reshape(B, H, n, G, D) / torch.where(l == 0, 1.0, l)
    lse = (m + l.log()).squeeze(-1)
    b, i, _ = _tokens(state)
    return o[b, :, i].reshape(T, H * G, D).to(torch.bfloat16), lse[b, :, i].reshape(T, H * G)


def _plain_keep(state):
    """Every kept row is read before any is written."""
    P = state["case"]["page"]
    starts, lens = state["starts"].long(), state["kv_lens"].long()
    past = lens - (starts[1:] - starts[:-1])
    k = torch.arange(state["kept"].shape[1], device=DEVICE)
    b, k = torch.nonzero(k < state["counts"][:, None], as_tuple=True)
    table = state["table"].long()
    src, dst = past[b] + state["kept"].long()[b, k], past[b] + k
    from_page, to_page = table[b, src // P], table[b, dst // P]
    for data, scales in state["layers"]:
        raw = data if scales is None else data.view(torch.uint8)
        raw[to_page, :, :, dst % P] = raw[from_page, :, :, src % P]
        if scales is not None:
            scales[to_page, :, :, dst % P] = scales[from_page, :, :, src % P]


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    lens = _lengths(case)
    op = case["op"]
    T = sum(n for _, n in lens)
    if op == "assign":
        P, moved, tokens = case["page"], 0, 0
        for b, (p, n) in enumerate(lens):
            done = b % 32 == 31 and case["past"] > 0
            moved += abs((0 if done else -(-(p + n) // P)) - -(-p // P))
            tokens += 0 if done else n
        return {"bytes": 16 * len(lens) + 8 * moved + 8 * tokens, "flops": tokens}
    if op == "tree":
        words = -(-max(n for _, n in lens) // 64)
        return {"bytes": 8 * len(lens) + T * (8 + 8 * words), "flops": T * words}
    H, D, G = case["kv_heads"], case["head_dim"], case["group"]
    row = 2 * H * (2 * D if case["dtype"] == "bf16" else D + 1)               # one token's K and V in the cache
    if op == "rotary":
        return {"bytes": T * (row + 4 * H * D + 4 * H * G * D + (4 if _drafted(case) else 0)) + 8 * len(lens),
                "flops": 3 * T * H * (G + 1) * case["rotated"]}
    if op == "keep":
        moved = 0
        for _, n in lens:
            m = min(case["kept"], n)
            moved += min(m - 1, n - m)
        return {"bytes": case["layers"] * moved * 2 * row + 4 * case["kept"] * len(lens) + 12 * len(lens), "flops": 0}
    w, keys, pairs = case["window"], 0, 0
    for past, n in lens:
        seen = min(past, max(0, w - 1)) if w else past                       # the fewest new ones seen: one
        keys += seen + n
        pairs += n * (seen + min(n, 4))                                      # a tree of some depth
    words = -(-case["new"] // 64)
    return {"bytes": keys * row + T * (H * G * (4 * D + 4) + 8 * words), "flops": 4 * D * H * G * pairs}


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
    if case["op"] in ("assign", "tree", "keep"):
        return None                                                          # whole numbers, and rows moved as they are
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    table, lens, starts = s["table"].tolist(), s["kv_lens"].tolist(), s["starts"].tolist()
    return _exact_rotary(case, s, table, lens, starts) if case["op"] == "rotary" else _exact_attend(case, s, table, lens,
                                                                                                   starts)


def _exact_rotary(case, s, table, lens, starts):
    P, R = case["page"], case["rotated"]
    out = s["q"].double()
    data = s["data"].double()
    f = s["frequencies"].cpu()
    for b, n in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        pos = torch.arange(n - (hi - lo), n)
        at = pos.double() if s["positions"] is None else s["positions"][lo:hi].double().cpu()
        turn = torch.polar(torch.full((hi - lo, len(f)), s["amplitude"], dtype=torch.float64), torch.outer(at, f))
        turn = turn.to(DEVICE)[:, None]

        def rotated(x):
            x = x.double()
            a = x[..., :R].reshape(*x.shape[:2], *((2, R // 2) if case["layout"] == "half" else (R // 2, 2)))
            a = a if case["layout"] == "half" else a.transpose(-1, -2)
            z = torch.complex(a[..., 0, :].contiguous(), a[..., 1, :].contiguous()) * turn
            y = torch.stack([z.real, z.imag], -1 if case["layout"] == "interleaved" else -2).reshape(*x.shape[:2], R)
            return torch.cat([y, x[..., R:]], -1)

        out[lo:hi] = rotated(s["q"][lo:hi])
        x = torch.stack([rotated(s["k"][lo:hi]), s["v"][lo:hi].double()], 1)
        page = torch.tensor(table[b], device=DEVICE)[(pos // P).to(DEVICE)]
        row = (pos % P).to(DEVICE)
        if s["scales"] is not None:
            top = 1.75 * 2.0 ** FP8_MAX_EXP[case["dtype"]]
            m, e = torch.frexp(x.abs().amax(-1, keepdim=True) / top)         # m 2**e, m in [1/2, 1)
            x = _rounded(x / _power(torch.where(m == 0.5, e - 1, e).clamp_min(-126)), case["dtype"])
        data[page, :, :, row] = x
    return [out, data] + ([] if s["scales"] is None else [None])


def _exact_attend(case, s, table, lens, starts):
    H, G, D, P, w = case["kv_heads"], case["group"], case["head_dim"], case["page"], case["window"]
    if 4 * D * H * G * sum((b - a) * n for a, b, n in zip(starts, starts[1:], lens)) > 4e12:
        return None
    out = torch.empty(s["tokens"], H * G, D, dtype=torch.float64, device=DEVICE)
    lse = torch.empty(s["tokens"], H * G, dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(lens):
        pages = torch.tensor(table[b], device=DEVICE)[:-(-n // P)]
        x = s["data"].view(torch.uint8 if s["scales"] is not None else torch.bfloat16)[pages]
        x = x.view(s["data"].dtype).double()
        if s["scales"] is not None:
            x = x * _power(s["scales"][pages].long() - 127).unsqueeze(-1)
        x = x.permute(0, 3, 1, 2, 4).reshape(-1, 2, H, D)[:n]
        lo, hi = starts[b], starts[b + 1]
        past = n - (hi - lo)
        hidden = torch.ones(hi - lo, n, dtype=torch.bool)
        for i, row in enumerate(s["masks"][lo:hi].tolist()):
            named = [64 * at + bit for at, word in enumerate(row) for bit in range(64) if word >> bit & 1]
            named = [j for j in named if j < hi - lo]
            hidden[i, max(0, past + max(1, len(named)) - w) if w else 0:past] = False
            hidden[i, [past + j for j in named]] = False
        hidden = hidden.to(DEVICE)[:, None]
        for h in range(H):
            K, V = x[:, 0, h].contiguous(), x[:, 1, h].contiguous()
            q = s["q"][lo:hi, h * G:(h + 1) * G].double()
            z = (q.reshape(-1, D) @ K.T.contiguous() * s["scale"]).reshape(hi - lo, G, n)
            z = z.masked_fill(hidden, float("-inf"))
            r = torch.logsumexp(z, -1)
            e = torch.exp(z - r.unsqueeze(-1))
            out[lo:hi, h * G:(h + 1) * G] = (e.reshape(-1, n) @ V).reshape(hi - lo, G, D)
            lse[lo:hi, h * G:(h + 1) * G] = r
    return out, lse
